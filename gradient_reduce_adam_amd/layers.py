"""Binding of the layer operators (``dplayer.h``): forwards that read a plan's
parameters and backwards that write gradients straight into its accumulators.

The functions keep the C names and take torch tensors, whose shapes, types and
row strides are the arguments of the C calls: activations are 2-D ``[tokens,
dim]`` with elements of a row next to each other (``stride(1) == 1``), on the
device that is current.  Arguments given per replica are sequences of the
plan's ``n`` tensors.  A shape, type or device that does not fit raises
``ValueError``; what the library refuses raises :class:`DpError`.  ``plan`` is
a :class:`Plan` (whose methods of the same purpose call these functions).
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

from . import DP_BF16, DP_F16, DP_F32, _check, _stream, lib

DPL_MAX_TOKENS = 1 << 24
DPL_MAX_NORM_DIM = 16384
DPL_GROUP = 32

# every exported symbol of dplayer.h
EXPORTS = ("dpl_embed", "dpl_embed_workspace", "dpl_accumulate_embed")


class Table(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_int32), ("id_bytes", ctypes.c_int32), ("dim", ctypes.c_int64),
                ("scale", ctypes.c_double)]


def _register() -> None:
    vp, i32, i64, sz, c_int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    PP, PS = ctypes.POINTER(vp), ctypes.POINTER(sz)
    sig = {
        "dpl_embed": [vp, ctypes.POINTER(Table), i64, vp, c_int, vp, i64, vp],
        "dpl_embed_workspace": [vp, ctypes.POINTER(Table), i64, PS],
        "dpl_accumulate_embed": [vp, ctypes.POINTER(Table), i64, PP, c_int, PP, i64, i32, i32, vp, sz, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = args


_register()


def _dtype(t) -> int:
    import torch
    code = {torch.bfloat16: DP_BF16, torch.float16: DP_F16, torch.float32: DP_F32}.get(t.dtype)
    if code is None:
        raise ValueError(f"activations are bfloat16, float16 or float32, not {t.dtype}")
    return code


def _here(name: str, t) -> None:
    import torch
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _rows(name: str, t, tokens: Optional[int] = None, dim: Optional[int] = None, dtype=None) -> int:
    """The row stride of an activation tensor, after checking it."""
    _here(name, t)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [tokens, dim] with contiguous rows, not {tuple(t.shape)} of strides "
                         f"{t.stride()}")
    if (tokens is not None and t.shape[0] != tokens) or (dim is not None and t.shape[1] != dim):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected ({tokens}, {dim})")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    # the stride of a single row is never used and may be anything
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _same_stride(name: str, lds: Sequence[int]) -> int:
    if len(set(lds)) > 1:
        raise ValueError(f"{name}: every tensor must have the same row stride, got {sorted(set(lds))}")
    return lds[0]


def _ids(name: str, t, tokens: Optional[int] = None) -> int:
    """The element size of a token id tensor, after checking it."""
    import torch
    _here(name, t)
    if t.dtype not in (torch.int32, torch.int64) or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 or int64 tensor")
    if tokens is not None and t.shape[0] != tokens:
        raise ValueError(f"{name} holds {t.shape[0]} tokens, expected {tokens}")
    return t.element_size()


def _replicas(plan, name: str, xs: Sequence) -> Sequence:
    xs = list(xs)
    if len(xs) != plan.n:
        raise ValueError(f"{name}: {len(xs)} tensors for {plan.n} replicas")
    return xs


def _array(xs: Sequence):
    return (ctypes.c_void_p * len(xs))(*[x.data_ptr() for x in xs])


def _workspace(workspace):
    if workspace is None:
        return None, 0
    _here("workspace", workspace)
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _query(fn, *args) -> int:
    out = ctypes.c_size_t()
    _check(fn(*args, ctypes.byref(out)))
    return out.value


# ---- embedding -----------------------------------------------------------------
def dpl_embed(plan, tensor: int, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * W[ids[t]] from plan tensor ``tensor``, rows of
    ``out.shape[1]`` parameters; zeros for an id outside the table."""
    size = _ids("ids", ids)
    ld = _rows("out", out, ids.shape[0])
    table = Table(tensor, size, out.shape[1], scale)
    _check(lib.dpl_embed(plan.handle, ctypes.byref(table), ids.shape[0], ids.data_ptr(), _dtype(out), out.data_ptr(),
                         ld, _stream(stream)))


def dpl_embed_workspace(plan, tensor: int, dim: int, tokens: int) -> int:
    return _query(lib.dpl_embed_workspace, plan.handle, ctypes.byref(Table(tensor, 8, dim, 1.0)), tokens)


def dpl_accumulate_embed(plan, tensor: int, ids: Sequence, dy: Sequence, first: bool, workspace, scale: float = 1.0,
                         more: bool = False, stream=None) -> None:
    """The lookup's gradient from every replica's token ids and gradient rows,
    into the accumulators of plan tensor ``tensor``."""
    ids, dy = _replicas(plan, "ids", ids), _replicas(plan, "dy", dy)
    tokens, dim = dy[0].shape
    sizes = {_ids("ids", x, tokens) for x in ids}
    if len(sizes) > 1:
        raise ValueError("ids: every replica's must have the same type")
    ld = _same_stride("dy", [_rows("dy", x, tokens, dim, dy[0].dtype) for x in dy])
    table = Table(tensor, sizes.pop(), dim, scale)
    addr, nbytes = _workspace(workspace)
    _check(lib.dpl_accumulate_embed(plan.handle, ctypes.byref(table), tokens, _array(ids), _dtype(dy[0]), _array(dy),
                                    ld, int(bool(first)), int(bool(more)), addr, nbytes, _stream(stream)))
