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
DPL_MAX_NORM_DIM = 8192
DPL_GROUP = 32

# every exported symbol of dplayer.h
EXPORTS = ("dpl_embed", "dpl_embed_workspace", "dpl_accumulate_embed", "dpl_block_norm", "dpl_block_norm_workspace",
           "dpl_accumulate_block_norm", "dpl_pack_activations", "dpl_unpack_activations",
           "dpl_linear_workspace", "dpl_accumulate_linear")


class Table(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_int32), ("id_bytes", ctypes.c_int32), ("dim", ctypes.c_int64),
                ("scale", ctypes.c_double)]


class Norms(ctypes.Structure):
    _fields_ = [("post_w", ctypes.c_int32), ("post_b", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("pre_w", ctypes.c_int32), ("pre_b", ctypes.c_int32), ("centered", ctypes.c_int32),
                ("dim", ctypes.c_int64), ("eps", ctypes.c_double), ("residual_scale", ctypes.c_double)]


class NormRows(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("s", "y", "dx", "ds", "dh", "dy")]


@dataclass(frozen=True)
class BlockNorm:
    """The norms around a block (``dpl_norms``): plan tensors of the weights,
    biases and the gate, None where there is none."""
    pre_w: Optional[int] = None
    pre_b: Optional[int] = None
    post_w: Optional[int] = None
    post_b: Optional[int] = None
    gate: Optional[int] = None
    centered: bool = False
    eps: float = 1e-5
    residual_scale: float = 1.0

    def struct(self, dim: int) -> Norms:
        at = [-1 if t is None else int(t) for t in (self.post_w, self.post_b, self.gate, self.pre_w, self.pre_b)]
        return Norms(*at, int(self.centered), dim, self.eps, self.residual_scale)


class Linear(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_int32), ("transposed", ctypes.c_int32), ("inputs", ctypes.c_int64),
                ("outputs", ctypes.c_int64)]


class LinearRows(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("codes", "scales", "dy")]


def _register() -> None:
    vp, i32, i64, sz, c_int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    PP, PS = ctypes.POINTER(vp), ctypes.POINTER(sz)
    sig = {
        "dpl_embed": [vp, ctypes.POINTER(Table), i64, vp, c_int, vp, i64, vp],
        "dpl_embed_workspace": [vp, ctypes.POINTER(Table), i64, PS],
        "dpl_accumulate_embed": [vp, ctypes.POINTER(Table), i64, PP, c_int, PP, i64, i32, i32, vp, sz, vp],
        "dpl_block_norm": [vp, ctypes.POINTER(Norms), i64, c_int, vp, i64, vp, i64, vp, i64, vp, i64, vp],
        "dpl_block_norm_workspace": [vp, ctypes.POINTER(Norms), i64, PS],
        "dpl_accumulate_block_norm": [vp, ctypes.POINTER(Norms), i64, c_int, ctypes.POINTER(NormRows), i64, i32, i32,
                                      vp, sz, vp],
        "dpl_pack_activations": [i64, i64, c_int, vp, i64, vp, i64, vp, i64, vp],
        "dpl_unpack_activations": [i64, i64, c_int, vp, i64, vp, i64, vp, i64, vp],
        "dpl_linear_workspace": [vp, ctypes.POINTER(Linear), i64, PS],
        "dpl_accumulate_linear": [vp, ctypes.POINTER(Linear), i64, c_int, ctypes.POINTER(LinearRows), i64, i64, i64,
                                  i32, i32, vp, sz, vp],
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


# ---- norms around a block ----------------------------------------------------------
def dpl_block_norm(plan, norms: BlockNorm, h, y, s, x=None, stream=None) -> None:
    """s = residual_scale * h + gate * N_post(y) and, with a norm before the
    next block, x = N_pre(s)."""
    tokens, dim = h.shape
    lds = [_rows(k, t, tokens, dim, h.dtype) if t is not None else dim
           for k, t in (("h", h), ("y", y), ("s", s), ("x", x))]
    d = norms.struct(dim)
    _check(lib.dpl_block_norm(plan.handle, ctypes.byref(d), tokens, _dtype(h), h.data_ptr(), lds[0], y.data_ptr(),
                              lds[1], s.data_ptr(), lds[2], x.data_ptr() if x is not None else None, lds[3],
                              _stream(stream)))


def dpl_block_norm_workspace(plan, norms: BlockNorm, dim: int, tokens: int) -> int:
    return _query(lib.dpl_block_norm_workspace, plan.handle, ctypes.byref(norms.struct(dim)), tokens)


def dpl_accumulate_block_norm(plan, norms: BlockNorm, s: Optional[Sequence], y: Optional[Sequence],
                              dx: Optional[Sequence], ds: Optional[Sequence], dh: Optional[Sequence],
                              dy: Optional[Sequence], first: bool, workspace, more: bool = False,
                              stream=None) -> None:
    """The backward from every replica's rows: dh, dy, and the gradients of
    the weights and the gate into the accumulators.  None for what is not there
    or not wanted."""
    given = {k: None if v is None else _replicas(plan, k, v)
             for k, v in (("s", s), ("y", y), ("dx", dx), ("ds", ds), ("dh", dh), ("dy", dy))}
    one = next((v[0] for v in given.values() if v is not None), None)
    if one is None:
        raise ValueError("no rows are given")
    tokens, dim = one.shape
    ld = _same_stride("rows", [_rows(k, t, tokens, dim, one.dtype) for k, v in given.items() if v is not None
                               for t in v])
    rows = (NormRows * plan.n)(*[NormRows(*[v[r].data_ptr() if v is not None else None for v in given.values()])
                                 for r in range(plan.n)])
    addr, nbytes = _workspace(workspace)
    d = norms.struct(dim)
    _check(lib.dpl_accumulate_block_norm(plan.handle, ctypes.byref(d), tokens, _dtype(one), rows, ld,
                                         int(bool(first)), int(bool(more)), addr, nbytes, _stream(stream)))


# ---- activations in 8 bits -----------------------------------------------------------
def _packed(codes, scales, tokens: int, dim: int):
    import torch
    return (_rows("codes", codes, tokens, dim, torch.uint8),
            _rows("scales", scales, tokens, -(-dim // DPL_GROUP), torch.uint8))


def dpl_pack_activations(x, codes, scales, stream=None) -> None:
    """x [tokens, dim] as e4m3 bytes, codes [tokens, dim], and a scale byte for
    32 channels, scales [tokens, ceil(dim / 32)]."""
    tokens, dim = x.shape
    ld = _rows("x", x)
    ld_c, ld_s = _packed(codes, scales, tokens, dim)
    _check(lib.dpl_pack_activations(tokens, dim, _dtype(x), x.data_ptr(), ld, codes.data_ptr(), ld_c,
                                    scales.data_ptr(), ld_s, _stream(stream)))


def dpl_unpack_activations(codes, scales, x, stream=None) -> None:
    """The values that codes and scales stand for, into x."""
    tokens, dim = x.shape
    ld = _rows("x", x)
    ld_c, ld_s = _packed(codes, scales, tokens, dim)
    _check(lib.dpl_unpack_activations(tokens, dim, _dtype(x), codes.data_ptr(), ld_c, scales.data_ptr(), ld_s,
                                      x.data_ptr(), ld, _stream(stream)))


def dpl_linear_workspace(plan, tokens: int, inputs: int, outputs: int, tensor: Optional[int] = None) -> int:
    """The bytes for a tensor of inputs x outputs elements (the first such one
    of the plan unless given)."""
    if tensor is None:
        tensor = next((i for i, x in enumerate(plan.numel) if x == inputs * outputs), -1)
    return _query(lib.dpl_linear_workspace, plan.handle, ctypes.byref(Linear(tensor, 0, inputs, outputs)), tokens)


def dpl_accumulate_linear(plan, tensor: int, dy: Sequence, codes: Sequence, scales: Sequence, first: bool,
                          workspace=None, transposed: bool = False, more: bool = False, stream=None) -> None:
    """A linear layer's weight gradient from every replica's output gradients
    dy [tokens, outputs] and packed inputs, into the accumulators of plan tensor
    ``tensor``: outputs x inputs, or inputs x outputs if ``transposed``."""
    import torch
    dy, codes, scales = _replicas(plan, "dy", dy), _replicas(plan, "codes", codes), _replicas(plan, "scales", scales)
    (tokens, outputs), inputs = dy[0].shape, codes[0].shape[1]
    ld_dy = _same_stride("dy", [_rows("dy", t, tokens, outputs, dy[0].dtype) for t in dy])
    ld_c = _same_stride("codes", [_rows("codes", t, tokens, inputs, torch.uint8) for t in codes])
    ld_s = _same_stride("scales", [_rows("scales", t, tokens, -(-inputs // DPL_GROUP), torch.uint8) for t in scales])
    rows = (LinearRows * plan.n)(*[LinearRows(codes[r].data_ptr(), scales[r].data_ptr(), dy[r].data_ptr())
                                   for r in range(plan.n)])
    addr, nbytes = _workspace(workspace)
    d = Linear(tensor, int(bool(transposed)), inputs, outputs)
    _check(lib.dpl_accumulate_linear(plan.handle, ctypes.byref(d), tokens, _dtype(dy[0]), rows, ld_c, ld_s, ld_dy,
                                     int(bool(first)), int(bool(more)), addr, nbytes, _stream(stream)))
