"""Binding of the layer operators (``dplayer.h``): forwards that read a plan's
parameters and backwards that write gradients straight into its accumulators.

The functions keep the C names and take torch tensors, whose shapes, types and
row strides are the arguments of the C calls: activations are 2-D ``[tokens,
dim]`` with elements of a row next to each other (``stride(1) == 1``), on the
device that is current.  Arguments given per replica are sequences of the
plan's ``n`` tensors.  A shape, type or device that does not fit raises
``ValueError``; what the library refuses raises :class:`DpError`.  ``plan`` is
a :class:`Plan` (whose methods of the same purpose call these functions).
Without torch the workspace queries work, and the other calls raise ImportError.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from typing import Optional, Sequence

try:
    import torch
except ImportError:
    torch = None

from . import DP_BF16, DP_F16, DP_F32, _check, lib

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
    _refs: dict = field(default_factory=dict, init=False, repr=False, compare=False)  # by the rows' width

    def ref(self, dim: int):
        """A reference to the ``dpl_norms`` of these norms on rows of dim elements."""
        if dim not in self._refs:
            at = [-1 if t is None else int(t) for t in (self.post_w, self.post_b, self.gate, self.pre_w, self.pre_b)]
            self._refs[dim] = ctypes.byref(Norms(*at, int(self.centered), dim, self.eps, self.residual_scale))
        return self._refs[dim]

    def __reduce__(self):  # copies and pickles leave the references behind
        return BlockNorm, (self.pre_w, self.pre_b, self.post_w, self.post_b, self.gate, self.centered, self.eps,
                           self.residual_scale)


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
        "dpl_accumulate_block_norm": [vp, ctypes.POINTER(Norms), i64, c_int, vp, i64, i32, i32, vp, sz, vp],
        "dpl_pack_activations": [i64, i64, c_int, vp, i64, vp, i64, vp, i64, vp],
        "dpl_unpack_activations": [i64, i64, c_int, vp, i64, vp, i64, vp, i64, vp],
        "dpl_linear_workspace": [vp, ctypes.POINTER(Linear), i64, PS],
        "dpl_accumulate_linear": [vp, ctypes.POINTER(Linear), i64, c_int, vp, i64, i64, i64, i32, i32, vp, sz, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = args


_register()


if torch is not None:
    _DTYPES = {torch.bfloat16: DP_BF16, torch.float16: DP_F16, torch.float32: DP_F32}
    _IDS = (torch.int32, torch.int64)
    # a launch costs the host about 4 us; the stream's handle without a Stream object saves 2 more
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_device = torch.cuda.current_device
else:
    def _current_device() -> int:
        raise ImportError("the layer operators take torch tensors, and torch cannot be imported")


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype(t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"activations are bfloat16, float16 or float32, not {t.dtype}")
    return code


def _elsewhere(name: str, t, device: int):
    return ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")


def _rows(name: str, t, device: int, tokens: Optional[int] = None, dim: Optional[int] = None, dtype=None) -> int:
    """The row stride of an activation tensor, after checking it."""
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    shape = t.shape
    if len(shape) != 2 or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be [tokens, dim] with contiguous rows, not {tuple(shape)} of strides "
                         f"{t.stride()}")
    if (tokens is not None and shape[0] != tokens) or (dim is not None and shape[1] != dim):
        raise ValueError(f"{name} is {tuple(shape)}, expected ({tokens}, {dim})")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    # the stride of a single row is never used and may be anything
    return t.stride(0) if shape[0] > 1 else shape[1]


def _like(name: str, t, device: int, shape, dtype) -> int:
    """_rows of a tensor whose shape is known: the common case in four look-ups."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == device:
        ld, one = t.stride()
        if one == 1 and shape[0] > 1:
            return ld
    return _rows(name, t, device, shape[0], shape[1], dtype)


def _alike(name: str, ts: Sequence, device: int) -> int:
    """The row stride of tensors that must all be like the first one."""
    first = ts[0]
    shape, dtype, strides = first.shape, first.dtype, first.stride()
    ld = _rows(name, first, device)
    for t in ts:
        if t.stride() != strides or t.shape != shape or t.dtype is not dtype or t.get_device() != device:
            other = _rows(name, t, device, shape[0], shape[1], dtype)
            if other != ld:
                raise ValueError(f"{name}: every tensor must have the same row stride, got {ld} and {other}")
    return ld


def _ids(name: str, t, device: int, tokens: Optional[int] = None) -> int:
    """The element size of a token id tensor, after checking it."""
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    if t.dtype not in _IDS or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 or int64 tensor")
    if tokens is not None and t.shape[0] != tokens:
        raise ValueError(f"{name} holds {t.shape[0]} tokens, expected {tokens}")
    return t.element_size()


def _replicas(plan, name: str, xs: Sequence) -> Sequence:
    xs = tuple(xs)
    if len(xs) != plan.n:
        raise ValueError(f"{name}: {len(xs)} tensors for {plan.n} replicas")
    return xs


def _array(xs: Sequence):
    return (ctypes.c_void_p * len(xs))(*[x.data_ptr() for x in xs])


def _workspace(workspace, device: int):
    if workspace is None:
        return None, 0
    if workspace.get_device() != device:
        raise _elsewhere("the workspace", workspace, device)
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
    dev = _current_device()
    size, tokens = _ids("ids", ids, dev), ids.shape[0]
    ld = _rows("out", out, dev, tokens)
    _check(lib.dpl_embed(plan.handle, ctypes.byref(Table(tensor, size, out.shape[1], scale)), tokens, ids.data_ptr(),
                         _dtype(out), out.data_ptr(), ld, _stream_of(stream, dev)))


def dpl_embed_workspace(plan, tensor: int, dim: int, tokens: int) -> int:
    return _query(lib.dpl_embed_workspace, plan.handle, ctypes.byref(Table(tensor, 8, dim, 1.0)), tokens)


def dpl_accumulate_embed(plan, tensor: int, ids: Sequence, dy: Sequence, first: bool, workspace, scale: float = 1.0,
                         more: bool = False, stream=None) -> None:
    """The lookup's gradient from every replica's token ids and gradient rows,
    into the accumulators of plan tensor ``tensor``."""
    dev = _current_device()
    ids, dy = _replicas(plan, "ids", ids), _replicas(plan, "dy", dy)
    (tokens, dim) = dy[0].shape
    sizes = {_ids("ids", x, dev, tokens) for x in ids}
    if len(sizes) > 1:
        raise ValueError("ids: every replica's must have the same type")
    ld = _alike("dy", dy, dev)
    table = Table(tensor, sizes.pop(), dim, scale)
    addr, nbytes = _workspace(workspace, dev)
    _check(lib.dpl_accumulate_embed(plan.handle, ctypes.byref(table), tokens, _array(ids), _dtype(dy[0]), _array(dy),
                                    ld, bool(first), bool(more), addr, nbytes, _stream_of(stream, dev)))


# ---- norms around a block ----------------------------------------------------------
def dpl_block_norm(plan, norms: BlockNorm, h, y, s, x=None, stream=None) -> None:
    """s = residual_scale * h + gate * N_post(y) and, with a norm before the
    next block, x = N_pre(s)."""
    dev = _current_device()
    (tokens, dim), dtype = h.shape, h.dtype
    ld_h, ld_y, ld_s = _rows("h", h, dev), _like("y", y, dev, h.shape, dtype), _like("s", s, dev, h.shape, dtype)
    ld_x, addr_x = (dim, None) if x is None else (_like("x", x, dev, h.shape, dtype), x.data_ptr())
    _check(lib.dpl_block_norm(plan.handle, norms.ref(dim), tokens, _dtype(h), h.data_ptr(), ld_h, y.data_ptr(), ld_y,
                              s.data_ptr(), ld_s, addr_x, ld_x, _stream_of(stream, dev)))


def dpl_block_norm_workspace(plan, norms: BlockNorm, dim: int, tokens: int) -> int:
    return _query(lib.dpl_block_norm_workspace, plan.handle, norms.ref(dim), tokens)


def dpl_accumulate_block_norm(plan, norms: BlockNorm, s: Optional[Sequence], y: Optional[Sequence],
                              dx: Optional[Sequence], ds: Optional[Sequence], dh: Optional[Sequence],
                              dy: Optional[Sequence], first: bool, workspace, more: bool = False,
                              stream=None) -> None:
    """The backward from every replica's rows: dh, dy, and the gradients of
    the weights and the gate into the accumulators.  None for what is not there
    or not wanted."""
    dev = _current_device()
    given = [None if v is None else _replicas(plan, k, v)
             for k, v in (("s", s), ("y", y), ("dx", dx), ("ds", ds), ("dh", dh), ("dy", dy))]
    there = [t for v in given if v is not None for t in v]
    if not there:
        raise ValueError("no rows are given")
    one = there[0]
    ld = _alike("rows", there, dev)
    tokens, dim = one.shape
    # the structs of all replicas, a pointer after the other
    rows = (ctypes.c_void_p * (6 * plan.n))(*[None if v is None else v[r].data_ptr() for r in range(plan.n)
                                              for v in given])
    addr, nbytes = _workspace(workspace, dev)
    _check(lib.dpl_accumulate_block_norm(plan.handle, norms.ref(dim), tokens, _dtype(one), rows, ld, bool(first),
                                         bool(more), addr, nbytes, _stream_of(stream, dev)))


# ---- activations in 8 bits -----------------------------------------------------------
def dpl_pack_activations(x, codes, scales, stream=None) -> None:
    """x [tokens, dim] as e4m3 bytes, codes [tokens, dim], and a scale byte for
    32 channels, scales [tokens, ceil(dim / 32)]."""
    dev = _current_device()
    ld = _rows("x", x, dev)
    tokens, dim = x.shape
    _check(lib.dpl_pack_activations(tokens, dim, _dtype(x), x.data_ptr(), ld, codes.data_ptr(),
                                    _like("codes", codes, dev, x.shape, torch.uint8), scales.data_ptr(),
                                    _like("scales", scales, dev, (tokens, -(-dim // DPL_GROUP)), torch.uint8),
                                    _stream_of(stream, dev)))


def dpl_unpack_activations(codes, scales, x, stream=None) -> None:
    """The values that codes and scales stand for, into x."""
    dev = _current_device()
    ld = _rows("x", x, dev)
    tokens, dim = x.shape
    _check(lib.dpl_unpack_activations(tokens, dim, _dtype(x), codes.data_ptr(),
                                      _like("codes", codes, dev, x.shape, torch.uint8), scales.data_ptr(),
                                      _like("scales", scales, dev, (tokens, -(-dim // DPL_GROUP)), torch.uint8),
                                      x.data_ptr(), ld, _stream_of(stream, dev)))


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
    dev = _current_device()
    dy, codes, scales = _replicas(plan, "dy", dy), _replicas(plan, "codes", codes), _replicas(plan, "scales", scales)
    ld_dy, ld_c, ld_s = _alike("dy", dy, dev), _alike("codes", codes, dev), _alike("scales", scales, dev)
    (tokens, outputs), inputs = dy[0].shape, codes[0].shape[1]
    _rows("codes", codes[0], dev, tokens, inputs, torch.uint8)
    _rows("scales", scales[0], dev, tokens, -(-inputs // DPL_GROUP), torch.uint8)
    # the structs of all replicas, a pointer after the other
    rows = (ctypes.c_void_p * (3 * plan.n))(*[t.data_ptr() for xs in zip(codes, scales, dy) for t in xs])
    addr, nbytes = _workspace(workspace, dev)
    _check(lib.dpl_accumulate_linear(plan.handle, ctypes.byref(Linear(tensor, bool(transposed), inputs, outputs)),
                                     tokens, _dtype(dy[0]), rows, ld_c, ld_s, ld_dy, bool(first), bool(more), addr,
                                     nbytes, _stream_of(stream, dev)))
