"""Binding of the attention and its positions (``dpattn.h``).

The functions keep the C names and take torch tensors ``[tokens, heads, dim]``
of any row and head strides (views of one projection among them) whose
elements lie next to each other, on the device that is current.  A shape, type
or device that does not fit raises ``ValueError``; what the library refuses
raises :class:`DpError`.  Without torch the workspace query works, and the other
calls raise ImportError.
"""
from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass, field
from typing import Optional, Tuple

from . import DP_BF16, DP_F16, _check, lib
from .layers import _current_device, _dtype, _elsewhere, _query, _stream_of, _workspace

try:
    import torch
except ImportError:
    torch = None

DPA_MAX_TOKENS = 1 << 24
DPA_MAX_HEADS = 1024
DPA_MAX_DIM = 128
DPA_MAX_AXES = 4
DPA_MAX_PAIRS = 256
DPA_MAX_TENSORS = 4

# every exported symbol of dpattn.h
EXPORTS = ("dpa_rotary", "dpa_attention", "dpa_attention_workspace", "dpa_attention_backward")


class Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("ld", ctypes.c_int64), ("head", ctypes.c_int64)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("sections", ctypes.c_int32 * DPA_MAX_AXES), ("interleaved", ctypes.c_int32),
                ("own_ladder", ctypes.c_int32), ("reserved", ctypes.c_int32), ("base", ctypes.c_double)]


class RotaryRows(ctypes.Structure):
    _fields_ = [("x", Rows), ("y", Rows), ("heads", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int64), ("scale", ctypes.c_double),
                ("tokens", ctypes.c_int64), ("tokens_k", ctypes.c_int64), ("sequences", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("offsets_k", ctypes.c_void_p), ("offset_bytes", ctypes.c_int32),
                ("step", ctypes.c_int32)]


@dataclass(frozen=True)
class Rotary:
    """Rotary positions (``dpa_rotary_desc``): the pairs of elements that turn with each axis of a position, (i, i +
    half) or, ``interleaved``, (2 i, 2 i + 1); one ladder of frequencies over all of them, or one for each axis."""
    sections: Tuple[int, ...]
    base: float = 10000.0
    interleaved: bool = False
    own_ladder: bool = False
    _refs: list = field(default_factory=list, init=False, repr=False, compare=False)

    def ref(self):
        """A reference to the ``dpa_rotary_desc``."""
        if not self._refs:
            sections = (ctypes.c_int32 * DPA_MAX_AXES)(*self.sections)
            self._refs.append(ctypes.byref(RotaryDesc(len(self.sections), sections, int(self.interleaved),
                                                      int(self.own_ladder), 0, self.base)))
        return self._refs[0]

    def __reduce__(self):  # copies and pickles leave the reference behind
        return Rotary, (self.sections, self.base, self.interleaved, self.own_ladder)


@dataclass(frozen=True)
class Attention:
    """Which keys a query sees, by its place among them, and the factor of the products (1 / sqrt(dim) unless
    given)."""
    causal: bool = False
    window: int = 0
    scale: Optional[float] = None


def _register() -> None:
    vp, i32, i64, sz, c_int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    sig = {  # descriptions and rows by their addresses
        "dpa_rotary": [vp, i64, i32, vp, i32, i64, i64, i32, vp, c_int, i32, vp],
        "dpa_attention": [vp, c_int, vp, vp, vp, vp, vp, vp],
        "dpa_attention_workspace": [i64, i32, ctypes.POINTER(sz)],
        "dpa_attention_backward": [vp, c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = args


_register()


# A call's structs are packed as bytes, which takes a fifth of the time of a ctypes structure each.
_ROTARY_ROWS = struct.Struct("PqqPqqii")
_ROTARY_CALL = [struct.Struct(_ROTARY_ROWS.format * n) for n in range(DPA_MAX_TENSORS + 1)]
_DESC, _ROWS = struct.Struct("iiiiqdqqqPPii"), struct.Struct("Pqq")
_pack = _ROWS.pack
_POSITION_BYTES = {} if torch is None else {torch.int32: 4, torch.int64: 8}


def _heads(name: str, t, device: int, shape=None, dtype=None):
    """The address and the strides of a tensor of heads, after checking it."""
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    have, strides = t.shape, t.stride()
    if len(have) != 3 or (strides[2] != 1 and have[2] > 1):
        raise ValueError(f"{name} must be [tokens, heads, dim] with contiguous heads, not {tuple(have)} of strides "
                         f"{strides}")
    if shape is not None and have != shape:
        raise ValueError(f"{name} is {tuple(have)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    return t.data_ptr(), strides[0], strides[1]


# ---- positions -----------------------------------------------------------------
def dpa_rotary(rotary: Rotary, positions, x, y, inverse: bool = False, stream=None) -> None:
    """y = x turned by the positions of its rows, or back if ``inverse``.  x and y are a tensor each or sequences of up
    to four of them, with the same rows and their own heads; y may be x.  positions: int32 or int64, ``[tokens, axes]``
    of any strides, or ``[tokens]`` for one axis."""
    dev = _current_device()
    xs, ys = x if isinstance(x, (list, tuple)) else (x,), y if isinstance(y, (list, tuple)) else (y,)
    count, axes = len(xs), len(rotary.sections)
    if count != len(ys) or not 1 <= count <= DPA_MAX_TENSORS:
        raise ValueError(f"{count} tensors x and {len(ys)} tensors y (the same number, up to {DPA_MAX_TENSORS})")
    if not 1 <= axes <= DPA_MAX_AXES:
        raise ValueError(f"{axes} axes (up to {DPA_MAX_AXES})")
    one, rows = xs[0], []
    dtype, first = one.dtype, one.shape
    for a, b in zip(xs, ys):
        shape = a.shape
        rows += (*_heads("x", a, dev, None, dtype), *_heads("y", b, dev, shape, dtype), shape[1], 0)
        if shape[0] != first[0] or shape[2] != first[2]:
            raise ValueError(f"x: {tuple(shape)} beside {tuple(first)}")
    tokens = first[0]
    if positions.get_device() != dev:
        raise _elsewhere("positions", positions, dev)
    bits = _POSITION_BYTES.get(positions.dtype)
    if bits is None:
        raise ValueError(f"positions are int32 or int64, not {positions.dtype}")
    shape, strides = positions.shape, positions.stride()
    if len(shape) == 1 and axes == 1:
        shape, strides = (shape[0], 1), (strides[0], 0)
    if len(shape) != 2 or shape[0] != tokens or shape[1] != axes:
        raise ValueError(f"positions are {tuple(positions.shape)}, expected ({tokens}, {axes})")
    _check(lib.dpa_rotary(rotary.ref(), tokens, first[2], positions.data_ptr(), bits, strides[0], strides[1], count,
                          _ROTARY_CALL[count].pack(*rows), _dtype(one), bool(inverse), _stream_of(stream, dev)))


# ---- attention -----------------------------------------------------------------
def _offsets(name: str, t, device: int):
    """The address, the number of sequences, the size of an offset and the step between the sequences'."""
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    spans = t.dim() == 2 and t.shape[1] == 2
    if t.dtype not in (torch.int32, torch.int64) or not t.is_contiguous() or not (spans or (t.dim() == 1 and t.shape[0])):
        raise ValueError(f"{name} must be a contiguous int32 or int64 tensor [sequences + 1], or [sequences, 2] of begins "
                         "and ends")
    return t.data_ptr(), t.shape[0] if spans else t.shape[0] - 1, t.element_size(), 2 if spans else 1


def _describe(attention: Attention, qs, ks, sequences: Optional[int], offsets, offsets_k, device: int):
    """The dpa_attention_desc of a call whose queries and keys have the shapes qs and ks."""
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError(f"q and k must be [tokens, heads, dim], not {tuple(qs)} and {tuple(ks)}")
    tokens, heads, dim = qs
    tokens_k, kv_heads, dim_k = ks
    if dim_k != dim:
        raise ValueError(f"heads of {dim} elements in q and of {dim_k} in k")
    at, at_k, size, step = 0, 0, 0, 0
    if offsets is not None or offsets_k is not None:
        given = [_offsets(n, t, device) for n, t in (("offsets", offsets), ("offsets_k", offsets_k)) if t is not None]
        if len(given) == 2 and given[0][1:] != given[1][1:]:
            raise ValueError("offsets and offsets_k must have the same type and shape")
        _, count, size, step = given[0]
        if sequences is not None and sequences != count:
            raise ValueError(f"offsets of {count} sequences, expected {sequences}")
        sequences = count
        at = given[0][0] if offsets is not None else 0
        at_k = given[-1][0] if offsets_k is not None else 0
    scale = attention.scale if attention.scale is not None else 1.0 / math.sqrt(max(dim, 1))
    return _DESC.pack(heads, kv_heads, dim, bool(attention.causal), attention.window, scale, tokens, tokens_k,
                      1 if sequences is None else sequences, at, at_k, size, step)


_SIXTEEN = (DP_BF16, DP_F16)


def _attention_dtype(q) -> int:
    code = _dtype(q)
    if code not in _SIXTEEN:
        raise ValueError(f"the attention takes bfloat16 or float16, not {q.dtype}")
    return code


def _lse(lse, qs, device: int) -> int:
    if lse.get_device() != device:
        raise _elsewhere("lse", lse, device)
    have = lse.shape
    if lse.dtype is not torch.float32 or len(have) != 2 or have[0] != qs[1] or have[1] != qs[0] or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of [heads, tokens] = ({qs[1]}, {qs[0]})")
    return lse.data_ptr()


def dpa_attention(attention: Attention, q, k, v, out, lse, sequences: Optional[int] = None, offsets=None, offsets_k=None,
                  stream=None) -> None:
    """out = softmax(scale q k^T) v and the logarithms lse [heads, tokens] of the rows' sums, over the sequences: all
    rows one sequence, or ``sequences`` of one length, or those at ``offsets`` (``[sequences + 1]``, or ``[sequences, 2]``
    of begins and ends; ``offsets_k`` for the keys where they lie elsewhere).  q and out are [tokens, heads, dim], k and v
    [tokens_k, kv_heads, dim]."""
    dev, dtype, qs, ks = _current_device(), q.dtype, q.shape, k.shape
    code, desc = _attention_dtype(q), _describe(attention, qs, ks, sequences, offsets, offsets_k, dev)
    _check(lib.dpa_attention(desc, code, _pack(*_heads("q", q, dev)), _pack(*_heads("k", k, dev, None, dtype)),
                             _pack(*_heads("v", v, dev, ks, dtype)), _pack(*_heads("out", out, dev, qs, dtype)),
                             _lse(lse, qs, dev), _stream_of(stream, dev)))


def dpa_attention_workspace(tokens: int, heads: int) -> int:
    return _query(lib.dpa_attention_workspace, tokens, heads)


def dpa_attention_backward(attention: Attention, q, k, v, out, lse, dout, dq, dk, dv, workspace,
                           sequences: Optional[int] = None, offsets=None, offsets_k=None, stream=None) -> None:
    """The gradients dq, dk and dv of ``dpa_attention`` from dout, with the out and lse that it left."""
    dev, dtype, qs, ks = _current_device(), q.dtype, q.shape, k.shape
    code, desc = _attention_dtype(q), _describe(attention, qs, ks, sequences, offsets, offsets_k, dev)
    rows = [_pack(*_heads(*x)) for x in (("q", q, dev), ("k", k, dev, None, dtype), ("v", v, dev, ks, dtype),
                                         ("out", out, dev, qs, dtype), ("dout", dout, dev, qs, dtype),
                                         ("dq", dq, dev, qs, dtype), ("dk", dk, dev, ks, dtype), ("dv", dv, dev, ks, dtype))]
    addr, nbytes = _workspace(workspace, dev)
    _check(lib.dpa_attention_backward(desc, code, *rows[:4], _lse(lse, qs, dev), *rows[4:], addr, nbytes,
                                      _stream_of(stream, dev)))
