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


# A call's structs are packed into one buffer at once, which takes a third of the time of a ctypes
# structure each: a dpa_rotary_rows, and a dpa_attention_desc with the rows of the call's tensors behind it.
_ROTARY_ROWS = struct.Struct("PqqPqqii")
_DESC = "iiiiqdqqqPPii"
_FORWARD, _BACKWARD = struct.Struct(_DESC + "Pqq" * 4), struct.Struct(_DESC + "Pqq" * 8)
_DESC_BYTES, _ROWS_BYTES = ctypes.sizeof(AttentionDesc), ctypes.sizeof(Rows)


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
    xs, ys = (list(v) if isinstance(v, (list, tuple)) else [v] for v in (x, y))
    if len(xs) != len(ys) or not 1 <= len(xs) <= DPA_MAX_TENSORS:
        raise ValueError(f"{len(xs)} tensors x and {len(ys)} tensors y (the same number, up to {DPA_MAX_TENSORS})")
    one, axes = xs[0], len(rotary.sections)
    if not 1 <= axes <= DPA_MAX_AXES:
        raise ValueError(f"{axes} axes (up to {DPA_MAX_AXES})")
    rows = []
    for a, b in zip(xs, ys):
        rows += (*_heads("x", a, dev, None, one.dtype), *_heads("y", b, dev, a.shape, one.dtype), a.shape[1], 0)
        if a.shape[0] != one.shape[0] or a.shape[2] != one.shape[2]:
            raise ValueError(f"x: {tuple(a.shape)} beside {tuple(one.shape)}")
    tokens, _, dim = one.shape
    if positions.get_device() != dev:
        raise _elsewhere("positions", positions, dev)
    if positions.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"positions are int32 or int64, not {positions.dtype}")
    at = positions.unsqueeze(1) if positions.dim() == 1 else positions
    if tuple(at.shape) != (tokens, axes):
        raise ValueError(f"positions are {tuple(positions.shape)}, expected ({tokens}, {axes})")
    buf = ctypes.create_string_buffer(_ROTARY_ROWS.size * len(xs))
    for i in range(len(xs)):
        _ROTARY_ROWS.pack_into(buf, i * _ROTARY_ROWS.size, *rows[8 * i:8 * i + 8])
    _check(lib.dpa_rotary(rotary.ref(), tokens, dim, at.data_ptr(), at.element_size(), at.stride(0), at.stride(1),
                          len(xs), ctypes.addressof(buf), _dtype(one), bool(inverse), _stream_of(stream, dev)))


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


def _describe(attention: Attention, q, k, sequences: Optional[int], offsets, offsets_k, device: int):
    """The fields of a dpa_attention_desc."""
    if len(q.shape) != 3 or len(k.shape) != 3:
        raise ValueError(f"q and k must be [tokens, heads, dim], not {tuple(q.shape)} and {tuple(k.shape)}")
    tokens, heads, dim = q.shape
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
    return (heads, k.shape[1], dim, bool(attention.causal), attention.window, scale, tokens, k.shape[0],
            1 if sequences is None else sequences, at, at_k, size, step)


_SIXTEEN = (DP_BF16, DP_F16)


def _attention_dtype(q) -> int:
    code = _dtype(q)
    if code not in _SIXTEEN:
        raise ValueError(f"the attention takes bfloat16 or float16, not {q.dtype}")
    return code


def _lse(lse, q, device: int) -> int:
    if lse.get_device() != device:
        raise _elsewhere("lse", lse, device)
    if lse.dtype is not torch.float32 or tuple(lse.shape) != (q.shape[1], q.shape[0]) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of [heads, tokens] = ({q.shape[1]}, {q.shape[0]})")
    return lse.data_ptr()


def dpa_attention(attention: Attention, q, k, v, out, lse, sequences: Optional[int] = None, offsets=None, offsets_k=None,
                  stream=None) -> None:
    """out = softmax(scale q k^T) v and the logarithms lse [heads, tokens] of the rows' sums, over the sequences: all
    rows one sequence, or ``sequences`` of one length, or those at ``offsets`` (``[sequences + 1]``, or ``[sequences, 2]``
    of begins and ends; ``offsets_k`` for the keys where they lie elsewhere).  q and out are [tokens, heads, dim], k and v
    [tokens_k, kv_heads, dim]."""
    dev, dtype = _current_device(), q.dtype
    code, desc = _attention_dtype(q), _describe(attention, q, k, sequences, offsets, offsets_k, dev)
    buf = ctypes.create_string_buffer(_FORWARD.size)
    _FORWARD.pack_into(buf, 0, *desc, *_heads("q", q, dev), *_heads("k", k, dev, None, dtype),
                       *_heads("v", v, dev, k.shape, dtype), *_heads("out", out, dev, q.shape, dtype))
    a = ctypes.addressof(buf)
    r = range(a + _DESC_BYTES, a + _FORWARD.size, _ROWS_BYTES)
    _check(lib.dpa_attention(a, code, *r, _lse(lse, q, dev), _stream_of(stream, dev)))


def dpa_attention_workspace(tokens: int, heads: int) -> int:
    return _query(lib.dpa_attention_workspace, tokens, heads)


def dpa_attention_backward(attention: Attention, q, k, v, out, lse, dout, dq, dk, dv, workspace,
                           sequences: Optional[int] = None, offsets=None, offsets_k=None, stream=None) -> None:
    """The gradients dq, dk and dv of ``dpa_attention`` from dout, with the out and lse that it left."""
    dev, dtype, qs, ks = _current_device(), q.dtype, q.shape, k.shape
    code, desc = _attention_dtype(q), _describe(attention, q, k, sequences, offsets, offsets_k, dev)
    buf = ctypes.create_string_buffer(_BACKWARD.size)
    _BACKWARD.pack_into(buf, 0, *desc, *_heads("q", q, dev), *_heads("k", k, dev, None, dtype),
                        *_heads("v", v, dev, ks, dtype), *_heads("out", out, dev, qs, dtype),
                        *_heads("dout", dout, dev, qs, dtype), *_heads("dq", dq, dev, qs, dtype),
                        *_heads("dk", dk, dev, ks, dtype), *_heads("dv", dv, dev, ks, dtype))
    a = ctypes.addressof(buf)
    r = range(a + _DESC_BYTES, a + _BACKWARD.size, _ROWS_BYTES)
    addr, nbytes = _workspace(workspace, dev)
    _check(lib.dpa_attention_backward(a, code, *r[:4], _lse(lse, q, dev), *r[4:], addr, nbytes, _stream_of(stream, dev)))
