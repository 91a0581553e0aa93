"""Binding of the distillation loss (``dploss.h``).

Tensors are on the device that is current; a shape, type or device that does
not fit raises ``ValueError``, what the library refuses :class:`DpError`.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

from . import _check, lib
from .layers import _current_device, _dtype, _elsewhere, _rows, _stream_of

try:
    import torch
except ImportError:
    torch = None

DPD_MAX_TOKENS = 1 << 21
DPD_MAX_VOCAB = 1 << 18
DPD_MAX_TOP = 1024

# every exported symbol of dploss.h
EXPORTS = ("dpd_distill",)


class DistillDesc(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_double), ("soft", ctypes.c_double), ("hard", ctypes.c_double),
                ("scale", ctypes.c_double), ("vocab", ctypes.c_int64), ("top", ctypes.c_int32),
                ("id_bytes", ctypes.c_int32)]


@dataclass(frozen=True)
class Distillation:
    """loss = soft temperature^2 KL(teacher || student at the temperature) + hard (cross entropy of the label)."""
    temperature: float = 1.0
    soft: float = 1.0
    hard: float = 0.0


def _register() -> None:
    vp, i64, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.dpd_distill.restype = c_int
    lib.dpd_distill.argtypes = [vp, i64, c_int, vp, i64, c_int, vp, i64, vp, i64, vp, vp, vp, vp,
                                vp, i64, vp]


_register()

_DESC = struct.Struct("ddddqii")


def _line(name: str, t, device: int, tokens: int, dtype) -> int:
    """The address of one value a row, None for none."""
    if t is None:
        return None
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    if t.dtype is not dtype or tuple(t.shape) != (tokens,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {tokens} rows")
    return t.data_ptr()


def dpd_distill(distillation: Distillation, logits, teacher, ids, loss, dlogits=None, total=None, labels=None, weight=None,
                scale: float = 1.0, stream=None) -> None:
    """loss [tokens] (or None) of the logits [tokens, vocab] against the teacher's logits [tokens, top] of the tokens ids
    [tokens, top], and scale * weight[t] times its gradient into dlogits (may be logits).  total [tokens]: the logarithm of
    the teacher's whole sum at the temperature, whose remainder is then one more class.  labels [tokens]: of the type of
    ids."""
    dev = _current_device()
    ld = _rows("logits", logits, dev)
    tokens, vocab = logits.shape
    ld_teacher = _rows("teacher", teacher, dev, tokens)
    top = teacher.shape[1]
    ld_ids = _rows("ids", ids, dev, tokens, top)
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"ids are int32 or int64, not {ids.dtype}")
    at, ld_d = (None, vocab) if dlogits is None else (dlogits.data_ptr(),
                                                      _rows("dlogits", dlogits, dev, tokens, vocab, logits.dtype))
    f32 = torch.float32
    desc = ctypes.create_string_buffer(_DESC.pack(distillation.temperature, distillation.soft, distillation.hard, scale, vocab,
                                                  top, ids.element_size()))
    _check(lib.dpd_distill(ctypes.addressof(desc), tokens, _dtype(logits), logits.data_ptr(), ld, _dtype(teacher),
                           teacher.data_ptr(), ld_teacher, ids.data_ptr(), ld_ids, _line("total", total, dev, tokens, f32),
                           _line("labels", labels, dev, tokens, ids.dtype), _line("weight", weight, dev, tokens, f32),
                           _line("loss", loss, dev, tokens, f32), at, ld_d, _stream_of(stream, dev)))
