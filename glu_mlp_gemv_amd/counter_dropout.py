"""Python face of include/glu_dropout.h: dropout whose mask is computed from a counter and never stored."""
from __future__ import annotations

import ctypes
import operator
from typing import Optional, Union

import torch

from . import fp8
from .api import _raise_for, library
from .fp8 import (DTYPES, _INPUTS, _matrix, _on, _output, _ptr, _refuse_tangents, _rows, _taken, _vector,
                  _wants_gradient)

_WORD = (1 << 64) - 1


def drop_of(p: float) -> int:
    """How many of 65536 draws drop an element."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be 0 to 1, got {p}")
    return round(65536 * p)


def _dropout(x, p, seed, offset, residual, out, stream):
    M, K, dev = _matrix("x", x, _INPUTS)
    dt = x.dtype
    ldx = _rows("x", x, dt, M, K, dev)
    ldr = 0 if residual is None else _rows("residual", residual, dt, M, K, dev)
    drop = drop_of(p)
    at = seed if isinstance(seed, torch.Tensor) else None
    if at is not None:
        _vector("seed", at, torch.int64, 1, dev)
    ctx, handle = _on(dev, stream, x, residual, out, at)
    with ctx:
        out, ldo = _output("out", out, dt, M, K, dev)
        st = library().glu_dropout(x.data_ptr(), ldx, _ptr(residual), ldr, out.data_ptr(), ldo, M, K, drop,
                                   0 if at is not None else operator.index(seed) & _WORD, _ptr(at),
                                   operator.index(offset) & _WORD, DTYPES[dt], handle)
    if st:
        _raise_for(st)
    return out


def dropout(x: torch.Tensor, p: float, seed: Union[int, torch.Tensor], offset: int = 0,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """residual + x with each element dropped with probability p, the others divided by 1 - p; rounded once.

    x and residual [M, K], bf16, fp16 or fp32.  p is applied in steps of 2^-16.  The mask is that of Philox4x32-10 for
    (seed, offset) and an element's row and column, whatever the type and strides: the same call on a gradient is the backward,
    and a layer or step of its own offset has a mask of its own.  seed is a 64-bit int, or an int64 tensor [1] on
    the device that is read when the kernel runs, so that a captured graph can draw anew on each replay.  ``out`` may be ``x``
    or ``residual``.  Operands that require a gradient have one, through ``autograd.dropout``; with an output or
    stream they are refused.
    """
    if out is None and stream is None:
        r = (fp8._fast or fp8._load_fast()).dropout(x, drop_of(p), seed, offset, residual)
        if _taken(r):
            return r
    _refuse_tangents("dropout", x, residual)
    if _wants_gradient(x, residual):
        if out is not None or stream is not None:
            raise RuntimeError("dropout with out or stream has no gradient, and an operand requires one: call it without "
                               "them, or under torch.no_grad()")
        from .autograd import dropout as differentiable
        return differentiable(x, p, seed, offset, residual)
    return _dropout(x, p, seed, offset, residual, out, stream)


def _declare(lib):
    """Argument types of include/glu_dropout.h (called once by ``api.library``)."""
    vp, i64, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64
    lib.glu_dropout.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, u64, vp, u64, ctypes.c_int, vp]
    lib.glu_dropout.restype = ctypes.c_int
