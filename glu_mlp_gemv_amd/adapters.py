"""Python face of include/glu_adapter.h: low-rank adapters of many requests beside a shared projection.

    t[m] = x[m] @ a[i].T,  out[m] = y[m] + scale[i] * (t[m] @ b[i].T)      i = index[m]

a [L, R, K] and b [L, N, R] hold L adapters in the layout of two linear layers' weights, index [M] (int32) names each row's; a
row whose index is not in 0 .. L - 1 has none.  As in ``fp8``, only argument marshalling happens here, and with
``stream`` the work runs there and the tensors given are recorded on it.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from . import fp8
from .api import _raise_for, library
from .fp8 import (_bytes, _matrix, _on, _output, _ptr, _refuse, _refuse_tangents, _rows, _taken, _vector,
                  _wants_gradient)

MAX_RANK = 256
_TYPES = (torch.bfloat16, torch.float16)
_CODES = {torch.bfloat16: 0, torch.float16: 1}


class Adapter(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("a_stack", ctypes.c_int64), ("a_row", ctypes.c_int64),
                ("b_stack", ctypes.c_int64), ("b_row", ctypes.c_int64)]


class Sizes(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("M", "N", "K", "R", "L")]


def _stack(name: str, t, dtype, shape, dev):
    """(matrix stride, row stride) of L matrices with contiguous rows."""
    _refuse(name, t, (dtype,), shape, dev)
    L, rows, cols = shape
    stack, row, one = t.stride()
    if cols > 1 and one != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous, got strides {tuple(t.stride())}")
    if rows <= 1:
        row = cols
    if row < cols or (L > 1 and stack < (rows - 1) * row + cols):
        raise ValueError(f"{name}: rows or adapters overlap (strides {tuple(t.stride())})")
    return stack if L > 1 else rows * row, row


def _adapter(prefix: str, a, b, dtype, K: int, N: int, dev, L=None, R=None):
    """(Adapter, L, R) of a pair of stacks."""
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        _refuse(prefix + "a", a, (dtype,), (None, None, K), dev)
    L, R = a.shape[0] if L is None else L, a.shape[1] if R is None else R
    if L < 1 or not 1 <= R <= MAX_RANK:
        raise ValueError(f"{prefix}a: at least one adapter of rank 1 to {MAX_RANK}, got {tuple(a.shape)}")
    sa = _stack(prefix + "a", a, dtype, (L, R, K), dev)
    sb = _stack(prefix + "b", b, dtype, (L, N, R), dev)
    return Adapter(a.data_ptr(), b.data_ptr(), *sa, *sb), L, R


@functools.lru_cache(maxsize=256)
def _workspace(mats: int, *sizes) -> int:
    return _bytes("glu_adapter_workspace", mats, ctypes.byref(Sizes(*sizes)))


@functools.lru_cache(maxsize=256)
def _grad_workspace(*sizes) -> int:
    return _bytes("glu_adapter_backward_workspace", ctypes.byref(Sizes(*sizes)))


def _scratch(need: int, dev):
    return torch.empty(need // 4, dtype=torch.float32, device=dev) if need else None


def _add(y, x, a, b, index, scale, out, return_low, stream):
    M, N, dev = _matrix("y", y, _TYPES)
    dt = y.dtype
    ldy = _rows("y", y, dt, M, N, dev)
    _, K, _ = _matrix("x", x, (dt,))
    ldx = _rows("x", x, dt, M, K, dev)
    ab, L, R = _adapter("", a, b, dt, K, N, dev)
    _vector("index", index, torch.int32, M, dev)
    if scale is not None:
        _vector("scale", scale, torch.float32, L, dev)
    need = _workspace(1, M, N, K, R, L)
    ctx, handle = _on(dev, stream, y, x, a, b, index, scale, out)
    with ctx:
        out, ldo = _output("out", out, dt, M, N, dev)
        low = torch.empty(M, R, dtype=torch.float32, device=dev) if return_low else None
        ws = _scratch(need, dev)
        st = library().glu_adapter_add(y.data_ptr(), ldy, x.data_ptr(), ldx, ab, index.data_ptr(), _ptr(scale),
                                       out.data_ptr(), ldo, _ptr(low), Sizes(M, N, K, R, L), _CODES[dt], _ptr(ws), need,
                                       handle)
    if st:
        _raise_for(st)
    return out, low


def adapter_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
                scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, return_low: bool = False,
                stream: Optional[torch.cuda.Stream] = None):
    """y + scale[i] * (x @ a[i].T) @ b[i].T per row, i = index[row], rounded once; rows without an adapter are y.

    y [M, N] is what the shared projection of x [M, K] gave; y, x, a [L, R, K] and b [L, N, R] are all bf16 or fp16, index
    [M] int32, scale [L] fp32 (None: 1).  The rank R is 1 to 256; smaller ranks in a stack are padded with zeros.  ``out``
    may be ``y`` (in place).  With ``return_low`` also x @ a[i].T [M, R] in fp32, which ``adapter_backward`` takes.
    Operands that require a gradient have one, through ``autograd.adapter_add``; together with an output, stream or
    ``return_low`` they are refused.
    """
    if out is None and stream is None and not return_low:
        r = (fp8._fast or fp8._load_fast()).adapter(y, x, a, b, index, scale)
        if _taken(r):
            return r
    _refuse_tangents("adapter_add", y, x, a, b, scale)
    if _wants_gradient(y, x, a, b, scale):
        if out is not None or return_low or stream is not None:
            raise RuntimeError("adapter_add with out, return_low or stream has no gradient, and an operand requires one: "
                               "call it without them, or under torch.no_grad()")
        from .autograd import adapter_add as differentiable
        return differentiable(y, x, a, b, index, scale)
    out, low = _add(y, x, a, b, index, scale, out, return_low, stream)
    return (out, low) if return_low else out


def adapter_glu(gate: torch.Tensor, up: torch.Tensor, x: torch.Tensor, gate_a: torch.Tensor, gate_b: torch.Tensor,
                up_a: torch.Tensor, up_b: torch.Tensor, index: torch.Tensor, scale: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """silu(g) * u, where g and u are ``adapter_add`` of gate and of up [M, N] before any rounding; rounded once.

    Both pairs of stacks have the same L and R, and share index and scale.  ``out`` may be ``gate`` or ``up``.  Has no
    gradient: operands that require one are refused where autograd records.
    """
    if out is None and stream is None:
        r = (fp8._fast or fp8._load_fast()).adapter(gate, up, x, gate_a, gate_b, up_a, up_b, index, scale)
        if _taken(r):
            return r
    _refuse_tangents("adapter_glu", gate, up, x, gate_a, gate_b, up_a, up_b, scale)
    if _wants_gradient(gate, up, x, gate_a, gate_b, up_a, up_b, scale):
        raise RuntimeError("adapter_glu has no gradient, and an operand requires one: call it under torch.no_grad(), or "
                           "train with adapter_add on gate and up")
    M, N, dev = _matrix("gate", gate, _TYPES)
    dt = gate.dtype
    ldg, ldu = _rows("gate", gate, dt, M, N, dev), _rows("up", up, dt, M, N, dev)
    _, K, _ = _matrix("x", x, (dt,))
    ldx = _rows("x", x, dt, M, K, dev)
    gab, L, R = _adapter("gate_", gate_a, gate_b, dt, K, N, dev)
    uab, _, _ = _adapter("up_", up_a, up_b, dt, K, N, dev, L, R)
    _vector("index", index, torch.int32, M, dev)
    if scale is not None:
        _vector("scale", scale, torch.float32, L, dev)
    need = _workspace(2, M, N, K, R, L)
    ctx, handle = _on(dev, stream, gate, up, x, gate_a, gate_b, up_a, up_b, index, scale, out)
    with ctx:
        out, ldo = _output("out", out, dt, M, N, dev)
        ws = _scratch(need, dev)
        st = library().glu_adapter_glu(gate.data_ptr(), ldg, up.data_ptr(), ldu, x.data_ptr(), ldx, gab, uab,
                                       index.data_ptr(), _ptr(scale), out.data_ptr(), ldo, Sizes(M, N, K, R, L),
                                       _CODES[dt], _ptr(ws), need, handle)
    if st:
        _raise_for(st)
    return out


def adapter_backward(dout: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
                     low: torch.Tensor, scale: Optional[torch.Tensor] = None,
                     wanted: Sequence[bool] = (True, True, True), stream: Optional[torch.cuda.Stream] = None):
    """(dx, da, db) of ``adapter_add`` for the gradient dout [M, N] of its result (y's gradient is dout itself).

    low is the forward's (``return_low``).  dx has zeros where a row has no adapter, da and db where an adapter has no
    rows.  ``wanted`` says which of the three are computed; the others are None.  Rows are summed in fp32, in an order
    fixed by the sizes and index.
    """
    if stream is None and all(wanted):
        r = (fp8._fast or fp8._load_fast()).adapter_grad(dout, x, a, b, index, low, scale)
        if _taken(r):
            return r
    M, N, dev = _matrix("dout", dout, _TYPES)
    dt = dout.dtype
    ldd = _rows("dout", dout, dt, M, N, dev)
    _, K, _ = _matrix("x", x, (dt,))
    ldx = _rows("x", x, dt, M, K, dev)
    ab, L, R = _adapter("", a, b, dt, K, N, dev)
    _vector("index", index, torch.int32, M, dev)
    _rows("low", low, torch.float32, M, R, dev)
    if not low.is_contiguous():
        raise ValueError("low must be contiguous")
    if scale is not None:
        _vector("scale", scale, torch.float32, L, dev)
    need = _grad_workspace(M, N, K, R, L)
    ctx, handle = _on(dev, stream, dout, x, a, b, index, low, scale)
    with ctx:
        dx, da, db = (torch.empty(s, dtype=dt, device=dev) if w else None
                      for s, w in zip(((M, K), (L, R, K), (L, N, R)), wanted))
        ws = _scratch(need, dev)
        st = library().glu_adapter_backward(dout.data_ptr(), ldd, x.data_ptr(), ldx, ab, index.data_ptr(), _ptr(scale),
                                            low.data_ptr(), _ptr(dx), K, _ptr(da), _ptr(db), Sizes(M, N, K, R, L),
                                            _CODES[dt], _ptr(ws), need, handle)
    if st:
        _raise_for(st)
    return dx, da, db


def _declare(lib):
    """Argument types of include/glu_adapter.h (called once by ``api.library``)."""
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    ap, sp, bp = ctypes.POINTER(Adapter), ctypes.POINTER(Sizes), ctypes.POINTER(ctypes.c_int64)
    tail = [sp, i32, vp, i64, vp]
    for name, args in {
        "glu_adapter_add": [vp, i64, vp, i64, ap, vp, vp, vp, i64, vp] + tail,
        "glu_adapter_glu": [vp, i64, vp, i64, vp, i64, ap, ap, vp, vp, vp, i64] + tail,
        "glu_adapter_workspace": [i32, sp, bp],
        "glu_adapter_backward": [vp, i64, vp, i64, ap, vp, vp, vp, vp, i64, vp, vp] + tail,
        "glu_adapter_backward_workspace": [sp, bp],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
