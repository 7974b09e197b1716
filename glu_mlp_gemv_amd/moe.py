"""Python face of include/glu_moe.h: a mixture-of-experts GLU layer for a few tokens.

As in ``fp8``, only argument marshalling happens here, and with ``stream`` the work runs there and the tensors given are
recorded on it.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import fp8
from .adapters import _CODES, _TYPES, _scratch, _stack
from .api import _raise_for, library
from .fp8 import (DTYPES, E4M3, _bytes, _matrix, _on, _output, _ptr, _refuse, _refuse_tangents, _rows, _taken,
                  _wants_gradient, groups)

MAX_EXPERTS = 1024
MAX_TOP = 32


class Matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("stack", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("scale_stack", ctypes.c_int64), ("scale_ld", ctypes.c_int64)]


class Sizes(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("M", "K", "N", "E", "top")]


@functools.lru_cache(maxsize=256)
def _workspace(*sizes) -> int:
    return _bytes("glu_moe_workspace", ctypes.byref(Sizes(*sizes)))


def _experts(name: str, w, scale, dtype, shape, dev) -> Matrix:
    strides = _stack(name, w, dtype, shape, dev)
    if dtype is not E4M3:
        if scale is not None:
            raise ValueError(f"{name}_scale without e4m3 weights")
        return Matrix(w.data_ptr(), None, *strides, 0, 0)
    E, rows, cols = shape
    return Matrix(w.data_ptr(), _ptr(scale), *strides,
                  *_stack(name + "_scale", scale, torch.float32, (E, groups(rows), groups(cols)), dev))


def moe_glu(x: torch.Tensor, logits: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, top: int,
            normalize: bool = True, gate_scale: Optional[torch.Tensor] = None, up_scale: Optional[torch.Tensor] = None,
            down_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """sum over the ``top`` experts e of each row of p[e] * (silu(x @ gate[e].T) * (x @ up[e].T)) @ down[e].T.

    x [M, K] bf16 or fp16; logits [M, E] in fp32 or x's type; gate and up [E, N, K], down [E, K, N] in x's type, or e4m3
    with one fp32 scale per 128 x 128 block ([E, N / 128, K / 128], [E, K / 128, N / 128], rounded up), as
    ``fp8_quantize_weight`` gives them per expert.  A row's experts are those of its largest logits, of equal ones
    the lowest; p is the softmax over them, or with ``normalize=False`` over all experts.  -inf masks an expert: a row whose
    logits are all -inf is 0.  Sums and the activation are fp32 (the second product takes it as two 16-bit numbers, in fp32's range), the
    result is rounded once.

    Each chosen expert's gate and up are read once per 64 rows, down once per 32 rows of its own or fewer: meant for the tokens of
    a decode step, right for any number.  At most 1024 experts, 32 per row.  Has no gradient: operands that require one are refused where autograd records.
    """
    if out is None and stream is None:
        r = (fp8._fast or fp8._load_fast()).moe(x, logits, gate, up, down, top, normalize is True or bool(normalize), gate_scale,
                                                up_scale, down_scale)
        if _taken(r):
            return r
    _refuse_tangents("moe_glu", x, logits, gate, up, down, gate_scale, up_scale, down_scale)
    if _wants_gradient(x, logits, gate, up, down, gate_scale, up_scale, down_scale):
        raise RuntimeError("moe_glu has no gradient, and an operand requires one: call it under torch.no_grad()")
    M, K, dev = _matrix("x", x, _TYPES)
    dt = x.dtype
    ldx = _rows("x", x, dt, M, K, dev)
    _refuse("logits", logits, (torch.float32, dt), (M, None), dev)
    E = logits.shape[1]
    ldl = _rows("logits", logits, logits.dtype, M, E, dev)
    if not 1 <= E <= MAX_EXPERTS or not 1 <= top <= min(E, MAX_TOP):
        raise ValueError(f"1 to {MAX_EXPERTS} experts and 1 to {MAX_TOP} of them per row, got {E} and {top}")
    wt = getattr(gate, "dtype", None)
    if wt is not E4M3:
        wt = dt
    _refuse("gate", gate, (dt, E4M3), (E, None, K), dev)
    N = gate.shape[1]
    mats = [_experts("gate", gate, gate_scale, wt, (E, N, K), dev), _experts("up", up, up_scale, wt, (E, N, K), dev),
            _experts("down", down, down_scale, wt, (E, K, N), dev)]
    need = _workspace(M, K, N, E, top)
    ctx, handle = _on(dev, stream, x, logits, gate, up, down, gate_scale, up_scale, down_scale, out)
    with ctx:
        out, ldo = _output("out", out, dt, M, K, dev)
        ws = _scratch(need, dev)
        st = library().glu_moe_glu(x.data_ptr(), ldx, logits.data_ptr(), ldl, DTYPES[logits.dtype], *mats, out.data_ptr(),
                                   ldo, Sizes(M, K, N, E, top), int(normalize), _CODES[dt], DTYPES[wt], _ptr(ws), need,
                                   handle)
    if st:
        _raise_for(st)
    return out


def moe_logits(x: torch.Tensor, router: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """x @ router.T in fp32, [M, E]: the logits of ``moe_glu``, not rounded to x's type, which would change their order.

    x [M, K] and router [E, K], both bf16 or fp16.  Has no gradient: operands that require one are refused where autograd
    records.
    """
    _refuse_tangents("moe_logits", x, router)
    if _wants_gradient(x, router):
        raise RuntimeError("moe_logits has no gradient, and an operand requires one: call it under torch.no_grad()")
    M, K, dev = _matrix("x", x, _TYPES)
    dt = x.dtype
    ldx = _rows("x", x, dt, M, K, dev)
    _refuse("router", router, (dt,), (None, K), dev)
    E = router.shape[0]
    ldr = _rows("router", router, dt, E, K, dev)
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, got {E}")
    ctx, handle = _on(dev, stream, x, router)
    with ctx:
        out = torch.empty(M, E, dtype=torch.float32, device=dev)
        st = library().glu_moe_logits(x.data_ptr(), ldx, router.data_ptr(), ldr, out.data_ptr(), M, K, E, _CODES[dt], handle)
    if st:
        _raise_for(st)
    return out


def _declare(lib):
    """Argument types of include/glu_moe.h (called once by ``api.library``)."""
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    mp, sp = ctypes.POINTER(Matrix), ctypes.POINTER(Sizes)
    for name, args in {
        "glu_moe_glu": [vp, i64, vp, i64, i32, mp, mp, mp, vp, i64, sp, i32, i32, i32, vp, i64, vp],
        "glu_moe_workspace": [sp, ctypes.POINTER(i64)],
        "glu_moe_logits": [vp, i64, vp, i64, vp, i64, i64, i64, i32, vp],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
