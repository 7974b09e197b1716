"""Python face of include/glu_fp8.h: RMS norm, conversion to block-scaled e4m3, products on it.

As in ``api``, only argument marshalling happens here: tensors are checked, their device pointers
and torch's current HIP stream go to ``libglu_gemv.so``, and a non-OK status becomes a ``GluError``.

Block-scaled e4m3: a stored ``torch.float8_e4m3fn`` value q stands for ``q * scale``.  Activations
[M, K] have an fp32 scale per row and 128 columns, [M, ceil(K / 128)], which the functions here return stored
group by group (``scale.t()`` is contiguous) and accept at any strides; weights [N, K] one per block of
128 x 128, [ceil(N / 128), ceil(K / 128)].

Row-strided views are taken at the stride they report.  With ``stream`` the work runs there and the
results belong to that stream's memory pool; the tensors given are recorded on it.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from .api import _raise_for, _row_stride, library

E4M3 = torch.float8_e4m3fn
GROUP = 128
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, E4M3: 3}
KERNEL_NAMES = ("none", "zero", "stream", "tile", "any")
_NO_CONTEXT = contextlib.nullcontext()


class Matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("scale_row", ctypes.c_int64), ("scale_block", ctypes.c_int64)]


class ProductPlan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("tile", ctypes.c_int), ("width", ctypes.c_int), ("splits", ctypes.c_int),
                ("launches", ctypes.c_int), ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel_name"] = KERNEL_NAMES[self.kernel]
        return d


def groups(n: int) -> int:
    """Scales along a dimension of n."""
    return -(-n // GROUP)


def _tensor(name: str, t, dtypes, ndim: int, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")


_INPUTS = (torch.bfloat16, torch.float16, torch.float32)
_F32 = (torch.float32,)
_E4M3 = (E4M3,)


def _like(name: str, t, shape, dtype, dev):
    """An output of this shape: the one given, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _tensor(name, t, (dtype,), len(shape), dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _row_scales(name: str, t, rows: int, cols: int, dev):
    """A new [rows, groups] scale tensor stored group by group, or the given one, whose columns must be contiguous."""
    if t is None:
        return torch.empty((groups(cols), rows), dtype=torch.float32, device=dev).t()
    _tensor(name, t, _F32, 2, dev)
    if tuple(t.shape) != (rows, groups(cols)):
        raise ValueError(f"{name} must be {(rows, groups(cols))}, got {tuple(t.shape)}")
    _row_stride(name, t.t())
    return t


def _on(dev, stream, *tensors):
    """(context, stream handle) of a call on ``stream`` or the device's current stream."""
    if stream is None:
        ctx = _NO_CONTEXT if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
        return ctx, torch.cuda.current_stream(dev).cuda_stream
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream), stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _norm_args(x, weight, residual, residual_out):
    _tensor("x", x, _INPUTS, 2)
    dev, dt = x.device, x.dtype
    M, K = x.shape
    _tensor("weight", weight, (dt,), 1, dev)
    if weight.shape[0] != K:
        raise ValueError(f"weight must be ({K},), got {tuple(weight.shape)}")
    if K > 1 and weight.stride(0) != 1:
        raise ValueError(f"weight: elements must be contiguous, got stride {weight.stride(0)}")
    if residual is not None:
        _tensor("residual", residual, (dt,), 2, dev)
        if residual.shape != x.shape:
            raise ValueError(f"residual must be {tuple(x.shape)}, got {tuple(residual.shape)}")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    return dev, dt, M, K


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                 return_rstd: bool = False, stream: Optional[torch.cuda.Stream] = None):
    """(y, h): h = x + residual in x's type (x itself without a residual), y = h / rms(h) * weight.

    x and residual [M, K], weight [K], all bf16, fp16 or fp32; rms(h) = sqrt(mean(h^2) + eps) per
    row, in fp32, and y rounded once.  ``residual_out`` may be ``residual`` or ``x`` (in place).  With
    ``return_rstd`` also 1 / rms [M] in fp32, which ``add_rms_norm_backward`` takes.
    """
    dev, dt, M, K = _norm_args(x, weight, residual, residual_out)
    ctx, handle = _on(dev, stream, x, weight, residual, out, residual_out)
    with ctx:
        out = _like("out", out, (M, K), dt, dev)
        h = x if residual is None else _like("residual_out", residual_out, (M, K), dt, dev)
        rstd = torch.empty(M, dtype=torch.float32, device=dev) if return_rstd else None
        has = residual is not None
        st = library().glu_add_rms_norm(
            x.data_ptr(), _row_stride("x", x), _ptr(residual), _row_stride("residual", residual) if has else 0,
            weight.data_ptr(), h.data_ptr() if has else None, _row_stride("residual_out", h) if has else 0,
            out.data_ptr(), _row_stride("out", out), _ptr(rstd), M, K, eps, DTYPES[dt], handle)
    _raise_for(st)
    return (out, h, rstd) if return_rstd else (out, h)


def add_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                     residual_out: Optional[torch.Tensor] = None, return_rstd: bool = False,
                     stream: Optional[torch.cuda.Stream] = None):
    """(q, scale, h): ``add_rms_norm`` with y converted to block-scaled e4m3 before any rounding to x's type."""
    dev, dt, M, K = _norm_args(x, weight, residual, residual_out)
    ctx, handle = _on(dev, stream, x, weight, residual, out, scale_out, residual_out)
    with ctx:
        out = _like("out", out, (M, K), E4M3, dev)
        scale = _row_scales("scale_out", scale_out, M, K, dev)
        h = x if residual is None else _like("residual_out", residual_out, (M, K), dt, dev)
        rstd = torch.empty(M, dtype=torch.float32, device=dev) if return_rstd else None
        has = residual is not None
        st = library().glu_add_rms_norm_fp8(
            x.data_ptr(), _row_stride("x", x), _ptr(residual), _row_stride("residual", residual) if has else 0,
            weight.data_ptr(), h.data_ptr() if has else None, _row_stride("residual_out", h) if has else 0,
            out.data_ptr(), _row_stride("out", out), scale.data_ptr(), scale.stride(1), _ptr(rstd), M, K, eps,
            DTYPES[dt], handle)
    _raise_for(st)
    return (out, scale, h, rstd) if return_rstd else (out, scale, h)


def add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          dresidual: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                          dweight: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(dx, dweight) of ``add_rms_norm`` for the gradient ``dy`` of y and ``dresidual`` of h.

    h and rstd are the forward's.  dx is the gradient of x and of the residual alike.  dweight sums the
    rows in fp32 in a fixed order.  ``dx`` may be ``dresidual`` (in place).
    """
    _tensor("h", h, _INPUTS, 2)
    dev, dt = h.device, h.dtype
    M, K = h.shape
    _tensor("dy", dy, (dt,), 2, dev)
    _tensor("weight", weight, (dt,), 1, dev)
    _tensor("rstd", rstd, _F32, 1, dev)
    if dy.shape != h.shape or weight.shape[0] != K or rstd.shape[0] != M:
        raise ValueError(f"shape mismatch: dy {tuple(dy.shape)}, h {tuple(h.shape)}, weight {tuple(weight.shape)}, "
                         f"rstd {tuple(rstd.shape)}")
    for name, t in (("weight", weight), ("rstd", rstd)):
        if t.shape[0] > 1 and t.stride(0) != 1:
            raise ValueError(f"{name}: elements must be contiguous, got stride {t.stride(0)}")
    if dresidual is not None:
        _tensor("dresidual", dresidual, (dt,), 2, dev)
        if dresidual.shape != h.shape:
            raise ValueError(f"dresidual must be {tuple(h.shape)}, got {tuple(dresidual.shape)}")
    lib = library()
    need = ctypes.c_int64(0)
    _raise_for(lib.glu_add_rms_norm_backward_workspace(M, K, ctypes.byref(need)))
    ctx, handle = _on(dev, stream, dy, h, weight, rstd, dresidual, dx, dweight)
    with ctx:
        dx = _like("dx", dx, (M, K), dt, dev)
        dweight = _like("dweight", dweight, (K,), dt, dev)
        if K > 1 and dweight.stride(0) != 1:
            raise ValueError(f"dweight: elements must be contiguous, got stride {dweight.stride(0)}")
        ws = torch.empty(need.value // 4, dtype=torch.float32, device=dev) if need.value else None
        st = lib.glu_add_rms_norm_backward(
            dy.data_ptr(), _row_stride("dy", dy), h.data_ptr(), _row_stride("h", h), weight.data_ptr(),
            rstd.data_ptr(), _ptr(dresidual), 0 if dresidual is None else _row_stride("dresidual", dresidual),
            dx.data_ptr(), _row_stride("dx", dx), dweight.data_ptr(), M, K, DTYPES[dt], _ptr(ws), need.value, handle)
    _raise_for(st)
    return dx, dweight


def fp8_quantize(x: torch.Tensor, out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """(q, scale) of activations x [M, K] (bf16, fp16 or fp32): scale [M, ceil(K / 128)] per row and 128 columns."""
    _tensor("x", x, _INPUTS, 2)
    dev = x.device
    M, K = x.shape
    ctx, handle = _on(dev, stream, x, out, scale_out)
    with ctx:
        out = _like("out", out, (M, K), E4M3, dev)
        scale = _row_scales("scale_out", scale_out, M, K, dev)
        st = library().glu_fp8_quantize(x.data_ptr(), _row_stride("x", x), out.data_ptr(), _row_stride("out", out),
                                        scale.data_ptr(), scale.stride(1), M, K, DTYPES[x.dtype], handle)
    _raise_for(st)
    return out, scale


def fp8_quantize_weight(w: torch.Tensor, out: Optional[torch.Tensor] = None,
                        scale_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(q, scale) of a weight w [N, K] (bf16, fp16 or fp32): one scale per 128 x 128 block."""
    _tensor("w", w, _INPUTS, 2)
    dev = w.device
    N, K = w.shape
    ctx, handle = _on(dev, stream, w, out, scale_out)
    with ctx:
        out = _like("out", out, (N, K), E4M3, dev)
        scale = _like("scale_out", scale_out, (groups(N), groups(K)), torch.float32, dev)
        st = library().glu_fp8_quantize_weight(w.data_ptr(), _row_stride("w", w), out.data_ptr(),
                                               _row_stride("out", out), scale.data_ptr(),
                                               _row_stride("scale_out", scale), N, K, DTYPES[w.dtype], handle)
    _raise_for(st)
    return out, scale


def _product(x, x_scale, weights, out_dtype, out, scale_out, plan, stream):
    _tensor("x", x, _E4M3, 2)
    dev = x.device
    M, K = x.shape
    _tensor("x_scale", x_scale, _F32, 2, dev)
    if tuple(x_scale.shape) != (M, groups(K)):
        raise ValueError(f"x_scale must be {(M, groups(K))}, got {tuple(x_scale.shape)}")
    N = weights[0][1].shape[0] if isinstance(weights[0][1], torch.Tensor) and weights[0][1].dim() == 2 else -1
    mats = []
    for name, w, s in weights:
        _tensor(name, w, _E4M3, 2, dev)
        _tensor(name + "_scale", s, _F32, 2, dev)
        if tuple(w.shape) != (N, K):
            raise ValueError(f"{name} must be {(N, K)}, got {tuple(w.shape)}")
        if tuple(s.shape) != (groups(N), groups(K)):
            raise ValueError(f"{name}_scale must be {(groups(N), groups(K))}, got {tuple(s.shape)}")
        mats.append(Matrix(w.data_ptr(), s.data_ptr(), _row_stride(name, w), _row_stride(name + "_scale", s), 1))
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype must be one of {[str(d) for d in DTYPES]}, got {out_dtype}")
    e4m3 = out_dtype is E4M3
    if scale_out is not None and not e4m3:
        raise ValueError("scale_out without an e4m3 output")
    n, dt = len(mats), DTYPES[out_dtype]
    lib = library()
    need = ctypes.c_int64(0)
    if plan is None:
        _raise_for(lib.glu_fp8_workspace(n, M, N, K, dt, ctypes.byref(need)))
    else:
        _raise_for(lib.glu_fp8_product_workspace(n, M, N, K, dt, ctypes.byref(plan), ctypes.byref(need)))
    xm = Matrix(x.data_ptr(), x_scale.data_ptr(), _row_stride("x", x), x_scale.stride(0), x_scale.stride(1))
    ctx, handle = _on(dev, stream, x, x_scale, out, scale_out, *(t for _, w, s in weights for t in (w, s)))
    with ctx:
        out = _like("out", out, (M, N), out_dtype, dev)
        scale = _row_scales("scale_out", scale_out, M, N, dev) if e4m3 else None
        ws = torch.empty(need.value // 4, dtype=torch.float32, device=dev) if need.value else None
        tail = (out.data_ptr(), _row_stride("out", out), _ptr(scale), scale.stride(1) if e4m3 else 0, M, N, K, dt)
        if plan is not None:
            st = lib.glu_fp8_product_tuned(ctypes.byref(xm), ctypes.byref(mats[0]),
                                           ctypes.byref(mats[1]) if n == 2 else None, *tail, ctypes.byref(plan),
                                           _ptr(ws), need.value, handle)
        elif n == 2:
            st = lib.glu_fp8_dual_glu(ctypes.byref(xm), ctypes.byref(mats[0]), ctypes.byref(mats[1]), *tail, _ptr(ws),
                                      need.value, handle)
        else:
            st = lib.glu_fp8_linear(ctypes.byref(xm), ctypes.byref(mats[0]), *tail, _ptr(ws), need.value, handle)
    _raise_for(st)
    return (out, scale) if e4m3 else out


def fp8_linear(x: torch.Tensor, x_scale: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               scale_out: Optional[torch.Tensor] = None, plan: Optional[ProductPlan] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """x @ weight.T on block-scaled e4m3: x [M, K] with x_scale [M, K / 128], weight [N, K] with its blocks' scales.

    Returns [M, N] in ``out_dtype`` (bf16, fp16, fp32), or for float8_e4m3fn the pair (q, scale).  fp32 accumulation
    over the K-blocks, one rounding.  K and the row strides should be multiples of 16 and the rows 16-byte
    aligned; other layouts are read byte by byte, slower.
    """
    return _product(x, x_scale, (("weight", weight, weight_scale),), out_dtype, out, scale_out, plan, stream)


def fp8_dual_glu(x: torch.Tensor, x_scale: torch.Tensor, gate: torch.Tensor, gate_scale: torch.Tensor,
                 up: torch.Tensor, up_scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                 plan: Optional[ProductPlan] = None, stream: Optional[torch.cuda.Stream] = None):
    """silu(x @ gate.T) * (x @ up.T) on block-scaled e4m3 operands, both weights read in place.

    As ``fp8_linear``; the activation is evaluated in fp32 on the fp32 sums and the result rounded once, to
    ``out_dtype`` or to block-scaled e4m3 (a pair) for the projection that follows.
    """
    return _product(x, x_scale, (("gate", gate, gate_scale), ("up", up, up_scale)), out_dtype, out, scale_out, plan,
                    stream)


def product_plan(mats: int, M: int, N: int, K: int, out_dtype: torch.dtype = torch.bfloat16, fast: bool = True) -> dict:
    """The launch a product would make (host only): mats 1 for ``fp8_linear``, 2 for ``fp8_dual_glu``."""
    p = ProductPlan()
    _raise_for(library().glu_fp8_product_plan(mats, M, N, K, DTYPES[out_dtype], int(fast), ctypes.byref(p)))
    return p.as_dict()


def _declare(lib):
    """Argument types of include/glu_fp8.h (called once by ``api.library``)."""
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    mp, pp, bp = ctypes.POINTER(Matrix), ctypes.POINTER(ProductPlan), ctypes.POINTER(ctypes.c_int64)
    norm = [vp, i64, vp, i64, vp, vp, i64, vp, i64]
    tail = [vp, i64, vp, i64, i64, i64, i64, i32]
    for name, args in {
        "glu_add_rms_norm": norm + [vp, i64, i64, f32, i32, vp],
        "glu_add_rms_norm_fp8": norm + [vp, i64, vp, i64, i64, f32, i32, vp],
        "glu_add_rms_norm_backward": [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, i64, i32, vp, i64, vp],
        "glu_add_rms_norm_backward_workspace": [i64, i64, bp],
        "glu_fp8_quantize": [vp, i64, vp, i64, vp, i64, i64, i64, i32, vp],
        "glu_fp8_quantize_weight": [vp, i64, vp, i64, vp, i64, i64, i64, i32, vp],
        "glu_fp8_linear": [mp, mp] + tail + [vp, i64, vp],
        "glu_fp8_dual_glu": [mp, mp, mp] + tail + [vp, i64, vp],
        "glu_fp8_product_plan": [i32, i64, i64, i64, i32, i32, pp],
        "glu_fp8_workspace": [i32, i64, i64, i64, i32, bp],
        "glu_fp8_product_tuned": [mp, mp, mp] + tail + [pp, vp, i64, vp],
        "glu_fp8_product_workspace": [i32, i64, i64, i64, i32, pp, bp],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
