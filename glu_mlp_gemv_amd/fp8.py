"""Python face of include/glu_fp8.h: RMS norm, conversion to block-scaled e4m3, products on it.

As in ``api``, only argument marshalling happens here: tensors are checked, their device pointers
and torch's current HIP stream go to ``libglu_gemv.so``, and a non-OK status becomes a ``GluError``.  Calls
that give no outputs, plan or stream try the extension module ``_fast`` first (csrc/glu_torch.cpp): it does the
same for operands in the usual form, in a third of the time, and leaves the rest, refusals among them, to the
code here.

Block-scaled e4m3: a stored ``torch.float8_e4m3fn`` value q stands for ``q * scale``.  Activations
[M, K] have an fp32 scale per row and 128 columns, [M, ceil(K / 128)], which the functions here return stored
group by group (``scale.t()`` is contiguous) and accept at any strides; weights [N, K] one per block of
128 x 128, [ceil(N / 128), ceil(K / 128)].

The conversions and products carry no gradient.  Row-strided views are taken at the stride they report.  With ``stream`` the work runs there and the
results belong to that stream's memory pool; the tensors given are recorded on it.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib
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
                ("launches", ctypes.c_int), ("workspace_bytes", ctypes.c_int64), ("columns", ctypes.c_int64)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel_name"] = KERNEL_NAMES[self.kernel]
        return d


# in the order that _fast.bind takes them
_BOUND = ("glu_add_rms_norm", "glu_add_rms_norm_fp8", "glu_add_rms_norm_backward",
          "glu_add_rms_norm_backward_workspace", "glu_fp8_quantize", "glu_fp8_quantize_weight", "glu_fp8_linear",
          "glu_fp8_dual_glu", "glu_fp8_workspace", "glu_fp8_product_workspace")
_fast = None


def _load_fast():
    """The extension module, bound to the library that ``api`` has loaded (raises if it is not built)."""
    global _fast
    lib = library()
    try:
        module = importlib.import_module("glu_mlp_gemv_amd._fast")
    except ImportError as e:
        raise RuntimeError("glu_mlp_gemv_amd/_fast.so is not built; run __graft_entry__.build() "
                           "(or python -m glu_mlp_gemv_amd.build)") from e
    module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _BOUND))
    _fast = module
    return module


def _taken(result) -> bool:
    """Whether the extension module took the call; raises for a status."""
    if type(result) is int:
        _raise_for(result)
    return result is not None


def groups(n: int) -> int:
    """Scales along a dimension of n."""
    return -(-n // GROUP)


_INPUTS = (torch.bfloat16, torch.float16, torch.float32)


def _refuse(name: str, t, dtypes, shape, dev):
    """Says what is wrong with a tensor that is not of these types, this shape (None: any extent) and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dim() != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dims, got {t.dim()}")
    if any(want is not None and n != want for n, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _matrix(name: str, t, dtypes):
    """(rows, columns, device) of the tensor that sets a call's sizes."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_cuda and t.dim() == 2):
        _refuse(name, t, dtypes, (None, None), None)
    rows, cols = t.shape
    return rows, cols, t.device


# The checks below are on the path of every call, some microseconds long in all: what is as expected passes one
# expression, and only what is not is looked at again.

def _rows(name: str, t, dtype, rows: int, cols: int, dev) -> int:
    """The row stride of a [rows, cols] operand."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (rows, cols) and t.device == dev):
        _refuse(name, t, (dtype,), (rows, cols), dev)
    ld, one = t.stride()
    return ld if one == 1 and ld >= cols and rows > 1 else _row_stride(name, t)


def _vector(name: str, t, dtype, n: int, dev):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n,) and t.device == dev):
        _refuse(name, t, (dtype,), (n,), dev)
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: elements must be contiguous, got stride {t.stride(0)}")


def _new(rows: int, cols: int, dtype, dev):
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _output(name: str, t, dtype, rows: int, cols: int, dev):
    """(tensor, row stride) of an output: the one given, checked, or a new one."""
    if t is None:
        return _new(rows, cols, dtype, dev), cols
    return t, _rows(name, t, dtype, rows, cols, dev)


def _row_scales(name: str, t, rows: int, cols: int, dev):
    """(tensor, group stride): a new [rows, groups] scale tensor stored group by group, or the given one, whose
    columns must be contiguous."""
    if t is None:
        return torch.empty_strided((rows, groups(cols)), (1, rows), dtype=torch.float32, device=dev), rows
    _refuse(name, t, (torch.float32,), (rows, groups(cols)), dev)
    _row_stride(name, t.t())
    return t, t.stride(1)


def _on(dev, stream, *tensors):
    """(context, stream handle) of a call on ``stream`` or the device's current stream."""
    if stream is None:
        index = dev.index
        ctx = _NO_CONTEXT if index == torch.cuda.current_device() else torch.cuda.device(dev)
        # current_stream().cuda_stream without building a Stream object; a torch without a GPU backend has no such name
        return ctx, torch._C._cuda_getCurrentRawStream(index)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream), stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _norm(x, weight, eps, residual, out, scale_out, residual_out, return_rstd, stream, e4m3):
    M, K, dev = _matrix("x", x, _INPUTS)
    dt = x.dtype
    ldx = _rows("x", x, dt, M, K, dev)
    _vector("weight", weight, dt, K, dev)
    ldr = 0
    if residual is not None:
        ldr = _rows("residual", residual, dt, M, K, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    ctx, handle = _on(dev, stream, x, weight, residual, out, scale_out, residual_out)
    with ctx:
        h, ldh = (x, 0) if residual is None else _output("residual_out", residual_out, dt, M, K, dev)
        rstd = torch.empty(M, dtype=torch.float32, device=dev) if return_rstd else None
        out, ldo = _output("out", out, E4M3 if e4m3 else dt, M, K, dev)
        head = (x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), None if residual is None else h.data_ptr(),
                ldh, out.data_ptr(), ldo)
        if e4m3:
            scale, lds = _row_scales("scale_out", scale_out, M, K, dev)
            st = library().glu_add_rms_norm_fp8(*head, scale.data_ptr(), lds, _ptr(rstd), M, K, eps, DTYPES[dt],
                                                handle)
        else:
            scale = None
            st = library().glu_add_rms_norm(*head, _ptr(rstd), M, K, eps, DTYPES[dt], handle)
    if st:
        _raise_for(st)
    return out, scale, h, rstd


def _wants_gradient(x, weight, residual) -> bool:
    """Whether autograd would record a call on these operands (none in a Function's own forward)."""
    return torch.is_grad_enabled() and (getattr(x, "requires_grad", False) or getattr(weight, "requires_grad", False)
                                        or getattr(residual, "requires_grad", False))


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                 return_rstd: bool = False, stream: Optional[torch.cuda.Stream] = None):
    """(y, h): h = x + residual in x's type (x itself without a residual), y = h / rms(h) * weight.

    x and residual [M, K], weight [K], all bf16, fp16 or fp32; rms(h) = sqrt(mean(h^2) + eps) per
    row, in fp32, and y rounded once.  ``residual_out`` may be ``residual`` or ``x`` (in place).  With
    ``return_rstd`` also 1 / rms [M] in fp32, which ``add_rms_norm_backward`` takes.  Operands that require a gradient
    have one, through ``autograd.rms_norm``; together with an output, stream or rstd they are refused.
    """
    plain = out is None and residual_out is None and stream is None and not return_rstd
    if plain:
        r = (_fast or _load_fast()).norm(x, weight, eps, residual, False)
        if _taken(r):
            return r[0], x if residual is None else r[1]
    if _wants_gradient(x, weight, residual):
        if not plain:
            raise RuntimeError("add_rms_norm with out, residual_out, return_rstd or stream has no gradient, and an operand "
                               "requires one: call it without them, or under torch.no_grad()")
        from .autograd import rms_norm
        return rms_norm(x, weight, eps, residual=residual)
    out, _, h, rstd = _norm(x, weight, eps, residual, out, None, residual_out, return_rstd, stream, False)
    return (out, h, rstd) if return_rstd else (out, h)


def add_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                     residual_out: Optional[torch.Tensor] = None, return_rstd: bool = False,
                     stream: Optional[torch.cuda.Stream] = None):
    """(q, scale, h): ``add_rms_norm`` with y converted to block-scaled e4m3 before any rounding to x's type.

    Has no gradient: operands that require one are refused where autograd records.
    """
    if out is None and scale_out is None and residual_out is None and stream is None and not return_rstd:
        r = (_fast or _load_fast()).norm(x, weight, eps, residual, True)
        if _taken(r):
            return r[0], r[2], x if residual is None else r[1]
    if _wants_gradient(x, weight, residual):
        raise RuntimeError("add_rms_norm_fp8 has no gradient, and an operand requires one: call it under torch.no_grad(), or "
                           "train with autograd.rms_norm")
    out, scale, h, rstd = _norm(x, weight, eps, residual, out, scale_out, residual_out, return_rstd, stream, True)
    return (out, scale, h, rstd) if return_rstd else (out, scale, h)


_grad_workspace = functools.lru_cache(maxsize=256)(lambda M, K: _bytes("glu_add_rms_norm_backward_workspace", M, K))


def _bytes(query: str, *args) -> int:
    """What a workspace query of the library answers (host only)."""
    need = ctypes.c_int64(0)
    _raise_for(getattr(library(), query)(*args, ctypes.byref(need)))
    return need.value


def add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          dresidual: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                          dweight: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(dx, dweight) of ``add_rms_norm`` for the gradient ``dy`` of y and ``dresidual`` of h.

    h and rstd are the forward's.  dx is the gradient of x and of the residual alike.  dweight sums the
    rows in fp32 in a fixed order.  ``dx`` may be ``dresidual`` (in place).
    """
    if dx is None and dweight is None and stream is None:
        r = (_fast or _load_fast()).norm_grad(dy, h, weight, rstd, dresidual)
        if _taken(r):
            return r
    M, K, dev = _matrix("h", h, _INPUTS)
    dt = h.dtype
    ldh = _rows("h", h, dt, M, K, dev)
    lddy = _rows("dy", dy, dt, M, K, dev)
    _vector("weight", weight, dt, K, dev)
    _vector("rstd", rstd, torch.float32, M, dev)
    lddr = 0 if dresidual is None else _rows("dresidual", dresidual, dt, M, K, dev)
    need = _grad_workspace(M, K)
    ctx, handle = _on(dev, stream, dy, h, weight, rstd, dresidual, dx, dweight)
    with ctx:
        dx, lddx = _output("dx", dx, dt, M, K, dev)
        if dweight is None:
            dweight = torch.empty_like(weight)
        else:
            _vector("dweight", dweight, dt, K, dev)
        ws = torch.empty(need // 4, dtype=torch.float32, device=dev) if need else None
        st = library().glu_add_rms_norm_backward(
            dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(), _ptr(dresidual), lddr,
            dx.data_ptr(), lddx, dweight.data_ptr(), M, K, DTYPES[dt], _ptr(ws), need, handle)
    if st:
        _raise_for(st)
    return dx, dweight


def fp8_quantize(x: torch.Tensor, out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """(q, scale) of activations x [M, K] (bf16, fp16 or fp32): scale [M, ceil(K / 128)] per row and 128 columns."""
    if out is None and scale_out is None and stream is None:
        r = (_fast or _load_fast()).quantize(x, False)
        if _taken(r):
            return r
    M, K, dev = _matrix("x", x, _INPUTS)
    ldx = _rows("x", x, x.dtype, M, K, dev)
    ctx, handle = _on(dev, stream, x, out, scale_out)
    with ctx:
        out, ldo = _output("out", out, E4M3, M, K, dev)
        scale, lds = _row_scales("scale_out", scale_out, M, K, dev)
        st = library().glu_fp8_quantize(x.data_ptr(), ldx, out.data_ptr(), ldo, scale.data_ptr(), lds, M, K,
                                        DTYPES[x.dtype], handle)
    if st:
        _raise_for(st)
    return out, scale


def fp8_quantize_weight(w: torch.Tensor, out: Optional[torch.Tensor] = None,
                        scale_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(q, scale) of a weight w [N, K] (bf16, fp16 or fp32): one scale per 128 x 128 block."""
    if out is None and scale_out is None and stream is None:
        r = (_fast or _load_fast()).quantize(w, True)
        if _taken(r):
            return r
    N, K, dev = _matrix("w", w, _INPUTS)
    ldw = _rows("w", w, w.dtype, N, K, dev)
    ctx, handle = _on(dev, stream, w, out, scale_out)
    with ctx:
        out, ldo = _output("out", out, E4M3, N, K, dev)
        scale, lds = _output("scale_out", scale_out, torch.float32, groups(N), groups(K), dev)
        st = library().glu_fp8_quantize_weight(w.data_ptr(), ldw, out.data_ptr(), ldo, scale.data_ptr(), lds, N, K,
                                               DTYPES[w.dtype], handle)
    if st:
        _raise_for(st)
    return out, scale


@functools.lru_cache(maxsize=256)
def _product_workspace(mats: int, M: int, N: int, K: int, dt: int, fast: bool) -> int:
    """Workspace bytes of a call on this layout: of the fast kernels, of aligned copies, or of reading in place."""
    if fast:
        return _bytes("glu_fp8_product_workspace", mats, M, N, K, dt, None)
    return (_bytes("glu_fp8_copy_workspace", mats, M, N, K, dt)  # 0: such a call is never copied
            or _bytes("glu_fp8_workspace", mats, M, N, K, dt))


def _fast_layout(K: int, *operands) -> bool:
    """Whether the library reads (tensor, row stride) pairs of K columns 16 aligned bytes at a time."""
    return K % 16 == 0 and all((t.data_ptr() | ld) % 16 == 0 and ld <= 1 << 23 for t, ld in operands)


def _product(x, x_scale, weights, out_dtype, out, scale_out, plan, stream):
    if out is None and scale_out is None and plan is None and stream is None:
        r = (_fast or _load_fast()).product(DTYPES.get(out_dtype, -1), x, x_scale, *weights[0][1:],
                                            *(weights[1][1:] if len(weights) == 2 else ()))
        if _taken(r):
            return r if len(r) == 2 else r[0]
    M, K, dev = _matrix("x", x, (E4M3,))
    G = groups(K)
    ldx = _rows("x", x, E4M3, M, K, dev)
    if not (isinstance(x_scale, torch.Tensor) and x_scale.dtype is torch.float32 and x_scale.shape == (M, G)
            and x_scale.device == dev):
        _refuse("x_scale", x_scale, (torch.float32,), (M, G), dev)
    sxm, sxg = x_scale.stride()
    N, _, _ = _matrix(weights[0][0], weights[0][1], (E4M3,))
    NG = groups(N)
    mats = []
    for name, w, s in weights:
        ldw, lds = _rows(name, w, E4M3, N, K, dev), _rows(name + "_scale", s, torch.float32, NG, G, dev)
        mats.append(Matrix(w.data_ptr(), s.data_ptr(), ldw, lds, 1))
    dt = DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError(f"out_dtype must be one of {[str(d) for d in DTYPES]}, got {out_dtype}")
    e4m3 = out_dtype is E4M3
    if scale_out is not None and not e4m3:
        raise ValueError("scale_out without an e4m3 output")
    n = len(mats)
    if plan is None:
        fast = _fast_layout(K, (x, ldx), *((w, m.ld) for (_, w, _), m in zip(weights, mats)))
        need = _product_workspace(n, M, N, K, dt, fast)
    else:
        need = _bytes("glu_fp8_product_workspace", n, M, N, K, dt, ctypes.byref(plan))
    ctx, handle = _on(dev, stream, x, x_scale, out, scale_out, *(t for _, w, s in weights for t in (w, s)))
    with ctx:
        out, ldo = _output("out", out, out_dtype, M, N, dev)
        scale, lds = _row_scales("scale_out", scale_out, M, N, dev) if e4m3 else (None, 0)
        ws = torch.empty(need // 4, dtype=torch.float32, device=dev) if need else None
        args = (Matrix(x.data_ptr(), x_scale.data_ptr(), ldx, sxm, sxg), *mats, out.data_ptr(), ldo, _ptr(scale), lds,
                M, N, K, dt)
        if plan is not None:
            up = (None,) if n == 1 else ()
            st = library().glu_fp8_product_tuned(*args[:2], *up, *args[2:], plan, _ptr(ws), need, handle)
        elif n == 2:
            st = library().glu_fp8_dual_glu(*args, _ptr(ws), need, handle)
        else:
            st = library().glu_fp8_linear(*args, _ptr(ws), need, handle)
    if st:
        _raise_for(st)
    return (out, scale) if e4m3 else out


def fp8_linear(x: torch.Tensor, x_scale: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               scale_out: Optional[torch.Tensor] = None, plan: Optional[ProductPlan] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """x @ weight.T on block-scaled e4m3: x [M, K] with x_scale [M, K / 128], weight [N, K] with its blocks' scales.

    Returns [M, N] in ``out_dtype`` (bf16, fp16, fp32), or for float8_e4m3fn the pair (q, scale), rounded once.  The sums
    are fp32, but for 16-bit outputs of more than 16 rows on aligned operands: those run on the matrix unit's 8-bit
    path, which within 8 neighbouring products drops what lies 13 to 14 bits below the largest (some 2^-16 of a result,
    without bias).  out_dtype=torch.float32 always has fp32 sums.

    K and the row strides should be multiples of 16 and the rows 16-byte aligned; other layouts are read as they are,
    slower, or above 16 rows of x copied first where that is faster.
    """
    return _product(x, x_scale, (("weight", weight, weight_scale),), out_dtype, out, scale_out, plan, stream)


def fp8_dual_glu(x: torch.Tensor, x_scale: torch.Tensor, gate: torch.Tensor, gate_scale: torch.Tensor,
                 up: torch.Tensor, up_scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                 plan: Optional[ProductPlan] = None, stream: Optional[torch.cuda.Stream] = None):
    """silu(x @ gate.T) * (x @ up.T) on block-scaled e4m3 operands, both weights read in place.

    As ``fp8_linear``, its sums among it; the activation is evaluated in fp32 on them and the result rounded once, to
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
        "glu_fp8_copy_workspace": [i32, i64, i64, i64, i32, bp],
        "glu_fp8_product_tuned": [mp, mp, mp] + tail + [pp, vp, i64, vp],
        "glu_fp8_product_workspace": [i32, i64, i64, i64, i32, pp, bp],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
