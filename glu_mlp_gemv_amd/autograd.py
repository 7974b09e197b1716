"""The dual-weight GLU, the RMS norm, low-rank adapters and dropout as autograd Functions over the library's entry points.

Mirrors the segKI "Plan B" design (DeepSpeed PR #8602, comment "Plan B:
Dual-Weight GEMV", section "Plan B Design"): the Function keeps hidden, gate_w and up_w, reads the weight
Parameters in place in both directions, and returns gradients for all three,
so training and generation share one forward and one set of weights.
Forward: glu_dual_gemv; backward: glu_dual_gemv_backward (up to 65536 rows
of hidden per call).  ``rms_norm`` does the same for the residual addition and
norm, ``adapter_add`` for adapters' weights and ``dropout`` in front of them.  Only argument marshalling happens here.
"""
from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import adapters, api, counter_dropout, fp8


class DualWeightGlu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, gate_w, up_w):
        ctx.save_for_backward(hidden, gate_w, up_w)
        return api.dual_gemv(hidden, gate_w, up_w)

    @staticmethod
    def backward(ctx, dout):
        hidden, gate_w, up_w = ctx.saved_tensors
        dh, dwg, dwu = api.dual_gemv_backward(hidden.contiguous(), gate_w.contiguous(), up_w.contiguous(),
                                              dout.contiguous())
        return dh, dwg, dwu


def dual_weight_glu(hidden: torch.Tensor, gate_w: torch.Tensor, up_w: torch.Tensor) -> torch.Tensor:
    """out = silu(hidden @ gate_w.T) * (hidden @ up_w.T) with bf16 rounding per tensor, differentiable."""
    return DualWeightGlu.apply(hidden, gate_w, up_w)


class AddRmsNorm(torch.autograd.Function):
    """y, and with a residual also the sum h, of fp8.add_rms_norm; backward: fp8.add_rms_norm_backward."""

    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        y, h, rstd = fp8.add_rms_norm(x, weight, eps, residual=residual, return_rstd=True)
        ctx.save_for_backward(h, weight, rstd)
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, h)

    # a gradient of the gradient would pass the library's calls by in silence: once_differentiable refuses it
    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        if dy is None:  # only the residual stream was used
            return dh, None, None, dh
        # an expanded gradient (of a sum, say) has overlapping rows, which the library refuses
        dx, dw = fp8.add_rms_norm_backward(dy.contiguous(), h, weight, rstd,
                                           dresidual=None if dh is None else dh.contiguous())
        return dx, dw, None, dx if ctx.needs_input_grad[3] else None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None):
    """(y, h) of fp8.add_rms_norm, differentiable (once) in x, weight and residual."""
    out = AddRmsNorm.apply(x, weight, eps, residual)
    return (out, x) if residual is None else out


class AdapterAdd(torch.autograd.Function):
    """adapters.adapter_add; backward: adapters.adapter_backward."""

    @staticmethod
    def forward(ctx, y, x, a, b, index, scale):
        if ctx.needs_input_grad[5]:
            raise RuntimeError("adapter_add has no gradient for scale")
        keep = any(ctx.needs_input_grad[1:4])
        out, low = adapters._add(y, x, a, b, index, scale, None, keep, None)
        if keep:
            ctx.save_for_backward(x, a, b, index, scale, low)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        wanted = ctx.needs_input_grad[1:4]
        if not any(wanted):
            return dout, None, None, None, None, None
        x, a, b, index, scale, low = ctx.saved_tensors
        # an expanded gradient (of a sum, say) has overlapping rows, which the library refuses
        return (dout if ctx.needs_input_grad[0] else None,
                *adapters.adapter_backward(dout.contiguous(), x, a, b, index, low, scale, wanted=wanted), None, None)


def adapter_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
                scale: Optional[torch.Tensor] = None):
    """adapters.adapter_add, differentiable (once) in y, x, a and b."""
    return AdapterAdd.apply(y, x, a, b, index, scale)


class Dropout(torch.autograd.Function):
    """counter_dropout.dropout; backward: the same call on the gradient."""

    @staticmethod
    def forward(ctx, x, p, seed, offset, residual):
        ctx.at = p, None if isinstance(seed, torch.Tensor) else seed, offset
        if ctx.needs_input_grad[0] and isinstance(seed, torch.Tensor):
            ctx.save_for_backward(seed)  # a seed changed in between is an error there, not another mask
        return counter_dropout._dropout(x, p, seed, offset, residual, None, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        dx = None
        if ctx.needs_input_grad[0]:
            p, seed, offset = ctx.at
            if seed is None:
                (seed,) = ctx.saved_tensors
            dx = counter_dropout._dropout(dout.contiguous(), p, seed, offset, None, None, None)
        return dx, None, None, None, dout if ctx.needs_input_grad[4] else None


def dropout(x: torch.Tensor, p: float, seed: Union[int, torch.Tensor], offset: int = 0,
            residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """counter_dropout.dropout, differentiable (once) in x and residual."""
    return Dropout.apply(x, p, seed, offset, residual)
