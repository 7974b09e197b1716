"""A decoder layer's MLP on 8-bit weights, from the operators of ``fp8``.

``Fp8GluMlp`` takes the bf16 weights of a trained layer, converts them once, and then runs, for a prefill or one
token, norm -> gate and up -> down in three calls whose intermediate activations stay in block-scaled e4m3:

    h = x + residual;  y = down(silu(gate(norm(h))) * up(norm(h)))

It infers: there is no gradient, and inputs that require one are refused where autograd records.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import fp8


class Fp8GluMlp:
    """norm_weight [K], gate and up [N, K], down [K, N], bf16 / fp16 / fp32 on one GPU."""

    def __init__(self, norm_weight: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                 eps: float = 1e-6):
        self.eps = eps
        self.norm_weight = norm_weight.detach()
        self.update(gate, up, down)

    def update(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor) -> None:
        """Convert new weights (after an optimiser step), into the tensors already held if there are any."""
        names = ("gate", "up", "down")
        for name, w in zip(names, (gate, up, down)):
            q, scale = getattr(self, name, (None, None))
            setattr(self, name, fp8.fp8_quantize_weight(w.detach(), out=q, scale_out=scale))

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        """(y, h) for x [M, K] and the residual stream: h = x + residual goes to the next layer with y."""
        q, scale, h = fp8.add_rms_norm_fp8(x, self.norm_weight, self.eps, residual=residual)
        a, a_scale = fp8.fp8_dual_glu(q, scale, *self.gate, *self.up, out_dtype=fp8.E4M3)
        return fp8.fp8_linear(a, a_scale, *self.down, out_dtype=x.dtype), h
