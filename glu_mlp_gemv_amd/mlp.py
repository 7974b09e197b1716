"""A decoder layer's MLP on 8-bit weights, from the operators of ``fp8``, or with a mixture of experts (``moe``).

``Fp8GluMlp`` takes the bf16 weights of a trained layer, converts them once, and then runs, for a prefill or one
token, norm -> gate and up -> down in three calls whose intermediate activations stay in block-scaled e4m3:

    h = x + residual;  y = down(silu(gate(norm(h))) * up(norm(h)))

A batch whose requests have low-rank adapters (``adapters``) runs the same projections with theirs beside them.  It infers:
there is no gradient, and inputs that require one are refused where autograd records.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import adapters as low_rank, fp8, moe


class MlpAdapters(NamedTuple):
    """Low-rank adapters of many requests for the three projections: (a, b) of each, as ``adapters`` takes them."""

    gate: Tuple[torch.Tensor, torch.Tensor]
    up: Tuple[torch.Tensor, torch.Tensor]
    down: Tuple[torch.Tensor, torch.Tensor]
    scale: Optional[torch.Tensor] = None


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

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, adapters: Optional[MlpAdapters] = None,
                 index: Optional[torch.Tensor] = None):
        """(y, h) for x [M, K] and the residual stream: h = x + residual goes to the next layer with y.

        With ``adapters``, of x's type (bf16 or fp16), index [M] (int32) names each row's: the 8-bit projections then leave
        in x's type, and the adapters see the norm's and the activation's values before their conversion.
        """
        if adapters is not None:
            return self._adapted(x, residual, adapters, index)
        q, scale, h = fp8.add_rms_norm_fp8(x, self.norm_weight, self.eps, residual=residual)
        a, a_scale = fp8.fp8_dual_glu(q, scale, *self.gate, *self.up, out_dtype=fp8.E4M3)
        return fp8.fp8_linear(a, a_scale, *self.down, out_dtype=x.dtype), h

    def _adapted(self, x, residual, w: MlpAdapters, index):
        n, h = fp8.add_rms_norm(x, self.norm_weight, self.eps, residual=residual)
        q = fp8.fp8_quantize(n)
        gate, up = (fp8.fp8_linear(*q, *m, out_dtype=x.dtype) for m in (self.gate, self.up))
        a = low_rank.adapter_glu(gate, up, n, *w.gate, *w.up, index, w.scale)
        y = fp8.fp8_linear(*fp8.fp8_quantize(a), *self.down, out_dtype=x.dtype)
        return low_rank.adapter_add(y, a, *w.down, index, w.scale), h


class ExpertGluMlp:
    """The same with a mixture of experts: norm -> router -> the chosen experts' gate, up and down.

    norm_weight [K] and router [E, K] in bf16 or fp16, gate and up [E, N, K], down [E, K, N] in the same type, or e4m3 with
    ``scales`` of all three (``moe.moe_glu``).  ``top`` experts per row, ranked by fp32 logits.
    """

    def __init__(self, norm_weight: torch.Tensor, router: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                 down: torch.Tensor, top: int, normalize: bool = True, eps: float = 1e-6, scales=(None, None, None)):
        self.norm_weight, self.router = norm_weight.detach(), router.detach()
        self.experts = tuple(w.detach() for w in (gate, up, down))
        self.scales = dict(zip(("gate_scale", "up_scale", "down_scale"), scales))
        self.top, self.normalize, self.eps = top, normalize, eps

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        """(y, h) for x [M, K] and the residual stream, as ``Fp8GluMlp``."""
        n, h = fp8.add_rms_norm(x, self.norm_weight, self.eps, residual=residual)
        return moe.moe_glu(n, moe.moe_logits(n, self.router), *self.experts, self.top, normalize=self.normalize, **self.scales), h
