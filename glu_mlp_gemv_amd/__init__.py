"""Dual-weight GLU GEMV for MI355X (gfx950).

``dual_gemv(hidden, gate_w, up_w, out=None)`` computes the decode-time GLU
projection out = bf16(bf16(silu(bf16(h @ Wg^T))) * bf16(h @ Wu^T)) from the
separate gate and up weight matrices, through the C-ABI library built from
``csrc/`` (declared in ``include/glu_gemv.h``).  The library is loaded on the
first call; if it is missing or cannot be loaded the call raises, there is no
fallback path.

``add_rms_norm`` (with ``add_rms_norm_fp8`` and ``add_rms_norm_backward``), ``fp8_quantize``,
``fp8_quantize_weight``, ``fp8_linear`` and ``fp8_dual_glu`` are the decoder MLP's path around that projection
on 8-bit (block-scaled e4m3) weights and activations (``include/glu_fp8.h``); ``mlp.Fp8GluMlp`` runs them
together.

``adapter_add``, ``adapter_glu`` and ``adapter_backward`` are low-rank adapters beside such projections, one per row of a
batch of many requests (``include/glu_adapter.h``), and ``dropout`` is what they are trained behind
(``include/glu_dropout.h``).  ``moe_glu`` is a mixture-of-experts GLU layer for a few tokens (``include/glu_moe.h``),
``mlp.ExpertGluMlp`` a decoder layer's MLP with it.

``inputs`` holds the seeded synthetic input generators.
"""
from . import inputs  # noqa: F401

_FP8 = ("add_rms_norm", "add_rms_norm_fp8", "add_rms_norm_backward", "fp8_quantize", "fp8_quantize_weight",
        "fp8_linear", "fp8_dual_glu")

_ADAPTERS = ("adapter_add", "adapter_glu", "adapter_backward")

__all__ = ["inputs", "dual_gemv", "library", "dropout", "moe_glu", *_FP8, *_ADAPTERS]


def __getattr__(name):
    if name in ("dual_gemv", "library", "status_string", "GluError"):
        from . import api
        return getattr(api, name)
    if name in _FP8:
        from . import fp8
        value = globals()[name] = getattr(fp8, name)
        return value
    if name in _ADAPTERS:
        from . import adapters
        value = globals()[name] = getattr(adapters, name)
        return value
    if name == "moe_glu":
        from . import moe
        value = globals()[name] = moe.moe_glu
        return value
    if name == "dropout":
        from . import counter_dropout
        value = globals()[name] = counter_dropout.dropout
        return value
    raise AttributeError(name)
