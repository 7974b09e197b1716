"""Calls without a gradient refuse operands that carry one, on the host and on the device (where the short path looks first)."""
import pytest
import torch
from torch.autograd import forward_ad

import glu_mlp_gemv_amd as glu

DEVICES = ["cpu", pytest.param("cuda:0", marks=pytest.mark.gpu)]
E4M3 = torch.float8_e4m3fn


def experts(dev):
    M, K, N, E = 2, 128, 128, 3
    w = torch.zeros(E, N, K, dtype=torch.uint8, device=dev).view(E4M3)
    return dict(x=torch.ones(M, K, dtype=torch.bfloat16, device=dev), logits=torch.zeros(M, E, device=dev), gate=w, up=w, down=w,
                top=2, **{n + "_scale": torch.ones(E, 1, 1, device=dev) for n in ("gate", "up", "down")})


@pytest.mark.parametrize("dev", DEVICES)
@pytest.mark.parametrize("name", ["gate_scale", "up_scale", "down_scale"])
def test_scales_of_experts(name, dev):
    k = experts(dev)
    k[name].requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        glu.moe_glu(**k)
    if dev != "cpu":
        with torch.no_grad():
            assert not glu.moe_glu(**k).any()


def calls(dev):
    """name -> (call, its operands that may carry a tangent)"""
    M, K, N, R, L = 3, 64, 64, 8, 2
    t = torch.bfloat16
    one = lambda *s, t=t: torch.ones(*s, dtype=t, device=dev)  # noqa: E731
    index = torch.zeros(M, dtype=torch.int32, device=dev)
    scale = one(L, t=torch.float32)
    moe = experts(dev)
    e = {k: v for k, v in moe.items() if k not in ("top", "gate", "up", "down")}
    return {
        "adapter_add": (lambda **k: glu.adapter_add(**k, index=index),
                        dict(y=one(M, N), x=one(M, K), a=one(L, R, K), b=one(L, N, R), scale=scale)),
        "adapter_glu": (lambda **k: glu.adapter_glu(**k, index=index),
                        dict(gate=one(M, N), up=one(M, N), x=one(M, K), gate_a=one(L, R, K), gate_b=one(L, N, R),
                             up_a=one(L, R, K), up_b=one(L, N, R), scale=scale)),
        "moe_glu": (lambda **k: glu.moe_glu(**{**moe, **k}), e),
        "dropout": (lambda **k: glu.dropout(**k, p=0.5, seed=1), dict(x=one(M, K), residual=one(M, K))),
        "add_rms_norm": (lambda **k: glu.add_rms_norm(**k, eps=1e-6), dict(x=one(M, K), weight=one(K), residual=one(M, K))),
        "add_rms_norm_fp8": (lambda **k: glu.add_rms_norm_fp8(**k, eps=1e-6),
                             dict(x=one(M, K), weight=one(K), residual=one(M, K))),
    }


@pytest.mark.parametrize("dev", DEVICES)
@pytest.mark.parametrize("call", calls("cpu"))
def test_tangents_of_forward_mode(call, dev):
    """They would be lost in silence: refused for every operand, under no_grad too, and not where forward mode is off."""
    f, operands = calls(dev)[call]
    with forward_ad.dual_level():
        for name, v in operands.items():
            k = {**operands, name: forward_ad.make_dual(v, torch.ones_like(v))}
            with pytest.raises(RuntimeError, match="forward mode"):
                f(**k)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward mode"):
                f(**k)
        if dev != "cpu":
            f(**operands)
            with torch.autograd.forward_ad._set_fwd_grad_enabled(False):
                f(**k)
