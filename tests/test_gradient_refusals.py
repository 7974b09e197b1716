"""Calls without a gradient refuse operands that carry one, on the host and on the device (where the short path looks first)."""
import pytest
import torch

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
