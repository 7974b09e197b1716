"""adapter_glu's activation over the whole range of gates."""
import math

import pytest
import torch

import adapter_ref as ref
import glu_mlp_gemv_amd as glu
from fp8_ref import check_store

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GATES = [0.0, 1e-6, -1e-6, 1.0, -1.0, 20.0, -20.0, -60.0, -86.5, 87.0, -87.0, 88.0, -88.0, -89.0, -92.0, -104.0, 300.0, -300.0, 1e30, -1e30,
         math.inf]


@pytest.mark.parametrize("M", [3, 400])
@pytest.mark.parametrize("up", [1.0, 2.0 ** 20, 2.0 ** 120])
def test_gates(M, up):
    """Rows without an adapter, whose sums are gate and up themselves.  From -87 down the result may be 0: silu there is below
    2^-119 in magnitude."""
    N, K, R, L, t = len(GATES), 64, 8, 2, torch.bfloat16
    gate = torch.tensor(GATES, device=DEV).to(t).expand(M, N).contiguous()
    u = torch.full_like(gate, up)
    a, b = torch.ones(L, R, K, dtype=t, device=DEV), torch.ones(L, N, R, dtype=t, device=DEV)
    out = glu.adapter_glu(gate, u, torch.ones(M, K, dtype=t, device=DEV), a, b, a, b, torch.full((M,), -1, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    g = gate.double()
    zero = torch.zeros_like(g)
    want, bound = ref.glu64(g, u.double(), zero, zero)
    bound = torch.where(g < -86.9, 2.0 ** -119 * up + bound, bound)
    fits = want.abs() < 3e38  # larger ones are infinite
    check_store("glu", out[fits].reshape(-1), want[fits], bound[fits])
    assert (out[~fits] == math.inf).all() and fits.logical_not().any()


def test_infinite_negative_gate_is_nan():
    """-inf / inf, as the elementary operations give."""
    t = torch.bfloat16
    gate = torch.full((2, 8), -math.inf, dtype=t, device=DEV)
    a, b = torch.ones(1, 4, 8, dtype=t, device=DEV), torch.ones(1, 8, 4, dtype=t, device=DEV)
    none = torch.full((2,), -1, dtype=torch.int32, device=DEV)
    assert glu.adapter_glu(gate, torch.ones_like(gate), torch.ones_like(gate), a, b, a, b, none).isnan().all()
