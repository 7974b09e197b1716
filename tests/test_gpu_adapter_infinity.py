"""Infinities among numbers past fp16's range: sums go to the infinity, and only what is NaN by the definition is NaN."""
import math

import pytest
import torch

import glu_mlp_gemv_amd as glu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("R", [4, 20, 64, 100])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_infinite_hidden_value(M, R, kind):
    """One rank's hidden value is infinite, the others are 2^20 and pull the other way."""
    K, N, t = 64, 70, T[kind]
    x = torch.ones(M, K, dtype=t, device=DEV)
    a = torch.full((1, R, K), 2.0 ** 14, dtype=t, device=DEV)
    a[0, R // 2] = math.inf
    sign = torch.where(torch.arange(N, device=DEV) % 2 == 0, 1.0, -1.0)
    b = -sign[None, :, None].expand(1, N, R).to(t).contiguous()
    b[0, :, R // 2] = sign.to(t)
    y = torch.zeros(M, N, dtype=t, device=DEV)
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    out, low = glu.adapter_add(y, x, a, b, index, return_low=True)
    torch.cuda.synchronize()
    assert torch.equal(out.float(), (math.inf * sign).expand(M, N))
    assert low[:, R // 2].eq(math.inf).all() and low[:, 0].eq(2.0 ** 20).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("R", [4, 20, 64])
@pytest.mark.parametrize("M", [2, 400, 1500])
def test_infinite_row_of_the_gradients(M, R, kind):
    """One row's d and t are infinite, the other rows' are 2^20 and pull the other way."""
    K, N, t = 72, 64, T[kind]
    row = M // 2
    x, dout = (torch.full((M, n), -1.0, dtype=t, device=DEV) for n in (K, N))
    x[row] = 1.0
    dout.abs_()
    a, b = (torch.full(s, 2.0 ** 14, dtype=t, device=DEV) for s in ((1, R, K), (1, N, R)))
    low = torch.full((M, R), -2.0 ** 20, device=DEV)
    low[row] = math.inf
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    db = glu.adapter_backward(dout, x, a, b, index, low)[2]
    dout[row] = math.inf  # d of that row; what it gives db with it is infinite or NaN
    dx, da, _ = glu.adapter_backward(dout, x, a, b, index, low)
    torch.cuda.synchronize()
    assert da.eq(math.inf).all() and db.eq(math.inf).all() and dx[row].eq(math.inf).all()
