"""moe_glu at the ends of its number formats: infinite scales of e4m3 blocks."""
import math

import pytest
import torch

import glu_mlp_gemv_amd as glu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 3, 4, 5, 40])
@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 6, 7])
def test_infinite_scale_of_the_last_block(M, blocks, kind):
    """A down projection whose last scale is infinite: its sums go to their own infinity, also where a kernel's stages reach
    past the columns."""
    K, N, E = 70, 128 * blocks - 16, 3
    x = torch.ones(M, K, dtype=T[kind], device=DEV)
    one = torch.full((E, N, K), 0x38, dtype=torch.uint8, device=DEV).view(E4M3)  # 1
    down = torch.full((E, K, N), 0x38, dtype=torch.uint8, device=DEV)
    down[:, K // 2:] = 0xb8  # -1
    g = -(-N // 128)
    s = torch.full((E, g, 1), 1.0 / K, device=DEV)
    ds = torch.ones(E, 1, g, device=DEV)
    ds[..., -1] = math.inf
    logits = torch.zeros(M, E, device=DEV)
    out = glu.moe_glu(x, logits, one, one, down.view(E4M3), 2, gate_scale=s, up_scale=s, down_scale=ds)
    torch.cuda.synchronize()
    want = torch.where(torch.arange(K, device=DEV) < K // 2, math.inf, -math.inf).expand(M, K)
    assert torch.equal(out.float(), want)
