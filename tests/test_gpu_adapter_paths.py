"""The new operators together, as a decoder layer and a training step use them."""
import pytest
import torch

import adapter_ref as ref
import dropout_ref
import glu_mlp_gemv_amd as glu
from fp8_ref import check_store
from glu_mlp_gemv_amd import mlp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


@pytest.mark.parametrize("M", [1, 5, 40])
def test_adapted_8bit_mlp(M):
    """Fp8GluMlp with adapters is its calls one after another; rows without one are the layer's own up to the conversions."""
    K, N, R, L, t = 256, 384, 16, 3, torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(M)
    gate, up, down = rand(g, N, K) * K ** -0.5, rand(g, N, K) * K ** -0.5, rand(g, K, N) * N ** -0.5
    layer = mlp.Fp8GluMlp(torch.ones(K, dtype=t, device=DEV), gate.to(t), up.to(t), down.to(t))
    pair = lambda n, k: ((rand(g, L, R, k) * k ** -0.5).to(t), (rand(g, L, n, R) * R ** -0.5).to(t))  # noqa: E731
    w = mlp.MlpAdapters(pair(N, K), pair(N, K), pair(K, N), torch.rand(L, generator=g, device=DEV) + 0.5)
    x, res = rand(g, M, K).to(t), rand(g, M, K).to(t)
    index = torch.randint(-1, L, (M,), generator=g, device=DEV).int()
    index[0] = 1
    y, h = layer(x, res, w, index)
    n, h2 = glu.add_rms_norm(x, layer.norm_weight, layer.eps, residual=res)
    q = glu.fp8_quantize(n)
    pre = [glu.fp8_linear(*q, *m, out_dtype=t) for m in (layer.gate, layer.up)]
    a, ea = ref.glu64(*(v for z in zip(*(ref.add64(p, n, *ab, index, w.scale) for p, ab in zip(pre, (w.gate, w.up)))) for v in z))
    act = glu.adapter_glu(*pre, n, *w.gate, *w.up, index, w.scale)
    torch.cuda.synchronize()
    check_store("activation", act, a, ea)
    out = glu.fp8_linear(*glu.fp8_quantize(act), *layer.down, out_dtype=t)
    want, bound = ref.add64(out, act, *w.down, index, w.scale)
    assert torch.equal(h, h2)
    check_store("y", y, want, bound)
    bare = layer(x, res, w, torch.full_like(index, -1))[0].double()
    plain = layer(x, res)[0].double()
    # 8-bit values of the activation, of 2^-4 at most each and unbiased, once from 16 bits and once from fp32
    assert float((bare - plain).norm() / plain.norm()) < 2.0 ** -4


@pytest.mark.parametrize("M", [6, 700])
def test_training_step(M):
    """residual + frozen projection + adapter behind dropout: gradients of x, a and b against the definition in 64 bits."""
    K, N, R, L, t = 128, 160, 8, 3, torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(M)
    weight = (rand(g, N, K) * K ** -0.5).to(t)
    x, a, b = ((rand(g, *s) * c).to(t).requires_grad_() for s, c in (((M, K), 1), ((L, R, K), K ** -0.5), ((L, N, R), R ** -0.5)))
    res, dout = rand(g, M, N).to(t), rand(g, M, N).to(t)
    index = torch.randint(-1, L, (M,), generator=g, device=DEV).int()
    scale = torch.rand(L, generator=g, device=DEV) + 0.5
    seed = torch.tensor([99], device=DEV)
    dropped = glu.dropout(x, 0.25, seed, 3)
    y = glu.adapter_add(x.detach() @ weight.t(), dropped, a, b, index, scale)
    out = glu.dropout(y, 0.5, 7, residual=res)
    out.backward(dout)
    # the chain, a call at a time: each gradient is the definition's of the one behind it
    dy = dropout_ref.dropout32(dout, 0.5, 7, 0)
    drop = dropout_ref.dropout32(x.detach(), 0.25, 99, 3)
    assert torch.equal(dropped, drop)
    low = ref.low64(drop, a, index)[0].float()
    (dx, edx), (da, eda), (db, edb) = ref.backward64(dy, drop, a.detach(), b.detach(), index, low, scale)
    # low as the kernel kept it is off by its own sums
    elow = ref.low64(drop, a.detach(), index)[1] + 2.0 ** -24 * low.abs()
    for l, rows in ref.adapters_of(index, L):
        edb[l] += float(scale[l]) * (dy[rows].double().abs().t() @ elow[rows])
    check_store("da", a.grad, da, eda)
    check_store("db", b.grad, db, edb)
    kept = dropout_ref.draws(M, K, 99, 3, DEV) >= round(65536 * 0.25)
    c = 65536 / (65536 - round(65536 * 0.25))
    # two roundings to bf16: of dx behind the mask, and of the product with c
    want = torch.where(kept, dx * c, 0.0)
    check_store("dx", x.grad, want, torch.where(kept, c * (edx + 2.0 ** -8 * (dx.abs() + edx)), 0.0))
