"""Logits of the experts' router: the C ABI's refusals on the host, the product and the layer that ranks by it on the GPU."""
import pytest
import torch

import glu_mlp_gemv_amd as glu
import moe_ref
from fp8_ref import U, check_store
from glu_mlp_gemv_amd import api, mlp, moe

OK, NULLP, SHAPE, ALIGN, ALIAS, LAUNCH, UNSUP, STRIDE = range(8)
ARG = 10
BF16, FP16, FP32, E4M3 = range(4)
P = [0x100000000 + i * 0x10000000 for i in range(3)]  # made up: every call here is refused or empty
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=FP32), ARG), (dict(dtype=E4M3), ARG), (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=-1), SHAPE),
    (dict(K=(1 << 24) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(x=None), NULLP), (dict(router=None), NULLP),
    (dict(logits=None), NULLP), (dict(ldx=63), STRIDE), (dict(ldr=63), STRIDE), (dict(ldx=1 << 62), STRIDE),
    (dict(x=P[0] + 1), ALIGN), (dict(logits=P[2] + 2), ALIGN), (dict(logits=P[0]), ALIAS), (dict(logits=P[1] + 4), ALIAS),
    (dict(M=0), OK), (dict(M=0, x=None, router=None, logits=None), OK),
])
def test_refusals(kw, status):
    k = dict(x=P[0], ldx=64, router=P[1], ldr=64, logits=P[2], M=3, K=64, E=8, dtype=BF16)
    k.update(kw)
    assert api.library().glu_moe_logits(k["x"], k["ldx"], k["router"], k["ldr"], k["logits"], k["M"], k["K"], k["E"], k["dtype"],
                                        None) == status


def operands(M, K, E, t, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(M, K, generator=g, device=DEV).to(t), (torch.randn(E, K, generator=g, device=DEV) * K ** -0.5).to(t))


def check_logits(got, x, router):
    """fp32 sums (twice an operation's rounding on the matrix unit): 64 numbers a wave and stage, 16 waves."""
    want = x.double() @ router.double().t()
    bound = 2 * U * (x.shape[1] / 16 + 40) * (x.double().abs() @ router.double().abs().t())
    check_store("logits", got, want, bound)
    return want, bound


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,E", [(1, 2560, 64), (1, 64, 1), (3, 7, 5), (16, 4100, 128), (17, 130, 17), (64, 1024, 256), (65, 200, 40),
                                   (200, 96, 1024), (1, 8, 1000), (5, 16384, 33)])
def test_product(M, K, E, kind):
    x, router = operands(M, K, E, T[kind], M + K)
    got = moe.moe_logits(x, router)
    torch.cuda.synchronize()
    check_logits(got, x, router)
    wide = torch.full((M, K + 3), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, 1:K + 1] = x
    far = torch.full((E, K + 5), float("nan"), dtype=x.dtype, device=DEV)
    far[:, :K] = router
    assert torch.equal(moe.moe_logits(wide[:, 1:K + 1], far[:, :K]), got), "rows apart, unaligned"
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = moe.moe_logits(x, router, stream=side)
    side.synchronize()
    assert torch.equal(other, got)


@pytest.mark.gpu
def test_rows_do_not_touch_each_other_and_empty_sizes():
    x, router = operands(20, 100, 30, torch.bfloat16, 1)
    want = moe.moe_logits(x, router)
    x[3], router[7] = float("nan"), float("inf")
    got = moe.moe_logits(x, router)
    fine = torch.ones_like(got, dtype=torch.bool)
    fine[3], fine[:, 7] = False, False
    torch.cuda.synchronize()
    assert torch.equal(got[fine], want[fine]) and got[3].isnan().all() and not got[:, 7].isfinite().any()
    assert moe.moe_logits(x[:0], router).shape == (0, 30)
    assert not moe.moe_logits(x[:, :0], router[:, :0]).any()


@pytest.mark.gpu
def test_python_refusals():
    x, router = operands(4, 64, 8, torch.bfloat16, 1)
    for bad, a in [(TypeError, (x.float(), router)), (TypeError, (x, router.half())), (ValueError, (x, router[:, :60])),
                   (ValueError, (x, router[:0])), (ValueError, (x, router[:1].expand(1025, 64))), (ValueError, (x.cpu(), router)),
                   (ValueError, (x[0], router)), (RuntimeError, (x.clone().requires_grad_(), router))]:
        with pytest.raises(bad):
            moe.moe_logits(*a)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,E,top", [(6, 256, 128, 8, 2), (40, 512, 96, 128, 8), (24, 1024, 64, 64, 6)])
def test_layer_ranks_by_unrounded_logits(M, K, N, E, top, kind):
    """mlp.ExpertGluMlp chooses the experts of logits in 64 bits, wherever their gap says so, and weighs them by those."""
    t = T[kind]
    g = torch.Generator(device=DEV).manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, res = rand(M, K).to(t), rand(M, K).to(t)
    gate, up, down = ((rand(E, a, b) * b ** -0.5).to(t) for a, b in ((N, K), (N, K), (K, N)))
    router = (1.0 + 0.1 * rand(E, K)).to(t)  # logits close together, of which 16 bits make ties
    router *= K ** -0.5
    norm = torch.ones(K, dtype=t, device=DEV)
    y, h = mlp.ExpertGluMlp(norm, router, gate, up, down, top)(x, res)
    n, h2 = glu.add_rms_norm(x, norm, 1e-6, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(h, h2)
    logits, bound = check_logits(moe.moe_logits(n, router), n, router)
    best = logits.sort(1, descending=True).values
    clear = (best[:, top - 1] - best[:, top] > 4 * bound.amax(1)) if top < E else torch.ones(M, dtype=torch.bool, device=DEV)
    assert clear.float().mean() > 0.5
    rounded = (moe_ref.chosen(logits.to(t), top) != moe_ref.chosen(logits, top)).any(1)
    assert kind == "fp16" or E < 64 or rounded.any(), "in 16 bits the choice would be another"
    want, err = moe_ref.moe64(n, logits, gate, up, down, top)
    # a logit off by `bound` changes weights by twice that, relative
    err = err + 4 * bound.amax(1, keepdim=True) * spread(n, logits, gate, up, down, top)
    check_store("y", y[clear], want[clear], err[clear])


def spread(n, logits, gate, up, down, top):
    """Sum over a row's experts of the magnitude that each adds."""
    out = torch.zeros(n.shape, dtype=torch.double, device=n.device)
    take = moe_ref.chosen(logits, top)
    p = moe_ref.weights(logits, take, True)
    for e in take.any(0).nonzero()[:, 0].tolist():
        rows = take[:, e].nonzero()[:, 0]
        a = n[rows].double() @ gate[e].double().t()
        a = a * torch.sigmoid(a) * (n[rows].double() @ up[e].double().t())
        out[rows] += p[rows, e, None] * (a @ down[e].double().t()).abs()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [3, 20, 70])
def test_layer_in_a_graph(M, kind):
    """Captured once and replayed over values of very different sizes, with eager work between: nothing is left of the last."""
    t, K, N, E, top = T[kind], 128, 100, 8, 2
    g = torch.Generator(device=DEV).manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    router, norm = (rand(E, K) * K ** -0.5).to(t), torch.ones(K, dtype=t, device=DEV)
    gate, up, down = ((rand(E, a, b) * b ** -0.5).to(t) for a, b in ((N, K), (N, K), (K, N)))
    x, res = rand(M, K).to(t), rand(M, K).to(t)
    layer = mlp.ExpertGluMlp(norm, router, gate, up, down, top)
    layer(x, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = layer(x, res)
    for size in (1.0, 2.0 ** 9, 2.0 ** -9, 1.0):
        x.copy_(rand(M, K))
        up.copy_(rand(E, N, K) * size)
        down.copy_(rand(E, K, N) / size / 16)
        graph.replay()
        eager, eager_h = layer(x, res)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(h, eager_h) and y.isfinite().all()
