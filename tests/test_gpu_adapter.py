"""adapter_add, adapter_glu and adapter_backward on the GPU against their definition in 64 bits."""
import pytest
import torch

import adapter_ref as ref
import glu_mlp_gemv_amd as glu
from fp8_ref import check_store
from glu_mlp_gemv_amd import adapters, autograd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "fp16": torch.float16}

# one row; one tile of 16 rows and one more; odd everything; every row its own adapter; ranks at and past a matrix instruction's 16
# and a tile's 64; more rows than a small batch; the largest rank; widths below a stage
SHAPES = [(1, 64, 64, 8, 1), (1, 2560, 9216, 16, 8), (2, 4100, 300, 4, 3), (3, 7, 9, 1, 2), (16, 128, 256, 16, 16),
          (17, 100, 75, 5, 3), (33, 130, 257, 17, 40), (64, 512, 520, 32, 16), (100, 1030, 1027, 24, 9),
          (256, 256, 192, 64, 31), (257, 64, 64, 64, 2), (300, 520, 333, 33, 5), (1000, 1030, 900, 48, 7),
          (40, 96, 100, 100, 6), (270, 200, 130, 256, 3), (5, 300, 70, 256, 2), (2050, 256, 260, 16, 3),
          # mixtures of more rows, ranks past a tile's among them, and rows past the largest mixture, an adapter for each
          (520, 192, 130, 20, 40), (1024, 72, 200, 8, 300), (600, 64, 68, 72, 50), (1100, 64, 70, 16, 1100)]


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def index_of(g, M, L, order):
    """Adapters by row, some rows without one; "wild": also numbers that name none."""
    if order == "segments":
        i = torch.arange(M, device=DEV) * L // M
        i[M - M // 5:] = -1
    else:
        i = torch.randint(-1, L, (M,), generator=g, device=DEV)
        if order == "wild":
            i[::3] = torch.tensor([L, -7, 2 ** 31 - 1, -2 ** 31], device=DEV).repeat(M)[:len(i[::3])]
    return i.to(torch.int32)


def operands(M, K, N, R, L, t, order, seed, sides=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    y = [rand(g, M, N).to(t) for _ in range(sides)]
    x = rand(g, M, K).to(t)
    ab = [((rand(g, L, R, K) * K ** -0.5).to(t), (rand(g, L, N, R) * R ** -0.5).to(t)) for _ in range(sides)]
    scale = torch.rand(L, generator=g, device=DEV) + 0.5
    return y, x, ab, index_of(g, M, L, order), scale


def spaced(t, gap=3):
    """The same values as a view whose rows lie apart, NaN between them."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + gap), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["mixed", "segments", "wild"])
@pytest.mark.parametrize("M,K,N,R,L", SHAPES)
def test_add(M, K, N, R, L, order, kind):
    print(f"[adapter add] {M=} {K=} {N=} {R=} {L=} {order} {kind}", flush=True)
    (y,), x, ((a, b),), index, scale = operands(M, K, N, R, L, T[kind], order, M + K)
    want, bound = ref.add64(y, x, a, b, index, scale)
    out, low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)
    torch.cuda.synchronize()
    check_store("out", out, want, bound)
    t, err = ref.low64(x, a, index)
    check_store("low", low, t, err)
    assert torch.equal(out[(index < 0) | (index >= L)], y[(index < 0) | (index >= L)])
    assert torch.equal(out, glu.adapter_add(y, x, a, b, index, scale)), "the same bits without low, and again"


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["mixed", "segments"])
@pytest.mark.parametrize("M,K,N,R,L", SHAPES)
def test_glu(M, K, N, R, L, order, kind):
    print(f"[adapter glu] {M=} {K=} {N=} {R=} {L=} {order} {kind}", flush=True)
    (g, u), x, ((ga, gb), (ua, ub)), index, scale = operands(M, K, N, R, L, T[kind], order, M + N, 2)
    want, bound = ref.glu64(*(v for pair in zip(ref.add64(g, x, ga, gb, index, scale), ref.add64(u, x, ua, ub, index, scale))
                              for v in pair))
    out = glu.adapter_glu(g, u, x, ga, gb, ua, ub, index, scale)
    torch.cuda.synchronize()
    check_store("out", out, want, bound)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["mixed", "segments", "wild"])
@pytest.mark.parametrize("M,K,N,R,L", SHAPES + [(512, 70, 300, 16, 4), (513, 70, 300, 16, 4), (3000, 600, 64, 16, 700),
                                                (5000, 260, 1030, 40, 3)])
def test_backward(M, K, N, R, L, order, kind):
    print(f"[adapter backward] {M=} {K=} {N=} {R=} {L=} {order} {kind}", flush=True)
    t = T[kind]
    (dout,), x, ((a, b),), index, scale = operands(M, K, N, R, L, t, order, M + R)
    dout *= 0.1
    low = ref.low64(x, a, index)[0].float()
    want = ref.backward64(dout, x, a, b, index, low, scale)
    got = glu.adapter_backward(dout, x, a, b, index, low, scale)
    torch.cuda.synchronize()
    for name, v, (w, bound) in zip(("dx", "da", "db"), got, want):
        check_store(name, v, w, bound)
    again = glu.adapter_backward(dout, x, a, b, index, low, scale)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "a second call gives the same bits"
    for wanted in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        part = glu.adapter_backward(dout, x, a, b, index, low, scale, wanted=wanted)
        for p, q, w in zip(part, got, wanted):
            assert torch.equal(p, q) if w else p is None


@pytest.mark.parametrize("M", [5, 300])
def test_views(M):
    """Rows apart, NaN in the gaps, unaligned starts, outputs in place; adapters as slices of a wider stack."""
    K, N, R, L = 100, 83, 6, 4
    (y,), x, ((a, b),), index, scale = operands(M, K, N, R, L, torch.bfloat16, "mixed", 5)
    out = glu.adapter_add(y, x, a, b, index, scale)
    vy, vx, va, vb = spaced(y), spaced(x), spaced(a), spaced(b, 5)
    assert torch.equal(out, glu.adapter_add(vy, vx, va, vb, index, scale))
    into = spaced(torch.zeros_like(y))
    assert glu.adapter_add(vy, vx, va, vb, index, scale, out=into) is into and torch.equal(out, into)
    assert glu.adapter_add(vy, vx, va, vb, index, scale, out=vy) is vy and torch.equal(out, vy)
    torch.cuda.synchronize()
    assert vy._base[..., N:].isnan().all() and into._base[..., N:].isnan().all(), "nothing is written between rows"
    low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)[1]
    for p, q in zip(glu.adapter_backward(y, x, a, b, index, low, scale),
                    glu.adapter_backward(spaced(y), vx, va, vb, index, low, scale)):
        assert torch.equal(p, q)
    g = glu.adapter_glu(y, y, x, a, b, a, b, index, scale)
    assert torch.equal(g, glu.adapter_glu(spaced(y), y, vx, va, vb, a, b, index, scale))
    u = y.clone()
    assert torch.equal(g, glu.adapter_glu(y, u, x, a, b, a, b, index, scale, out=u))


@pytest.mark.parametrize("M", [64, 65, 300, 1024])
def test_one_adapter_of_many_held(M):
    """A run of rows that the sizes alone do not tell from a mixture, and rows without an adapter in between."""
    (y,), x, ((a, b),), index, scale = operands(M, 128, 200, 16, 100, torch.bfloat16, "mixed", 6)
    index.fill_(71)
    index[5:40] = -1
    want, bound = ref.add64(y, x, a, b, index, scale)
    out, low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)
    torch.cuda.synchronize()
    check_store("out", out, want, bound)
    check_store("low", low, *ref.low64(x, a, index))


def test_no_scale_is_one():
    (y,), x, ((a, b),), index, _ = operands(20, 64, 64, 8, 3, torch.float16, "mixed", 1)
    assert torch.equal(glu.adapter_add(y, x, a, b, index), glu.adapter_add(y, x, a, b, index, torch.ones(3, device=DEV)))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [40, 400])
def test_nan_and_infinity_stay_in_their_rows(M, kind):
    t = T[kind]
    (y,), x, ((a, b),), index, scale = operands(M, 96, 100, 12, 5, t, "mixed", 9)
    clean = glu.adapter_add(y, x, a, b, index, scale)
    low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)[1]
    grads = glu.adapter_backward(y, x, a, b, index, low, scale)
    index[3], index[7] = 1, 2
    x2, a2, b2 = x.clone(), a.clone(), b.clone()
    a2[1] = float("nan")
    b2[2] = float("inf")
    x2[index == 1] = float("inf")
    x2[index == -1] = float("nan")
    out = glu.adapter_add(y, x2, a2, b2, index, scale)
    torch.cuda.synchronize()
    fine = (index != 1) & (index != 2)
    fine[3] = fine[7] = False
    assert torch.equal(out[fine], clean[fine])
    assert out[index == 1].isnan().all() and not out[index == 2].isfinite().all()
    dx, da, db = glu.adapter_backward(y, x2, a2, b2, index, low, scale)
    torch.cuda.synchronize()
    assert torch.equal(dx[fine], grads[0][fine])
    keep = (0, 3, 4)
    own = glu.adapter_backward(y, torch.where(fine[:, None], x, 0.0).to(t), a, b, index, low, scale)
    assert all(torch.equal(da[l], own[1][l]) and torch.equal(db[l], own[2][l]) for l in keep)


def test_large_and_tiny_hidden_values_in_fp16():
    """t of some 1e6 and of 1e-9, beyond fp16 on either side, are kept in 32 bits."""
    (y,), x, ((a, b),), index, scale = operands(24, 256, 64, 16, 3, torch.float16, "mixed", 3)
    x[:8] = x[:8] * 4000
    a *= 4
    x[8:16] = x[8:16] * 2.0 ** -14
    want, bound = ref.add64(torch.zeros_like(y), x, a, b * 2.0 ** -6, index, scale)
    out = glu.adapter_add(torch.zeros_like(y), x, a, b * 2.0 ** -6, index, scale)
    torch.cuda.synchronize()
    check_store("out", out, want, bound)


@pytest.mark.parametrize("M,N", [(0, 64), (5, 0), (0, 0)])
def test_empty(M, N):
    (y,), x, ((a, b),), index, scale = operands(max(M, 1), 64, max(N, 1), 8, 3, torch.bfloat16, "segments", 2)
    y, x, b, index = y[:M, :N], x[:M], b[:, :N], index[:M]
    out, low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)
    assert out.shape == (M, N)
    check_store("low", low, *ref.low64(x, a, index))
    dx, da, db = glu.adapter_backward(y, x, a, b, index, low, scale)
    torch.cuda.synchronize()
    assert dx.shape == (M, 64) and not dx.any() and not da.any() and not db.any() and db.shape == (3, N, 8)


@pytest.mark.parametrize("K,N", [(0, 96), (96, 0)])
def test_backward_of_empty_products(K, N):
    """One width empty, with more rows than one item."""
    M, R, L = 600, 8, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    t = torch.bfloat16
    dout, x = rand(g, M, N).to(t), rand(g, M, K).to(t)
    a, b, low = rand(g, L, R, K).to(t), rand(g, L, N, R).to(t), rand(g, M, R)
    index = index_of(g, M, L, "mixed")
    dx, da, db = glu.adapter_backward(dout, x, a, b, index, low)
    torch.cuda.synchronize()
    for name, v, (w, bound) in zip(("dx", "da", "db"), (dx, da, db), ref.backward64(dout, x, a, b, index, low, None)):
        check_store(name, v, w, bound)


@pytest.mark.parametrize("M,L", [(600, 3), (300, 100)])
def test_far_rows(M, L):
    """Rows 2^23 elements apart: offsets past 32 bits in x, y and out, with the largest row stride."""
    K, N, R, t = 128, 96, 16, torch.bfloat16
    (y,), x, ((a, b),), index, scale = operands(M, K, N, R, L, t, "mixed", 8)
    far = torch.empty(M, 1 << 23, dtype=t, device=DEV)
    vx, vy, out = far[:, :K], far[:, 1000:1000 + N], torch.empty_like(far)[:, :N]  # an output's span may hold no input
    vx.copy_(x)
    vy.copy_(y)
    want, low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)
    assert torch.equal(glu.adapter_add(vy, vx, a, b, index, scale, out=out), want)
    for p, q in zip(glu.adapter_backward(vy, vx, a, b, index, low, scale), glu.adapter_backward(y, x, a, b, index, low, scale)):
        assert torch.equal(p, q)


def test_no_columns_of_x():
    y = torch.randn(5, 64, device=DEV).bfloat16()
    x, a, b = y[:, :0], torch.empty(2, 4, 0, dtype=y.dtype, device=DEV), torch.ones(2, 64, 4, dtype=y.dtype, device=DEV)
    index = torch.tensor([0, 1, -1, 0, 1], dtype=torch.int32, device=DEV)
    assert torch.equal(glu.adapter_add(y, x, a, b, index), y)


@pytest.mark.parametrize("M", [7, 700])
def test_gradients_through_autograd(M):
    """Against the 64-bit definition, for every operand, with a gradient that autograd expands; and against differences."""
    t = torch.bfloat16
    (y,), x, ((a, b),), index, scale = operands(M, 64, 96, 8, 3, t, "mixed", 11)
    leaves = [v.clone().requires_grad_() for v in (y, x, a, b)]
    out = glu.adapter_add(*leaves, index, scale)
    assert torch.equal(out.detach(), glu.adapter_add(y, x, a, b, index, scale))
    w = torch.randn(96, device=DEV).to(t)
    (out * w).sum().backward()
    low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)[1]
    dout = w.expand(M, 96)
    assert torch.equal(leaves[0].grad, dout)
    for name, leaf, (want, bound) in zip(("dx", "da", "db"), leaves[1:], ref.backward64(dout, x, a, b, index, low, scale)):
        check_store(name, leaf.grad, want, bound)
    # a step along a direction in each of x, a and b, in 64 bits
    f = lambda x, a, b: (ref_out(y, x, a, b, index, scale) * w.double()).sum()  # noqa: E731
    for i, leaf in enumerate(leaves[1:]):
        ops = [x.double(), a.double(), b.double()]
        v = torch.randn(ops[i].shape, device=DEV, dtype=torch.double)
        up, down = list(ops), list(ops)
        up[i], down[i] = ops[i] + 1e-4 * v, ops[i] - 1e-4 * v
        slope = (f(*up) - f(*down)) / 2e-4
        along = (leaf.grad.double() * v).sum()
        # each element of the gradient is off by half a step of bf16 at most, and a little for its fp32 sums
        assert abs(slope - along) <= 2 * (2.0 ** -8 * leaf.grad.double().abs() * v.abs()).sum()
    frozen = glu.adapter_add(y, x, leaves[2], b, index, scale)
    torch.autograd.grad(frozen.sum(), leaves[2])
    y2 = y.clone().requires_grad_()
    assert torch.autograd.grad(glu.adapter_add(y2, x, a, b, index, scale).sum(), y2)[0].eq(1).all()


def ref_out(y, x, a, b, index, scale):
    out = y.double().clone()
    for l, rows in ref.adapters_of(index, a.shape[0]):
        out[rows] += float(scale[l]) * (x[rows] @ a[l].t() @ b[l].t())
    return out


def test_gradient_refusals():
    (y,), x, ((a, b),), index, scale = operands(4, 64, 64, 8, 2, torch.bfloat16, "mixed", 1)
    a.requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        glu.adapter_add(y, x, a, b, index, scale, out=y)
    with pytest.raises(RuntimeError, match="no gradient"):
        glu.adapter_glu(y, y, x, a, b, a, b, index, scale)
    with pytest.raises(RuntimeError, match="scale"):
        glu.adapter_add(y, x, a, b, index, scale.clone().requires_grad_())
    out = glu.adapter_add(y, x, a, b, index, scale)
    (grad,) = torch.autograd.grad(out.sum(), a, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()
    with torch.no_grad():
        glu.adapter_add(y, x, a, b, index, scale, out=y)


@pytest.mark.parametrize("M", [3, 600])
def test_graph_replays(M):
    """Forward and backward captured, replayed over new values with eager work between."""
    (y,), x, ((a, b),), index, scale = operands(M, 128, 192, 16, 4, torch.bfloat16, "mixed", 4)
    glu.adapter_backward(y, x, a, b, index, glu.adapter_add(y, x, a, b, index, scale, return_low=True)[1], scale)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)
        grads = glu.adapter_backward(out, x, a, b, index, low, scale)
    for seed in range(4):
        (y2,), x2, ((a2, b2),), index2, scale2 = operands(M, 128, 192, 16, 4, torch.bfloat16, "mixed", 50 + seed)
        for old, new in zip((y, x, a, b, index, scale), (y2, x2, a2, b2, index2, scale2)):
            old.copy_(new)
        graph.replay()
        eager, elow = glu.adapter_add(y2, x2, a2, b2, index2, scale2, return_low=True)
        egrads = glu.adapter_backward(eager, x2, a2, b2, index2, elow, scale2)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(low, elow)
        assert all(torch.equal(p, q) for p, q in zip(grads, egrads))


def test_streams():
    """The current stream, and a stream given, each after work that makes the operands there."""
    (y,), x, ((a, b),), index, scale = operands(50, 256, 320, 16, 4, torch.bfloat16, "mixed", 4)
    want = glu.adapter_add(y, x, a, b, index, scale)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2 = x * 1.0
        got = glu.adapter_add(y, x2, a, b, index, scale)
    assert torch.equal(glu.adapter_add(y, x, a, b, index, scale, stream=side), want)
    side.synchronize()
    assert torch.equal(got, want)
    low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)[1]
    grads = glu.adapter_backward(y, x, a, b, index, low, scale)
    torch.cuda.synchronize()
    other = glu.adapter_backward(y, x, a, b, index, low, scale, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(grads, other))


def test_argument_refusals():
    (y,), x, ((a, b),), index, scale = operands(4, 64, 64, 8, 2, torch.bfloat16, "mixed", 1)
    add = glu.adapter_add
    for bad, kw in [(TypeError, dict(y=y.float())), (TypeError, dict(x=x.half())), (TypeError, dict(a=a.half())),
                    (TypeError, dict(index=index.long())), (TypeError, dict(scale=scale.half())), (TypeError, dict(scale=2.0)),
                    (ValueError, dict(x=x[:3])), (ValueError, dict(a=a[:, :, :60])), (ValueError, dict(b=b[:1])),
                    (ValueError, dict(b=b[:, :, :4])), (ValueError, dict(index=index[:3])), (ValueError, dict(scale=scale[:1])),
                    (ValueError, dict(a=a[:0], b=b[:0])), (ValueError, dict(a=a[:, :0], b=b[:, :, :0])),
                    (ValueError, dict(x=x.t().contiguous().t())), (ValueError, dict(a=a[:1].expand(2, 8, 64))),
                    (ValueError, dict(y=y[:1].expand(4, 64))), (ValueError, dict(x=x.cpu())), (ValueError, dict(y=y[0]))]:
        with pytest.raises(bad):
            add(**{**dict(y=y, x=x, a=a, b=b, index=index, scale=scale), **kw})
    with pytest.raises(Exception, match="ALIAS"):
        add(y, x, a, b, index, scale, out=x)
    wide = torch.zeros(2, 257, 64, dtype=a.dtype, device=DEV)
    with pytest.raises(ValueError, match="rank"):
        add(y, x, wide, wide.transpose(1, 2).contiguous(), index, scale)
    low = torch.zeros(4, 8, device=DEV)
    with pytest.raises(TypeError):
        glu.adapter_backward(y, x, a, b, index, low.double(), scale)
    with pytest.raises(ValueError):
        glu.adapter_backward(y, x, a, b, index, low[:, :7], scale)
    assert adapters.MAX_RANK == 256 and autograd.AdapterAdd
