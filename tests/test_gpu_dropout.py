"""dropout on the GPU: bit for bit its definition."""
import pytest
import torch

import dropout_ref as ref
import glu_mlp_gemv_amd as glu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SHAPES = [(1, 1), (1, 7), (3, 8), (2, 9), (203, 2560), (33, 777), (1, 32768), (1500, 33), (700, 1030)]


def tensors(M, K, t, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(M, K, generator=g, device=DEV).to(t) for _ in range(2)]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,K", SHAPES)
def test_dropout(M, K, residual, kind):
    x, r = tensors(M, K, T[kind], M + K)
    res = r if residual else None
    for p, seed, offset in ((0.1, 3, 0), (0.5, -1, 2 ** 40 + 3), (0.0, 2 ** 63, 1), (1.0, 7, 7), (1 / 65536, 1 << 32, 1 << 33)):
        got = glu.dropout(x, p, seed, offset, residual=res)
        at = torch.tensor([seed - (1 << 64) if seed >= 1 << 63 else seed], device=DEV)
        same = glu.dropout(x, p, at, offset, residual=res)
        want = ref.dropout32(x, p, seed, offset, res)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(same, want), (p, seed, offset)
    assert torch.equal(glu.dropout(x, 0.0, 1, residual=None), x)


def test_share_and_independence():
    """A million draws: the kept share, and that of pairs under two offsets, within six deviations."""
    x = torch.ones(1000, 1024, device=DEV)
    a, b = (glu.dropout(x, 0.3, 12345, offset) != 0 for offset in (0, 1))
    n, keep = x.numel(), 1 - round(65536 * 0.3) / 65536
    for hits, share in ((a, keep), (b, keep), (a & b, keep * keep)):
        assert abs(int(hits.sum()) - n * share) < 6 * (n * share * (1 - share)) ** 0.5


def test_views_and_places():
    """Rows apart, unaligned, in place in x and in the residual; the mask is that of dense rows."""
    M, K = 37, 101
    x, r = tensors(M, K, torch.bfloat16, 1)
    want = glu.dropout(x, 0.2, 9, 4, residual=r)
    vx = torch.full((M, K + 5), float("nan"), dtype=x.dtype, device=DEV)
    vr = vx.clone()
    vx[:, 1:K + 1], vr[:, 3:K + 3] = x, r
    for out in (None, vx[:, 1:K + 1], vr[:, 3:K + 3]):
        a, b = vx.clone(), vr.clone()
        o = None if out is None else (a[:, 1:K + 1] if out.data_ptr() == vx[:, 1:K + 1].data_ptr() else b[:, 3:K + 3])
        got = glu.dropout(a[:, 1:K + 1], 0.2, 9, 4, residual=b[:, 3:K + 3], out=o)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert a[:, 0].isnan().all() and a[:, K + 1:].isnan().all() and b[:, :3].isnan().all() and b[:, K + 3:].isnan().all()


def test_dropped_specials_do_not_show():
    x, r = tensors(50, 64, torch.bfloat16, 1)
    gone = glu.dropout(torch.ones_like(x), 0.5, 3) == 0
    x[gone] = float("nan")
    x[:10][gone[:10]] = float("inf")
    out = glu.dropout(x, 0.5, 3, residual=r)
    torch.cuda.synchronize()
    assert out.isfinite().all() and torch.equal(out[gone], r[gone])


def test_far_rows():
    x, r = tensors(3, 100, torch.bfloat16, 4)
    far = torch.empty((1 << 32) + 1000, dtype=torch.bfloat16, device=DEV)
    vx, vr, out = (f.as_strided((3, 100), (1 << 31, 1)) for f in (far, far[200:], torch.empty_like(far)))
    vx.copy_(x)
    vr.copy_(r)
    glu.dropout(vx, 0.3, 5, residual=vr, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, ref.dropout32(x, 0.3, 5, 0, r))


def test_empty():
    for shape in ((0, 8), (8, 0)):
        x = torch.empty(shape, device=DEV)
        assert glu.dropout(x, 0.5, 1).shape == shape


def test_gradients():
    """The gradient is the same mask on the upstream one, the residual's is the upstream one; expanded, and by a seed tensor."""
    x, r = (t.requires_grad_() for t in tensors(20, 50, torch.float32, 2))
    seed = torch.tensor([77], device=DEV)
    for s in (77, seed):
        out = glu.dropout(x, 0.25, s, 5, residual=r)
        w = torch.randn(50, device=DEV)
        dx, dr = torch.autograd.grad((out * w).sum(), (x, r))
        assert torch.equal(dx, ref.dropout32(w.expand(20, 50), 0.25, 77, 5)) and torch.equal(dr, w.expand(20, 50))
    # differences, exact for a linear function up to fp32
    v = torch.randn_like(x)
    f = lambda x: (glu.dropout(x, 0.25, 77, 5).double() * w.double()).sum()  # noqa: E731
    with torch.no_grad():
        slope, along = f(x + v) - f(x - v), 2 * (dx.double() * v.double()).sum()
    assert abs(slope - along) <= 2.0 ** -20 * (dx.abs() * (x.abs() + v.abs())).sum().double() * 4
    out = glu.dropout(x, 0.25, seed, 5)
    seed.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        out.sum().backward()
    out = glu.dropout(x.detach(), 0.25, seed, 5, residual=r)
    assert torch.autograd.grad(out.sum(), r)[0].eq(1).all()
    with pytest.raises(RuntimeError, match="no gradient"):
        glu.dropout(x, 0.25, 1, out=torch.empty_like(x))
    (dx,) = torch.autograd.grad(glu.dropout(x, 0.5, 1).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_graph_draws_anew_by_the_seed_tensor():
    x, r = tensors(64, 200, torch.bfloat16, 3)
    seed = torch.tensor([5], device=DEV)
    glu.dropout(x, 0.3, seed, 2, residual=r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = glu.dropout(x, 0.3, seed, 2, residual=r)
        fixed = glu.dropout(x, 0.3, 5, 2)
    for s in (5, 6, 1 << 40):
        seed.fill_(s)
        graph.replay()
        want, same = glu.dropout(x, 0.3, s, 2, residual=r), glu.dropout(x, 0.3, 5, 2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(fixed, same)


def test_streams():
    x, r = tensors(64, 200, torch.bfloat16, 3)
    want = glu.dropout(x, 0.3, 1, residual=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = glu.dropout(x, 0.3, 1, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_argument_refusals():
    x, r = tensors(4, 8, torch.bfloat16, 3)
    for bad, args, kw in [(TypeError, (x.double(), 0.1, 1), {}), (TypeError, (x, 0.1, 1), dict(residual=r.half())),
                          (ValueError, (x, 1.5, 1), {}), (ValueError, (x, -0.1, 1), {}), (ValueError, (x[0], 0.1, 1), {}),
                          (ValueError, (x.cpu(), 0.1, 1), {}), (ValueError, (x, 0.1, 1), dict(residual=r[:3])),
                          (TypeError, (x, 0.1, torch.tensor([1], dtype=torch.int32, device=DEV)), {}),
                          (ValueError, (x, 0.1, torch.tensor([1, 2], device=DEV)), {}), (ValueError, (x.t(), 0.1, 1), {}),
                          (TypeError, (x, 0.1, 1.5), {})]:
        with pytest.raises(bad):
            glu.dropout(*args, **kw)
