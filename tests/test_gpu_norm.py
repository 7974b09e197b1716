"""add_rms_norm, add_rms_norm_fp8 and add_rms_norm_backward on the GPU against their definition in 64 bits."""
import pytest
import torch

import fp8_ref as ref
import glu_mlp_gemv_amd as glu
from glu_mlp_gemv_amd.api import GluError

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# one chunk, part of a group, odd widths, one lane past a wave, several waves, one and two chunks per lane, rows past a
# workgroup's registers
SHAPES = [(1, 1), (1, 2560), (3, 5), (7, 127), (5, 128), (2, 129), (4, 513), (203, 2560), (33, 777), (1030, 1025),
          (1100, 4096), (6, 8192), (2, 9001), (1, 32768), (3, 33000), (1500, 512), (1025, 96)]


def tensors(M, K, t, seed, *scales):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(M, K, generator=g, device=DEV) * s).to(t) for s in scales]


def weight(K, t, seed):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000)
    return (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(t)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, residual, kind):
    t = T[kind]
    print(f"[norm] M={M} K={K} {kind} residual={residual}", flush=True)
    x, r = tensors(M, K, t, M + K, 1.0, 3.0)
    w = weight(K, t, K)
    res = r if residual else None
    h, y, rstd, err = ref.norm64(x, w, EPS, res)
    gy, gh, grstd = glu.add_rms_norm(x, w, EPS, residual=res, return_rstd=True)
    torch.cuda.synchronize()
    ref.check_store("y", gy, y, err)
    assert torch.equal(gh, h)
    assert gh is x or residual
    assert ((grstd.double() - rstd).abs() <= 40 * ref.U * rstd).all()
    q, s, gh = glu.add_rms_norm_fp8(x, w, EPS, residual=res)
    torch.cuda.synchronize()
    assert q.dtype is ref.E4M3 and tuple(s.shape) == (M, ref.groups(K)) and s.t().is_contiguous()
    ref.check_e4m3("y in e4m3", q, s, y, err)
    assert torch.equal(gh, h)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,K", SHAPES + [(2, 17000), (70, 20000)])
def test_backward(M, K, residual, kind):
    t = T[kind]
    print(f"[norm grad] M={M} K={K} {kind} residual={residual}", flush=True)
    h, dy, dr = tensors(M, K, t, M + K, 3.0, 0.1, 0.1)
    w = weight(K, t, K)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dres = dr if residual else None
    dx, edx, dw, edw = ref.grad64(dy, h, w, rstd, dres)
    gx, gw = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dres)
    torch.cuda.synchronize()
    ref.check_store("dx", gx, dx, edx)
    ref.check_store("dweight", gw, dw, edw)
    gx2, gw2 = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dres)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2), "a second call gives the same bits"


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [2, 5, 7, 16, 17, 33, 64, 65, 300, 3090, 6001])
@pytest.mark.parametrize("K", [5, 192, 512, 520, 1030, 2560, 5100])
def test_backward_workgroups(M, K, kind):
    """Rows that one workgroup's teams share unevenly, and more."""
    t = T[kind]
    print(f"[norm grad] M={M} K={K} {kind}", flush=True)
    h, dy, dr = tensors(M, K, t, M * K, 3.0, 0.1, 0.1)
    w = weight(K, t, K)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, edx, dw, edw = ref.grad64(dy, h, w, rstd, dr)
    gx, gw = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dr)
    torch.cuda.synchronize()
    ref.check_store("dx", gx, dx, edx)
    ref.check_store("dweight", gw, dw, edw)


@pytest.mark.parametrize("M,K,residual", [(16390, 4099, False), (11000, 4099, True), (8300, 8200, False)])
def test_backward_past_the_cache(M, K, residual):
    """More than the last-level cache holds, which is then read past it."""
    t = torch.bfloat16
    print(f"[norm grad] M={M} K={K} residual={residual}", flush=True)
    h, dy, dr = tensors(M, K, t, M + K, 3.0, 0.1, 0.1)
    w = weight(K, t, K)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dres = dr if residual else None
    dx, edx, dw, edw = ref.grad64(dy, h, w, rstd, dres)
    gx, gw = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dres)
    torch.cuda.synchronize()
    ref.check_store("dx", gx, dx, edx)
    ref.check_store("dweight", gw, dw, edw)


def test_backward_many_columns():
    """More columns than one grid of threads joins."""
    M, K = 2, (1 << 27) + 33
    print(f"[norm grad] M={M} K={K}", flush=True)
    h, dy = tensors(M, K, torch.bfloat16, 8, 3.0, 0.1)
    w = weight(K, torch.bfloat16, 8)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    gx, gw = glu.add_rms_norm_backward(dy, h, w, rstd)
    torch.cuda.synchronize()
    # grad64 with the length of this mean's sum: K / 1024 steps a lane, 6 + 16 across lanes and waves
    r = rstd.double()[:, None]
    sums = [(dy[m].double() * w.double() * h[m].double() * r[m]) for m in range(M)]
    mean = torch.stack([s.mean() for s in sums])[:, None]
    near = torch.stack([s.abs().mean() for s in sums])[:, None] * ref.U * (K / 1024 + 40)
    del sums
    for at in (0, (1 << 26) - 300, K - 600):
        part = slice(at, at + 600)
        xh, g = h[:, part].double() * r, dy[:, part].double()
        a = g * w[part].double()
        ref.check_store("dx", gx[:, part], r * (a - xh * mean), r * (4 * ref.U * a.abs() + xh.abs() * (near + 4 * ref.U * mean.abs())))
        ref.check_store("dweight", gw[part], (g * xh).sum(0), 42 * ref.U * (g * xh).abs().sum(0))
    terms = dy.float() * (h.float() * rstd[:, None])
    # both sums in fp32
    tol = 1.01 * ref.half(torch.bfloat16) * terms.sum(0).abs() + 2 * 42 * ref.U * terms.abs().sum(0)
    assert ((gw.float() - terms.sum(0)).abs() <= tol).all()


def test_gradient_against_differences():
    """The backward's formula against central differences of the 64-bit definition, and the kernels'
    gradient through autograd against the same differences."""
    torch.manual_seed(3)
    M, K, step = 3, 130, 1e-4
    x, r = (torch.randn(M, K, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.1 * torch.randn(K, dtype=torch.float64)
    cy, ch = (torch.randn(M, K, dtype=torch.float64) for _ in range(2))

    def loss(x, r, w):
        h = x + r
        return float((h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w * cy).sum() + (h * ch).sum())

    leaves = [v.float().to(DEV).requires_grad_() for v in (x, w, r)]
    from glu_mlp_gemv_amd.autograd import rms_norm
    y, h = rms_norm(leaves[0], leaves[1], EPS, residual=leaves[2])
    ((y * cy.float().to(DEV)).sum() + (h * ch.float().to(DEV)).sum()).backward()
    torch.cuda.synchronize()
    assert torch.equal(leaves[0].grad, leaves[2].grad)
    gx, gw = leaves[0].grad.double().cpu(), leaves[1].grad.double().cpu()
    # differences: error step^2 f''' / 6 + rounding / step, both below 1e-6 here; fp32 gradients below 1e-5
    for i, j in ((0, 0), (1, 64), (2, 129)):
        d = torch.zeros_like(x)
        d[i, j] = step
        num = (loss(x + d, r, w) - loss(x - d, r, w)) / (2 * step)
        assert abs(num - float(gx[i, j])) < 2e-5 * (1 + abs(num))
    for j in (0, 77, 129):
        d = torch.zeros_like(w)
        d[j] = step
        num = (loss(x, r, w + d) - loss(x, r, w - d)) / (2 * step)
        assert abs(num - float(gw[j])) < 2e-5 * (1 + abs(num))


def test_autograd_forms():
    """No residual; a broadcast (expanded) gradient; a loss on the residual stream alone."""
    from glu_mlp_gemv_amd.autograd import rms_norm
    x, r = tensors(9, 300, torch.bfloat16, 5, 1.0, 1.0)
    w = weight(300, torch.bfloat16, 5)
    x.requires_grad_()
    w.requires_grad_()
    r.requires_grad_()
    y, h = rms_norm(x, w, EPS)
    assert h is x
    y.sum().backward()
    _, _, rstd, _ = ref.norm64(x.detach(), w.detach(), EPS, None)
    dx, edx, dw, edw = ref.grad64(torch.ones_like(x), x.detach(), w.detach(), rstd, None)
    # rstd itself carries 40 U, linearly into r and xhat
    ref.check_store("dx", x.grad, dx, edx + 200 * ref.U * dx.abs() + 200 * ref.U * (rstd[:, None] * w.detach().double().abs()))
    ref.check_store("dweight", w.grad, dw, edw + 80 * ref.U * (x.detach().double() * rstd[:, None]).abs().sum(0))
    x.grad = w.grad = None
    y, h = rms_norm(x, w, EPS, residual=r)
    h.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(r.grad, torch.ones_like(x)) and w.grad is None


@pytest.mark.parametrize("leaves", ["xwr", "x", "w", "r"])
@pytest.mark.parametrize("residual", [True, False])
def test_public_norm_keeps_gradients(residual, leaves):
    """add_rms_norm on operands that require a gradient is autograd's rms_norm, bit for bit."""
    from glu_mlp_gemv_amd.autograd import rms_norm
    made = tensors(9, 300, torch.bfloat16, 7, 1.0, 1.0, 1.0)
    w = weight(300, torch.bfloat16, 7)

    def grads(f):
        x, r, dy = (t.clone() for t in made)
        v = {"x": x, "w": w.clone(), "r": r}
        for name in leaves:
            v[name].requires_grad_()
        y, h = f(v["x"], v["w"], EPS, residual=v["r"] if residual else None)
        out = [y.detach().clone(), h.detach().clone()]
        if y.requires_grad:
            (y * dy + h).sum().backward()
        torch.cuda.synchronize()
        return out, [v[name].grad for name in leaves]
    (y, h), got = grads(glu.add_rms_norm)
    (wy, wh), want = grads(rms_norm)
    assert torch.equal(y, wy) and torch.equal(h, wh)
    for name, a, b in zip(leaves, got, want):
        assert (a is None) == (name == "r" and not residual)
        assert a is None or torch.equal(a, b)
    with torch.no_grad():
        (y, h), got = grads(glu.add_rms_norm)
    assert torch.equal(y, wy) and got == [None] * len(leaves)


def test_gradient_of_the_gradient_is_refused():
    from glu_mlp_gemv_amd.autograd import rms_norm
    x, r = tensors(5, 256, torch.float32, 6, 1.0, 1.0)
    w = weight(256, torch.float32, 6)
    x.requires_grad_()
    y, _ = rms_norm(x, w, EPS, residual=r)
    dx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.square().sum().backward()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_strides_and_alignment(kind):
    """Row-strided views that start at odd elements, and outputs into such views: what lies between is untouched."""
    t = T[kind]
    M, K = 21, 261
    big = tensors(M, 3 * K + 5, t, 9, 1.0)[0]
    x, r = big[:, 1:1 + K], big[:, K + 2:2 * K + 2]
    w = weight(K + 1, t, 9)[1:]
    h, y, _, err = ref.norm64(x, w, EPS, r)
    out = torch.full((M, K + 7), 5.0, dtype=t, device=DEV)
    ho = torch.full((M, K + 3), 7.0, dtype=t, device=DEV)
    gy, gh = glu.add_rms_norm(x, w, EPS, residual=r, out=out[:, 3:3 + K], residual_out=ho[:, 1:1 + K])
    torch.cuda.synchronize()
    ref.check_store("y", gy, y, err)
    assert torch.equal(gh, h)
    assert (out[:, :3] == 5).all() and (out[:, 3 + K:] == 5).all()
    assert (ho[:, :1] == 7).all() and (ho[:, 1 + K:] == 7).all()
    qo = torch.zeros((M, K + 9), dtype=torch.uint8, device=DEV)
    so = torch.full((ref.groups(K), M + 2), 9.0, device=DEV)
    q, s, _ = glu.add_rms_norm_fp8(x, w, EPS, residual=r, out=qo.view(ref.E4M3)[:, 5:5 + K], scale_out=so[:, :M].t())
    torch.cuda.synchronize()
    ref.check_e4m3("e4m3", q, s, y, err)
    assert (qo[:, :5] == 0).all() and (qo[:, 5 + K:] == 0).all() and (so[:, M:] == 9).all()


def test_in_place_residual():
    x, r = tensors(40, 1000, torch.bfloat16, 11, 1.0, 2.0)
    w = weight(1000, torch.bfloat16, 11)
    h, y, rstd, err = ref.norm64(x, w, EPS, r)
    gy, gh = glu.add_rms_norm(x, w, EPS, residual=r, residual_out=r)
    torch.cuda.synchronize()
    assert gh is r and torch.equal(r, h)
    ref.check_store("y", gy, y, err)
    dy, dr = tensors(40, 1000, torch.bfloat16, 12, 0.1, 0.1)
    rstd = rstd.float()
    dx, edx, dw, edw = ref.grad64(dy, h, w, rstd, dr)
    gx, gw = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dr, dx=dr)
    torch.cuda.synchronize()
    assert gx is dr
    ref.check_store("dx", gx, dx, edx)
    ref.check_store("dweight", gw, dw, edw)


@pytest.mark.parametrize("K", [256, 40000])
def test_special_values(K):
    """A zero row (finite quotients, y = 0), a NaN, an infinity and the type's lowest value in a row."""
    x = tensors(6, K, torch.bfloat16, 13, 1.0)[0]
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    x[0] = 0
    x[1, 130] = float("nan")
    x[2, 5] = float("inf")
    x[3, 7] = torch.finfo(torch.bfloat16).min
    y, _ = glu.add_rms_norm(x, w, EPS)
    q, s, _ = glu.add_rms_norm_fp8(x, w, EPS)
    torch.cuda.synchronize()
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and (s[0] == ref.TINY).all()
    assert y[1].isnan().all() and q[1].float().isnan().all() and s[1].isnan().all()
    assert y[2, 5].isnan() and (y[2, :5] == 0).all() and (y[2, 6:] == 0).all()  # r = 0: inf * 0 and finite * 0
    assert s[2, 0].isnan() and (s[2, 1] == ref.TINY)
    # the square of the lowest value overflows fp32: r = 0
    assert (y[3] == 0).all() and (q[3].float() == 0).all()
    _, yr, _, err = ref.norm64(x[4:], w, EPS, None)
    ref.check_store("rows beside", y[4:], yr, err[:])
    ref.check_e4m3("rows beside", q[4:], s[4:], yr, err)


def test_empty():
    for t in T.values():
        x = torch.empty(0, 300, dtype=t, device=DEV)
        w = weight(300, t, 1)
        y, h, rstd = glu.add_rms_norm(x, w, EPS, residual=x.clone(), return_rstd=True)
        assert y.shape == (0, 300) and h.shape == (0, 300) and rstd.shape == (0,)
        q, s, _ = glu.add_rms_norm_fp8(x, w, EPS)
        assert q.shape == (0, 300) and s.shape == (0, 3)
        dx, dw = glu.add_rms_norm_backward(x, x, w, rstd, dweight=torch.full((300,), 4.0, dtype=t, device=DEV))
        torch.cuda.synchronize()
        assert dx.shape == (0, 300) and (dw == 0).all()


def test_stream_and_graph():
    """Another stream, and a captured forward and backward replayed on new inputs between eager calls."""
    M, K = 130, 700
    t = torch.bfloat16
    x, r, dy = tensors(M, K, t, 21, 1.0, 3.0, 0.1)
    w = weight(K, t, 21)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, rstd = glu.add_rms_norm(x, w, EPS, residual=r, return_rstd=True, stream=side)
    q, s, _ = glu.add_rms_norm_fp8(x, w, EPS, residual=r, stream=side)
    dx, dw = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dy, stream=side)
    side.synchronize()
    ey, eh, erstd = glu.add_rms_norm(x, w, EPS, residual=r, return_rstd=True)
    eq, es, _ = glu.add_rms_norm_fp8(x, w, EPS, residual=r)
    edx, edw = glu.add_rms_norm_backward(dy, eh, w, erstd, dresidual=dy)
    torch.cuda.synchronize()
    for a, b in ((y, ey), (h, eh), (rstd, erstd), (s, es), (dx, edx), (dw, edw),
                 (q.view(torch.uint8), eq.view(torch.uint8))):
        assert torch.equal(a, b)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, h, rstd = glu.add_rms_norm(x, w, EPS, residual=r, return_rstd=True)
        q, s, _ = glu.add_rms_norm_fp8(x, w, EPS, residual=r)
        dx, dw = glu.add_rms_norm_backward(dy, h, w, rstd, dresidual=dy)
    for seed in (31, 32, 33):
        for dst, src in zip((x, r, dy), tensors(M, K, t, seed, 1.0, 3.0, 0.1)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        ey, eh, erstd = glu.add_rms_norm(x, w, EPS, residual=r, return_rstd=True)
        eq, es, _ = glu.add_rms_norm_fp8(x, w, EPS, residual=r)
        edx, edw = glu.add_rms_norm_backward(dy, eh, w, erstd, dresidual=dy)
        torch.cuda.synchronize()
        for a, b in ((y, ey), (h, eh), (s, es), (dx, edx), (dw, edw), (q.view(torch.uint8), eq.view(torch.uint8))):
            assert torch.equal(a, b)


def test_python_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        glu.add_rms_norm(x, w.float(), EPS)
    with pytest.raises(TypeError):
        glu.add_rms_norm(x.double(), w.double(), EPS)
    with pytest.raises(ValueError):
        glu.add_rms_norm(x, w[:255], EPS)
    with pytest.raises(ValueError):
        glu.add_rms_norm(x, w, EPS, residual=x[:3])
    with pytest.raises(ValueError):
        glu.add_rms_norm(x, w, EPS, residual_out=x)
    with pytest.raises(ValueError):
        glu.add_rms_norm(x.t(), torch.ones(4, dtype=x.dtype, device=DEV), EPS)
    with pytest.raises(ValueError):
        glu.add_rms_norm(x[:1].expand(4, 256), w, EPS)
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(GluError):
            glu.add_rms_norm(x, w, eps)
    with pytest.raises(GluError):
        glu.add_rms_norm(x, w, EPS, out=x)
    with pytest.raises(ValueError):
        glu.add_rms_norm_backward(x, x, w, torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        glu.add_rms_norm_fp8(x, w, EPS, scale_out=torch.zeros(4, 2, device=DEV)[:, ::1].t().contiguous())
    torch.cuda.synchronize()
