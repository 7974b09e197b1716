"""moe_glu on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import glu_mlp_gemv_amd as glu
import moe_ref as ref
from fp8_ref import check_store
from glu_mlp_gemv_amd import mlp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "fp16": torch.float16}

# M, K, N, E, top: one row; one expert; all experts; odd widths; more than 16 and than 32 rows of an expert; a second set of
# 64 rows, and one row of it; as many experts as a wave has lanes and more; many parts of few experts; most experts
SHAPES = [(1, 64, 64, 1, 1), (1, 2560, 1024, 64, 8), (2, 128, 256, 8, 8), (3, 100, 75, 5, 2), (5, 7, 9, 3, 2),
          (17, 130, 257, 4, 2), (40, 256, 192, 3, 3), (64, 512, 320, 16, 4), (65, 96, 130, 2, 1), (150, 200, 136, 9, 3),
          (37, 256, 128, 128, 8), (4, 1032, 1000, 200, 6), (1, 4100, 520, 7, 2), (9, 64, 32, 1024, 32), (64, 64, 48, 65, 1)]


def layer(M, K, N, E, top, t, seed, logits_type=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return (rand(M, K).to(t), rand(M, E).to(logits_type), (rand(E, N, K) * K ** -0.5).to(t),
            (rand(E, N, K) * K ** -0.5).to(t), (rand(E, K, N) * N ** -0.5).to(t))


def to_e4m3(w):
    """Each expert by the framework's own conversion."""
    q, s = zip(*(glu.fp8_quantize_weight(m) for m in w))
    return torch.stack([m.view(torch.uint8) for m in q]).view(torch.float8_e4m3fn), torch.stack(s)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("logits_type", ["fp32", "same"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("M,K,N,E,top", SHAPES)
def test_layer(M, K, N, E, top, normalize, logits_type, kind):
    print(f"[moe] {M=} {K=} {N=} {E=} {top=} {normalize=} {logits_type} {kind}", flush=True)
    t = T[kind]
    ops = layer(M, K, N, E, top, t, M + K, torch.float32 if logits_type == "fp32" else t)
    want, err = ref.moe64(*ops, top, normalize)
    out = glu.moe_glu(*ops, top, normalize=normalize)
    torch.cuda.synchronize()
    check_store("out", out, want, err)
    assert torch.equal(out, glu.moe_glu(*ops, top, normalize=normalize)), "a second call gives the same bits"


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,E,top", SHAPES)
def test_layer_e4m3(M, K, N, E, top, kind):
    print(f"[moe e4m3] {M=} {K=} {N=} {E=} {top=} {kind}", flush=True)
    x, logits, *w = layer(M, K, N, E, top, T[kind], M + N)
    (gate, gs), (up, us), (down, ds) = (to_e4m3(m) for m in w)
    want, err = ref.moe64(x, logits, gate, up, down, top, True, (gs, us, ds))
    out = glu.moe_glu(x, logits, gate, up, down, top, gate_scale=gs, up_scale=us, down_scale=ds)
    torch.cuda.synchronize()
    check_store("out", out, want, err)


@pytest.mark.parametrize("M", [3, 70])
def test_masked_tied_and_special_logits(M):
    K, N, E, top = 64, 96, 12, 4
    x, logits, gate, up, down = layer(M, K, N, E, top, torch.bfloat16, 7)
    logits = (logits * 2).round() / 2  # ties: the lowest expert first
    logits[0] = -math.inf
    logits[1, 2:] = -math.inf
    logits[2] = 0.0
    logits[2, 5] = -0.0
    if M > 40:
        logits[40] = 3.4e38
        logits[41, 3] = math.nan
        logits[42, :6] = torch.finfo(torch.float32).min
        logits[66] = -math.inf
        logits[43, 1] = math.inf
    take = ref.chosen(logits, top)
    assert take[0].sum() == 0 and take[1].sum() == 2 and take[2].nonzero()[:, 0].tolist() == [0, 1, 2, 3]
    want, err = ref.moe64(x, logits, gate, up, down, top)
    out = glu.moe_glu(x, logits, gate, up, down, top)
    torch.cuda.synchronize()
    fine = torch.ones(M, dtype=torch.bool, device=DEV)
    fine[41:44:2] = M <= 40
    check_store("out", out[fine], want[fine], err[fine])
    assert not out[0].any()
    if M > 40:
        assert out[41].isnan().all() and out[43].isnan().all() and not out[66].any()
    many = glu.moe_glu(x, logits, gate, up, down, top, normalize=False)
    want, err = ref.moe64(x, logits, gate, up, down, top, False)
    check_store("out", many[fine], want[fine], err[fine])


def test_other_experts_do_not_show():
    """NaN and infinity in experts that no row takes, and in an expert of one row."""
    M, K, N, E, top = 20, 128, 100, 10, 2
    x, logits, gate, up, down = layer(M, K, N, E, top, torch.float16, 3)
    logits[:, 4] = -math.inf
    logits[:, 6] = -50.0
    logits[3, 6] = 50.0
    clean = glu.moe_glu(x, logits, gate, up, down, top)
    gate[4], up[4], down[4] = math.nan, math.inf, math.nan
    down[6] = math.inf
    x[7] = math.nan
    out = glu.moe_glu(x, logits, gate, up, down, top)
    torch.cuda.synchronize()
    fine = [m for m in range(M) if m not in (3, 7)]
    assert torch.equal(out[fine], clean[fine]) and out[7].isnan().all() and not out[3].isfinite().all()


def test_views():
    """Rows and experts apart with NaN between, gate and up as halves of one tensor, an unaligned output."""
    M, K, N, E, top = 6, 100, 70, 5, 2
    x, logits, gate, up, down = layer(M, K, N, E, top, torch.bfloat16, 1)
    want = glu.moe_glu(x, logits, gate, up, down, top)
    both = torch.full((E, 2 * N + 1, K + 3), math.nan, dtype=x.dtype, device=DEV)
    both[:, :N, :K], both[:, N:2 * N, :K] = gate, up
    vd = torch.full((E + 2, K, N + 5), math.nan, dtype=x.dtype, device=DEV)[1:E + 1, :, :N]
    vd.copy_(down)
    vx = torch.full((M, K + 1), math.nan, dtype=x.dtype, device=DEV)[:, 1:]
    vx.copy_(x)
    vl = torch.full((M, E + 4), math.nan, device=DEV)[:, 2:E + 2]
    vl.copy_(logits)
    into = torch.full((M, K + 7), 3.0, dtype=x.dtype, device=DEV)
    out = glu.moe_glu(vx, vl, both[:, :N, :K], both[:, N:2 * N, :K], vd, top, out=into[:, 3:K + 3])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (into[:, :3] == 3).all() and (into[:, K + 3:] == 3).all()


def test_far_experts():
    """Experts 2^31 elements apart and more."""
    M, K, N, E, top = 5, 64, 48, 3, 2
    x, logits, gate, up, down = layer(M, K, N, E, top, torch.bfloat16, 2)
    far = torch.empty((1 << 32) + (1 << 20), dtype=torch.bfloat16, device=DEV)
    views = []
    for i, w in enumerate((gate, up, down)):
        v = far[i * 100000:].as_strided(w.shape, ((1 << 31) + 8, w.shape[2], 1))
        v.copy_(w)
        views.append(v)
    out = glu.moe_glu(x, logits, *views, top)
    torch.cuda.synchronize()
    assert torch.equal(out, glu.moe_glu(x, logits, gate, up, down, top))


@pytest.mark.parametrize("M,K,N", [(0, 64, 64), (3, 64, 0), (3, 0, 64)])
def test_empty(M, K, N):
    x, logits, gate, up, down = layer(M, K or 1, N or 1, 4, 2, torch.bfloat16, 1)
    out = glu.moe_glu(x[:, :K], logits, gate[:, :N, :K], up[:, :N, :K], down[:, :K, :N], 2)
    torch.cuda.synchronize()
    assert out.shape == (M, K) and not out.any()


def test_graph_replays():
    M, K, N, E, top = 5, 256, 128, 16, 3
    ops = layer(M, K, N, E, top, torch.bfloat16, 1)
    glu.moe_glu(*ops, top)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = glu.moe_glu(*ops, top)
    for seed in range(4):
        new = layer(M, K, N, E, top, torch.bfloat16, 20 + seed)
        for old, v in zip(ops, new):
            old.copy_(v)
        graph.replay()
        eager = glu.moe_glu(*new, top)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_streams():
    ops = layer(9, 256, 128, 16, 3, torch.bfloat16, 1)
    want = glu.moe_glu(*ops, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = glu.moe_glu(*ops, 3, stream=side)
    with torch.cuda.stream(side):
        again = glu.moe_glu(*ops, 3)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def test_argument_refusals():
    x, logits, gate, up, down = layer(3, 64, 32, 4, 2, torch.bfloat16, 1)
    ok = dict(x=x, logits=logits, gate=gate, up=up, down=down, top=2)
    s = torch.ones(4, 1, 1, device=DEV)
    for bad, kw in [(TypeError, dict(x=x.float())), (TypeError, dict(logits=logits.half())), (TypeError, dict(up=up.half())),
                    (TypeError, dict(gate=to_e4m3(gate)[0])), (ValueError, dict(top=0)), (ValueError, dict(top=5)),
                    (ValueError, dict(logits=logits[:2])), (ValueError, dict(logits=logits[:, :3])), (ValueError, dict(down=gate)),
                    (ValueError, dict(up=up[:, :31])), (ValueError, dict(gate=gate[:1].expand(4, 32, 64))),
                    (ValueError, dict(gate_scale=s)), (ValueError, dict(x=x.cpu())), (ValueError, dict(down=down.transpose(1, 2).contiguous().transpose(1, 2)))]:
        with pytest.raises(bad):
            glu.moe_glu(**{**ok, **kw})
    with pytest.raises(Exception, match="ALIAS"):
        glu.moe_glu(**ok, out=x)
    with pytest.raises(RuntimeError, match="no gradient"):
        glu.moe_glu(**{**ok, "x": x.clone().requires_grad_()})


def test_layer_of_a_decoder():
    """Norm, router and experts together, as mlp.ExpertGluMlp runs them."""
    M, K, N, E, top = 6, 256, 128, 8, 2
    x, _, gate, up, down = layer(M, K, N, E, top, torch.bfloat16, 4)
    g = torch.Generator(device=DEV).manual_seed(8)
    router = (torch.randn(E, K, generator=g, device=DEV) * K ** -0.5).bfloat16()
    norm = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    res = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    y, h = mlp.ExpertGluMlp(norm, router, gate, up, down, top)(x, res)
    n, h2 = glu.add_rms_norm(x, norm, 1e-6, residual=res)
    (logits,) = glu.api.grouped_gemv(n, [router])
    want, err = ref.moe64(n, logits, gate, up, down, top)
    torch.cuda.synchronize()
    assert torch.equal(h, h2)
    check_store("y", y, want, err)
    (gq, gs), (uq, us), (dq, ds) = (to_e4m3(m) for m in (gate, up, down))
    y8, _ = mlp.ExpertGluMlp(norm, router, gq, uq, dq, top, scales=(gs, us, ds))(x, res)
    want, err = ref.moe64(n, logits, gq, uq, dq, top, True, (gs, us, ds))
    check_store("y8", y8, want, err)
