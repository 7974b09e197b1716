"""moe_glu at the ends of its number formats: infinite scales of e4m3 blocks, and what is kept of the activation."""
import math

import pytest
import torch

import glu_mlp_gemv_amd as glu
import moe_ref
from adapter_ref import LEFT
from fp8_ref import U, check_store

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


# rows of an expert: one to some past what the second product takes at a time, in either of its forms; odd widths
ROWS = [(1, 200, 130), (2, 64, 300), (3, 70, 257), (4, 128, 1030), (5, 96, 64), (8, 130, 520), (9, 64, 75), (16, 40, 260),
        (17, 72, 136), (32, 33, 513), (33, 64, 130), (50, 48, 96), (64, 64, 200), (65, 40, 72)]


def wide64(x, logits, gate, up, down, top, scales=(None, None, None), floor=None):
    """out before its rounding, and its bound where the activation goes into the second product as two numbers.  floor: what
    fp16 numbers may lose of the largest of 32 columns, whose 16 they share a factor with; else half of 2^-24."""
    t, K, N = x.dtype, x.shape[1], gate.shape[1]
    take = moe_ref.chosen(logits, top)
    p = moe_ref.weights(logits, take, True)
    x = x.double()
    out = torch.zeros_like(x)
    err = out.clone()
    nk, nn = K / 16 + 40, N / 16 + 40  # chains of fp32 sums, as in moe_ref
    for e in take.any(0).nonzero()[:, 0].tolist():
        rows = take[:, e].nonzero()[:, 0]
        wg, wu, wd = (moe_ref.expert(w, s, e) for w, s in zip((gate, up, down), scales))
        g, u = x[rows] @ wg.t(), x[rows] @ wu.t()
        eg, eu = (2 * U * nk * (x[rows].abs() @ w.abs().t()) for w in (wg, wu))
        a = g * torch.sigmoid(g) * u
        ea = 1.1 * eg * (u.abs() + eu) + (g * torch.sigmoid(g)).abs() * eu + 8 * U * a.abs()
        # two roundings of at most half a step each, of bf16 numbers behind e4m3 weights, and of an fp16 number below 2^-14
        # half of 2^-24
        ea = ea + LEFT[t if scales[0] is None else torch.bfloat16] * (a.abs() + ea)
        if floor is not None:
            most = torch.nn.functional.pad(a.abs(), (0, -N % 32)).unflatten(1, (-1, 32)).amax(2).repeat_interleave(32, 1)[:, :N]
            ea = ea + floor * most
        elif t is torch.float16:
            ea = ea + 2.0 ** -25
        pe = p[rows, e, None]
        out[rows] += pe * (a @ wd.t())
        err[rows] += pe * (ea @ wd.abs().t() + 2 * U * nn * (a.abs() @ wd.abs().t()) + 100 * U * (a @ wd.t()).abs())
    return out, err + 40 * U * out.abs() + (top + 8) * U * err


def e4m3_of(w):
    q, s = zip(*(glu.fp8_quantize_weight(m) for m in w))
    return torch.stack([m.view(torch.uint8) for m in q]).view(E4M3), torch.stack(s)


def layer(M, K, N, E, t, e4m3, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, logits = rand(M, K).to(t), rand(M, E)
    w = [(rand(E, a, b) * b ** -0.5).to(t) for a, b in ((N, K), (N, K), (K, N))]
    if not e4m3:
        return x, logits, w, (None, None, None)
    w, s = zip(*(e4m3_of(m) for m in w))
    return x, logits, w, s


def run(x, logits, w, s, top):
    out = glu.moe_glu(x, logits, *w, top, gate_scale=s[0], up_scale=s[1], down_scale=s[2])
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("E,top", [(1, 1), (3, 2)])
@pytest.mark.parametrize("M,K,N", ROWS)
def test_activation_keeps_its_bits(M, K, N, E, top, e4m3, kind):
    """The activation is not rounded to x's type between the products."""
    print(f"[moe bits] {M=} {K=} {N=} {E=} {e4m3=} {kind}", flush=True)
    x, logits, w, s = layer(M, K, N, E, T[kind], e4m3, M + N)
    check_store("out", run(x, logits, w, s, top), *wide64(x, logits, *w, top, s))


# activations past fp16's range on either side, of very different sizes in one row, and results that fp16 holds
SIZES = {"large": (2.0 ** 10, 2.0 ** -13), "huge": (2.0 ** 14, 2.0 ** -21), "small": (2.0 ** -11, 2.0 ** 11)}


@pytest.mark.parametrize("size", [*SIZES, "mixed"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 9, 17, 33, 64])
def test_activations_past_the_range_of_fp16(M, e4m3, size):
    print(f"[moe range] {M=} {e4m3=} {size}", flush=True)
    K, N, E, top, t = 72, 213, 3, 2, torch.float16
    x, logits, w, s = layer(M, K, N, E, t, False, M)
    x.clamp_(-3, 3)
    up = down = None
    if size == "mixed":  # by runs of 32 columns, whose groups of 16 share a factor at most with each other
        up = 2.0 ** (9.0 - 5 * (torch.arange(N, device=DEV) // 32 % 4))  # down's stay below 2^15, fp16 numbers
        down = up ** -2 * 8
    else:
        up, down = (torch.full((N,), v, device=DEV) for v in SIZES[size])
    w = [(m.float() * f).to(t) for m, f in zip(w, (up[:, None], up[:, None], down))]
    if e4m3:
        w, s = zip(*(e4m3_of(m) for m in w))
    out = run(x, logits, w, s, top)
    want, err = wide64(x, logits, *w, top, s, floor=2.0 ** -39)
    assert want.abs().max() < 6e4
    check_store("out", out, want, err)


@pytest.mark.parametrize("M", [2, 7, 40])
def test_infinite_activations_in_fp16(M):
    """One infinite number of an activation, large finite ones beside it: results are that one's infinity."""
    K, N, E = 64, 70, 2
    x, logits, w, s = layer(M, K, N, E, torch.float16, False, M)
    x.abs_().clamp_(0.5, 3)
    w[0].abs_()
    w[1].mul_(2 ** 12)
    w[1][:, 37] = math.inf
    w[2][:, :, 37] = torch.where(torch.arange(K, device=DEV) % 2 == 0, 1.0, -1.0)
    want = (math.inf * w[2][0, :, 37].float()).expand(M, K)
    assert torch.equal(run(x, logits, w, s, 2).float(), want)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("M", [1, 2, 4, 7, 40])
def test_infinite_weights_of_the_second_product(M, e4m3, kind):
    """An infinite column of down, or scale of its last block: results are infinite by the activation's sign, whichever sign the
    second of its two numbers has."""
    K, N = 96, 200
    x, logits, w, s = layer(M, K, N, 1, T[kind], False, M)
    x.abs_()
    w[0].abs_()
    w[1].abs_()
    sign = torch.where(torch.arange(K, device=DEV) % 2 == 0, 1.0, -1.0)
    w[2].abs_().mul_(sign[None, :, None].to(w[2].dtype))
    if e4m3:
        w, s = zip(*(e4m3_of(m) for m in w))
        s[2][..., -1] = math.inf
    else:
        w[2][..., 71] = (math.inf * sign).to(w[2].dtype)
    assert torch.equal(run(x, logits, w, s, 1).float(), (math.inf * sign).expand(M, K))
