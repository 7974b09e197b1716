"""The e4m3 conversions and the block-scaled products on the GPU against their definition in 64 bits."""
import pytest
import torch

import fp8_ref as ref
import glu_mlp_gemv_amd as glu
from glu_mlp_gemv_amd import fp8
from glu_mlp_gemv_amd.api import GluError
from glu_mlp_gemv_amd.mlp import Fp8GluMlp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": E4M3}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def same_bits(a, b):
    return torch.equal(a.reshape(-1).contiguous().view(torch.uint8), b.reshape(-1).contiguous().view(torch.uint8))


# ---- conversions -------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 127), (5, 129), (77, 513), (130, 1000), (2050, 640), (16, 16),
                                 (515, 2048)])
def test_quantize(M, K, kind):
    """Both conversions give the bits of the IEEE division by the scale, in values spread over 40 binades."""
    g = gen(M * 7 + K)
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-12, 3, (M, 1), generator=g, device=DEV).float())
    x = (x * torch.exp2(torch.randint(-6, 6, (1, K), generator=g, device=DEV).float())).to(T[kind])
    print(f"[quantize] M={M} K={K} {kind}", flush=True)
    for f, block in ((glu.fp8_quantize, False), (glu.fp8_quantize_weight, True)):
        q, s = f(x)
        torch.cuda.synchronize()
        wq, ws = ref.quantize32(x.cpu(), block)
        assert torch.equal(s.cpu(), ws)
        assert same_bits(q.cpu(), wq)


def test_quantize_every_bf16():
    """Every finite bf16 value in groups of falling magnitude, and each group's largest exact multiple."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).flip(0)
    x = torch.cat([x, -x]).reshape(2, -1)
    q, s = glu.fp8_quantize(x.to(DEV))
    torch.cuda.synchronize()
    wq, ws = ref.quantize32(x, False)
    assert torch.equal(s.cpu(), ws) and same_bits(q.cpu(), wq)


def test_quantize_special_values():
    x = torch.randn(130, 300, generator=gen(4), device=DEV).to(torch.bfloat16)
    x[0, :] = 0
    x[1, 3] = float("nan")
    x[2, 140] = float("inf")
    x[2, 141] = float("-inf")
    x[3, 299] = torch.finfo(torch.bfloat16).min
    x[4, 0] = -0.0
    q, s = glu.fp8_quantize(x)
    torch.cuda.synchronize()
    f = q.float()
    assert (f[0] == 0).all() and (s[0] == ref.TINY).all()
    assert f[1, :128].isnan().all() and s[1, 0].isnan() and not f[1, 128:].isnan().any()
    assert f[2, 140:142].isnan().all() and torch.isinf(s[2, 1])
    rest = torch.cat([f[2, 128:140], f[2, 142:256]])
    assert (rest == 0).all()
    assert f[3, 299] == -448
    w = x.clone()
    w[1, 3] = 0
    w[2, 140:142] = 0
    wq, ws = ref.quantize32(w.cpu(), False)
    q, s = glu.fp8_quantize(w)
    torch.cuda.synchronize()
    assert torch.equal(s.cpu(), ws) and same_bits(q.cpu(), wq)
    q, s = glu.fp8_quantize_weight(x)
    torch.cuda.synchronize()
    assert s[0, 0].isnan() and torch.isinf(s[0, 1]) and not torch.isnan(s[1]).any()
    assert q[:128, :128].float().isnan().all() and q[2, 140].float().isnan() and (q[4:128, 128:256].float() == 0).all()


def test_quantize_strides():
    big = torch.randn(140, 700, generator=gen(5), device=DEV).to(torch.float16)
    x = big[:, 3:3 + 333]
    for f, block in ((glu.fp8_quantize, False), (glu.fp8_quantize_weight, True)):
        store = torch.full((140, 345), 0x11, dtype=torch.uint8, device=DEV)
        q, s = f(x, out=store.view(E4M3)[:, 7:7 + 333])
        torch.cuda.synchronize()
        wq, ws = ref.quantize32(x.cpu(), block)
        assert torch.equal(s.cpu(), ws) and same_bits(q.cpu(), wq)
        assert (store[:, :7] == 0x11).all() and (store[:, 340:] == 0x11).all()


def test_quantize_many_rows():
    """More rows than one grid of threads holds."""
    M = (1 << 28) + 5
    print(f"[many rows] quantize M={M}", flush=True)
    x = torch.randint(0x3f00, 0x4100, (M, 1), generator=gen(6), device=DEV, dtype=torch.int16).view(torch.bfloat16)
    q, s = glu.fp8_quantize(x)
    torch.cuda.synchronize()
    assert (q.view(torch.uint8) == 0x7e).all()  # a group of one: 448 of its scale
    for at in (0, (1 << 28) - 500, M - 500):
        assert torch.equal(s[at:at + 500].cpu(), ref.scale_of(x[at:at + 500].float().cpu()))
    assert ((s * 448 - x.float()).abs() <= 4 * ref.U * x.float()).all()


def test_quantize_empty():
    for shape in ((0, 256), (4, 0)):
        q, s = glu.fp8_quantize(torch.empty(shape, dtype=torch.bfloat16, device=DEV))
        assert q.shape == shape and s.shape == (shape[0], ref.groups(shape[1]))
        q, s = glu.fp8_quantize_weight(torch.empty(shape, dtype=torch.bfloat16, device=DEV))
        assert q.shape == shape and s.shape == (ref.groups(shape[0]), ref.groups(shape[1]))


# ---- products ------------------------------------------------------------------------

def operands(M, N, K, seed, mats=1):
    """Activations with some larger columns and weights, quantised by the definition; every block has its own scale."""
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(K, generator=g, device=DEV) * 0.5)
    x, sx = ref.quantize32(x, False)
    out = [x, sx.t().contiguous().t()]
    for _ in range(mats):
        w = torch.randn(N, K, generator=g, device=DEV) * 0.05
        w *= torch.exp(0.5 * torch.randn(ref.groups(N), generator=g, device=DEV)).repeat_interleave(128)[:N, None]
        out += ref.quantize32(w, True)
    return out


def expected(ops, tile=False):
    """The result and its bound; tile: on the matrix unit's 8-bit path."""
    y, e = ref.product64(*ops[:4])
    if tile:
        e = e + ref.matrix_unit(*ops[:4])[0]
    if len(ops) == 4:
        return y, e
    u, eu = ref.product64(*ops[:2], *ops[4:])
    if tile:
        eu = eu + ref.matrix_unit(*ops[:2], *ops[4:])[0]
    return ref.glu64(y, e, u, eu)


def rms(t):
    return float(t.double().square().mean().sqrt())


def check_rms(got, want, ops):
    """The 8-bit path's loss is without bias: the whole result's is a sum of independent ones."""
    _, err = ref.product64(*ops)
    assert rms(got.double() - want) <= rms(ref.matrix_unit(*ops)[1]) + rms(want) * ref.half(got.dtype) + rms(err)


def run(ops, out_dtype, **kw):
    return (glu.fp8_linear if len(ops) == 4 else glu.fp8_dual_glu)(*ops, out_dtype=out_dtype, **kw)


def check(name, got, want, err):
    if isinstance(got, tuple):
        ref.check_e4m3(name, *got, want, err)
    else:
        ref.check_store(name, got, want, err)


PRODUCTS = [(1, 2560, 9216), (1, 9216, 2560), (1, 1, 16), (2, 300, 128), (3, 129, 144), (4, 640, 1008), (5, 257, 2048),
            (8, 1024, 512), (9, 2000, 1040), (16, 500, 4096), (17, 384, 272), (32, 1100, 640), (33, 127, 400),
            (64, 256, 1024), (65, 640, 4096), (100, 4100, 528), (129, 1000, 144), (203, 513, 2048), (300, 130, 16),
            (1025, 700, 256), (1100, 1300, 912)]


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, mats):
    ops = operands(M, N, K, M + N + K, mats)
    for kind in ("bf16", "fp16", "fp32", "e4m3"):
        plan = fp8.product_plan(mats, M, N, K, T[kind])
        want, err = expected(ops, plan["kernel_name"] == "tile" and kind in ("bf16", "fp16"))
        print(f"[product] mats={mats} M={M} N={N} K={K} {kind} {plan}", flush=True)
        got = run(ops, T[kind])
        torch.cuda.synchronize()
        check(kind, got, want, err)
        if mats == 1 and kind != "e4m3":
            check_rms(got, want, ops)


@pytest.mark.parametrize("M", [3, 4, 5, 16])
def test_few_rows_on_tiles(M):
    """Up to 16 rows keep fp32 sums where tiles with K split serve them."""
    N, K = 5120, 17408
    ops = operands(M, N, K, M)
    want, err = expected(ops)
    for kind in ("bf16", "fp32", "e4m3"):
        plan = fp8.product_plan(1, M, N, K, T[kind])
        print(f"[few rows] M={M} {kind} {plan}", flush=True)
        assert plan["kernel_name"] == "tile" or kind == "e4m3"
        got = run(ops, T[kind])
        torch.cuda.synchronize()
        check(kind, got, want, err)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (6, 130, 257), (19, 64, 15), (70, 200, 1000 - 7), (2, 40, 1)])
def test_any_contraction_length(M, N, K, mats):
    """K that is no multiple of 16."""
    ops = operands(M, N, K, K, mats)
    want, err = expected(ops)
    for kind in ("bf16", "fp32", "e4m3"):
        print(f"[any K] mats={mats} M={M} N={N} K={K} {kind}", flush=True)
        got = run(ops, T[kind])
        torch.cuda.synchronize()
        check(kind, got, want, err)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,N,K,pad", [(17, 1, 33, 0), (300, 700, 1001, 0), (40, 130, 256, 1), (1100, 513, 272, 8)])
def test_copied_layouts(M, N, K, pad, mats):
    """More than 16 rows whose layout is not fast, by its length or by its strides, on the copies and in place."""
    ops = [t if t.dtype is not E4M3 else torch.nn.functional.pad(t.view(torch.uint8), (0, pad), value=0x7f).view(E4M3)[:, :K]
           for t in operands(M, N, K, K, mats)]
    want, err = expected(ops)
    for kind in ("bf16", "fp32", "e4m3"):
        print(f"[copied] mats={mats} M={M} N={N} K={K} pad={pad} {kind}", flush=True)
        got = run(ops, T[kind])
        place = run(ops, T[kind], plan=fp8.ProductPlan(4, 16, 4, 1))
        torch.cuda.synchronize()
        check(kind, got, want, err)
        check(kind + " in place", place, want, err)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,N,K,pad", [(700, 1000, 1001, 0), (515, 2100, 528, 3), (17, 4100, 6001, 0), (2050, 520, 1030, 4)])
def test_copies_that_pay(M, N, K, pad, mats):
    """Layouts that are not fast at sizes whose operands are copied."""
    ops = [t if t.dtype is not E4M3 else torch.nn.functional.pad(t.view(torch.uint8), (0, pad), value=0x7f).view(E4M3)[:, :K]
           for t in operands(M, N, K, K, mats)]
    want, err = expected(ops)
    for kind in ("bf16", "fp32", "e4m3"):
        print(f"[copies] mats={mats} M={M} N={N} K={K} pad={pad} {kind}", flush=True)
        got = run(ops, T[kind])
        torch.cuda.synchronize()
        check(kind, got, want, err)
        again = run(ops, T[kind])
        for a, b in zip(got if isinstance(got, tuple) else (got,), again if isinstance(again, tuple) else (again,)):
            assert same_bits(a, b)


def test_long_contraction():
    """Rows so far apart that 32-bit offsets within a tile would wrap: every row is read at its own place."""
    M, N, K = 17, 128, (1 << 25) + (1 << 20) + 5
    print(f"[long contraction] M={M} N={N} K={K}", flush=True)
    g = gen(1)
    # positive values of two neighbouring codes, in rows that differ by 2^(1/2) or more from the next 15
    x = torch.randint(0x30, 0x32, (M, K), generator=g, device=DEV, dtype=torch.uint8)
    w = torch.randint(0x20, 0x22, (N, K), generator=g, device=DEV, dtype=torch.uint8)
    w += (4 * (torch.arange(N, device=DEV) % 16)).to(torch.uint8)[:, None]
    x, w = x.view(E4M3), w.view(E4M3)
    sx = torch.rand(M, ref.groups(K), generator=g, device=DEV) + 0.5
    sw = torch.rand(1, ref.groups(K), generator=g, device=DEV) + 0.5
    want = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    step = 1 << 20
    for k in range(0, K, step):
        part = slice(k, min(k + step, K))
        n, blocks = part.stop - k, slice(k // 128, ref.groups(part.stop))
        want += (x[:, part].double() * ref.per_element(sx[:, blocks].double(), M, n, False)) @ (
            w[:, part].double() * ref.per_element(sw[:, blocks].double(), N, n, True)).t()
    got = glu.fp8_linear(x, sx, w, sw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    # all terms are positive: one addition per K-block and those of product64
    ref.check_store("fp32", got, want, ref.U * (ref.groups(K) + 100) * want)


def test_many_rows():
    """More rows than one grid of threads holds: of the operands' copies, and of a product's end."""
    M, N, K = 17, (1 << 28) + 5, 17
    print(f"[many rows] M={M} N={N} K={K}", flush=True)
    g = gen(2)
    x = torch.randint(0x20, 0x50, (M, K), generator=g, device=DEV, dtype=torch.uint8).view(E4M3)
    w = torch.randint(0x20, 0x50, (N, K), generator=g, device=DEV, dtype=torch.uint8).view(E4M3)
    sx = torch.rand(M, 1, generator=g, device=DEV) + 0.5
    sw = torch.rand(ref.groups(N), 1, generator=g, device=DEV) + 0.5
    got = glu.fp8_linear(x, sx, w, sw)
    torch.cuda.synchronize()
    for at in (0, 128 * 100000, (1 << 28) - 512, N // 128 * 128 - 512):  # whole blocks of 128 from there on
        part = slice(at, min(at + 700, N))
        want, err = ref.product64(x, sx, w[part], sw[at // 128:ref.groups(part.stop)])
        ref.check_store("bf16", got[:, part], want, err)
    del got, w, sw
    M, empty = (1 << 28) + 5, torch.empty(0, dtype=torch.uint8, device=DEV).view(E4M3)
    y = glu.fp8_linear(empty.view(M, 0), torch.ones(M, 0, device=DEV), empty.view(1, 0), torch.ones(1, 0, device=DEV),
                       out=torch.full((M, 1), 4.0, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert (y == 0).all()


def plans():
    """Every kernel the library can launch, at sizes past and inside its tiles, with and without split sums."""
    out = []
    for tile in range(5):
        for splits in (1, 3):
            out += [(3, tile, 0, splits, M, N, K) for M, N, K in ((5, 130, 784), (130, 640, 1024), (300, 515, 400))]
    for rows in (4, 16):
        for width in (1, 3, 8):
            out += [(2, rows, width, s, min(4, rows), 260, 1296) for s in (1, 2)]
    out += [(2, 16, 4, 1, 16, 300, 2000), (2, 16, 4, 2, 30, 300, 2000),
            (2, 16, 4, 1, 61, 300, 2000), (4, 16, 4, 1, 61, 300, 2000), (4, 16, 3, 2, 20, 100, 512)]
    out += [(2, rows, 4, 1, min(4, rows), 100, 2048) for rows in (4, 16)]
    return out


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("kernel,tile,width,splits,M,N,K", plans())
def test_every_launch_shape(kernel, tile, width, splits, M, N, K, mats):
    ops = operands(M, N, K, M + N + K, mats)
    strict, loose = expected(ops), expected(ops, kernel == 3)
    plan = fp8.ProductPlan(kernel, tile, width, splits)
    for kind in ("bf16", "fp32", "e4m3"):
        print(f"[plan] mats={mats} {kernel} {tile} {width} {splits} M={M} N={N} K={K} {kind}", flush=True)
        got = run(ops, T[kind], plan=plan)
        torch.cuda.synchronize()
        check(kind, got, *(loose if kind == "bf16" else strict))
        again = run(ops, T[kind], plan=plan)
        for a, b in zip(got if isinstance(got, tuple) else (got,), again if isinstance(again, tuple) else (again,)):
            assert same_bits(a, b), "a second call gives the same bits"


def unit_cases():
    """(M, N, K, plan) of 16-bit results on the 8-bit matrix path: as planned, every tile shape whole and split, weights read
    past the caches, columns in two launches."""
    out = [(M, N, K, None) for M, N, K in PRODUCTS if M > 16] + [(37, 12288, 4096, None), (203, 4096, 2048, None)]
    for tile in range(5):
        for splits in (1, 3):
            out += [(M, N, K, (3, tile, 0, splits)) for M, N, K in ((17, 130, 784), (130, 640, 1024), (300, 515, 400))]
    out += [(20, 4105, 16400, (3, tile, 0, 1)) for tile in (2, 3, 4)]
    out += [(150, 515, 784, (3, tile, 0, splits, 0, 0, columns)) for tile, splits, columns in ((0, 1, 256), (1, 2, 128),
                                                                                             (4, 1, 384))]
    return out


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,N,K,plan", unit_cases())
def test_root_mean_square(M, N, K, plan, mats):
    """The worst case that one output is allowed is far from what all of them lose together."""
    ops = operands(M, N, K, M + N + K, mats)
    for kind in ("bf16", "fp16"):
        print(f"[rms] mats={mats} M={M} N={N} K={K} {kind} {plan}", flush=True)
        got = run(ops, T[kind], plan=None if plan is None else fp8.ProductPlan(*plan))
        torch.cuda.synchronize()
        ref.check_unit_rms(kind, got, ops)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M", [40, 150])
def test_root_mean_square_of_strided_rows(M, mats):
    N, K = 300, 656
    ops = operands(M, N, K, M, mats)
    wide = [torch.nn.functional.pad(t.view(torch.uint8), (16, 80), value=0x7f).view(E4M3)[:, 16:16 + K] if t.dtype is E4M3
            else torch.nn.functional.pad(t, (1, 2), value=float("nan"))[:, 1:1 + t.shape[1]] for t in ops]
    for kind in ("bf16", "fp16"):
        store = torch.full((M, N + 11), 3.0, dtype=T[kind], device=DEV)
        got = run(wide, T[kind], out=store[:, 5:5 + N])
        torch.cuda.synchronize()
        ref.check_unit_rms(kind, got, ops)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("tile", [2, 3, 4])
def test_weights_past_the_cache(tile, mats):
    """More than 64 MiB of weights under one row of tiles, which are then read past the caches."""
    M, N, K = 20, 8210 // mats, 8208
    ops = operands(M, N, K, tile, mats)
    strict, loose = expected(ops), expected(ops, True)
    for kind in ("bf16", "fp32", "e4m3"):
        print(f"[past the cache] mats={mats} tile={tile} {kind}", flush=True)
        got = run(ops, T[kind], plan=fp8.ProductPlan(3, tile, 0, 1))
        torch.cuda.synchronize()
        check(kind, got, *(loose if kind == "bf16" else strict))


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("tile,splits,columns", [(0, 1, 256), (1, 2, 128), (4, 1, 384)])
def test_columns_in_two_launches(tile, splits, columns, mats):
    """The first columns by one shape, the others by their own: into strided outputs, with the scales of both."""
    M, N, K = 150, 515, 784
    ops = operands(M, N, K, 5, mats)
    strict, loose = expected(ops), expected(ops, True)
    plan = fp8.ProductPlan(3, tile, 0, splits, 0, 0, columns)
    for kind in ("bf16", "fp32", "e4m3"):
        store = torch.zeros(M, N + 5, dtype=torch.uint8 if kind == "e4m3" else T[kind], device=DEV)
        out = (store.view(E4M3) if kind == "e4m3" else store)[:, 2:2 + N]
        got = run(ops, T[kind], plan=plan, out=out)
        torch.cuda.synchronize()
        check(kind, got, *(loose if kind == "bf16" else strict))
        assert (store[:, :2] == 0).all() and (store[:, 2 + N:] == 0).all()


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M", [3, 40, 150])
@pytest.mark.parametrize("shift", [16, 1])
def test_product_strides(M, mats, shift):
    """Operands and outputs inside wider rows, 16-byte aligned and not; scales at any strides."""
    N, K = 300, 656
    ops = operands(M, N, K, M, mats)
    strict, loose = expected(ops), expected(ops, True)
    wide = []
    for i, t in enumerate(ops):
        if t.dtype is E4M3:
            big = torch.zeros(t.shape[0], K + 96 + (0 if shift == 16 else 5), dtype=torch.uint8, device=DEV)
            big[:] = 0x7f  # NaN around the rows: nothing of it may reach a sum
            v = big.view(E4M3)[:, shift:shift + K]
            v.view(torch.uint8).copy_(t.view(torch.uint8))
        elif i == 1:
            v = torch.full((M, 9), float("nan"), device=DEV)[:, 2:2 + t.shape[1]]
            v.copy_(t)
        else:
            v = torch.full((t.shape[0], t.shape[1] + 3), float("nan"), device=DEV)[:, 1:1 + t.shape[1]]
            v.copy_(t)
        wide.append(v)
    for kind in ("bf16", "fp32"):
        store = torch.full((M, N + 11), 3.0, dtype=T[kind], device=DEV)
        print(f"[strides] mats={mats} M={M} shift={shift} {kind}", flush=True)
        got = run(wide, T[kind], out=store[:, 5:5 + N])
        torch.cuda.synchronize()
        check(kind, got, *(loose if shift == 16 and M > 16 and kind != "fp32" else strict))
        assert (store[:, :5] == 3).all() and (store[:, 5 + N:] == 3).all()
    qs = torch.full((M, N + 9), 0x22, dtype=torch.uint8, device=DEV)
    ss = torch.full((ref.groups(N), M + 1), 2.0, device=DEV)
    got = run(wide, E4M3, out=qs.view(E4M3)[:, 1:1 + N], scale_out=ss[:, :M].t())
    torch.cuda.synchronize()
    check("e4m3", got, *strict)
    assert (qs[:, :1] == 0x22).all() and (qs[:, 1 + N:] == 0x22).all() and (ss[:, M:] == 2).all()


@pytest.mark.parametrize("M", [1, 6, 20, 200])
def test_product_special_values(M):
    """A NaN in x stays in its row, one in a weight in its column; zero operands give +0 and the smallest scale."""
    N, K = 400, 528
    ops = operands(M, N, K, 77, 2)
    ops[0].view(torch.uint8)[M - 1, 500] = 0x7f
    ops[2].view(torch.uint8)[150, 20] = 0xff
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[150] = False
    for t in (torch.float32, torch.bfloat16):
        y = run(ops, t)
        torch.cuda.synchronize()
        assert y[M - 1].isnan().all() and y[:, 150].isnan().all()
        assert not y[:M - 1][:, keep].isnan().any()
    zero = [torch.zeros_like(t.view(torch.uint8)).view(E4M3) if t.dtype is E4M3 else t for t in ops]
    q, s = run(zero, E4M3)
    torch.cuda.synchronize()
    assert (q.view(torch.uint8) == 0).all() and (s == ref.TINY).all()


@pytest.mark.parametrize("M", [1, 4, 9, 40])
@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 6, 7])
def test_scales_past_fp32(M, blocks):
    """Scales of the last K-block that are infinite, or whose product is: its sum goes to its own infinity, also where
    a kernel's steps reach past it."""
    N, K = 20, 128 * blocks - 16
    x = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)  # 1
    w = x[:1].repeat(N, 1)
    w[N // 2:] = 0xb8  # -1
    sx = torch.ones(M, blocks, device=DEV)
    sw = torch.ones(1, blocks, device=DEV)
    want = torch.where(torch.arange(N, device=DEV) < N // 2, 1.0, -1.0).expand(M, N) * float("inf")
    for a, b in ((float("inf"), 1.0), (1.0, float("inf")), (1e30, 1e30)):
        sx[:, -1], sw[:, -1] = a, b
        for plan in (None, fp8.ProductPlan(2, 16, 3, 1), fp8.ProductPlan(3, 4, 0, 1)):
            y = glu.fp8_linear(x.view(E4M3), sx, w.view(E4M3), sw, out_dtype=torch.float32, plan=plan)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        up = x[:1].repeat(N, 1).view(E4M3)
        one = torch.ones_like(sw)
        y = glu.fp8_dual_glu(x.view(E4M3), torch.ones_like(sx), up, one, w.view(E4M3), sw * sx[:1], out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_silu_range():
    """The activation over the whole range of gates: large either way, infinite, zero."""
    gates = torch.tensor([0.0, 1e-6, -1e-6, 1.0, -1.0, 20.0, -20.0, 87.0, -87.0, 88.5, -88.5, 300.0, -300.0, 1e30, -1e30,
                          3e38], dtype=torch.float64, device=DEV)
    N = gates.numel()
    one = torch.zeros(1, 16, dtype=torch.uint8, device=DEV)
    one[0, 0] = 0x38  # 1.0
    for i, g in enumerate(gates.tolist()):
        w = one.view(E4M3)
        unit = torch.ones(1, 1, device=DEV)
        sg = torch.full((1, 1), abs(g), device=DEV)
        gate = one.clone()
        gate[0, 0] |= 0x80 if g < 0 else 0
        y = glu.fp8_dual_glu(w, unit, gate.view(E4M3), sg, w, unit, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want = torch.tensor(torch.tensor(g).float().item(), dtype=torch.float64)
        want = want * torch.sigmoid(want)
        # 16 roundings; below 2^-119 the reciprocal of a huge sum may be flushed
        assert abs(float(y) - float(want)) <= 16 * ref.U * abs(float(want)) + 2.0 ** -118, (g, float(y), float(want))
    assert N == 16


def test_empty():
    for mats in (1, 2):
        for M, N, K in ((0, 256, 128), (4, 0, 128)):
            ops = [torch.zeros(M, K, dtype=torch.uint8, device=DEV).view(E4M3), torch.ones(M, 1, device=DEV)]
            for _ in range(mats):
                ops += [torch.zeros(N, K, dtype=torch.uint8, device=DEV).view(E4M3),
                        torch.ones(ref.groups(N), 1, device=DEV)]
            assert run(ops, torch.bfloat16).shape == (M, N)
            q, s = run(ops, E4M3)
            assert q.shape == (M, N) and s.shape == (M, ref.groups(N))
        ops = [torch.zeros(3, 0, dtype=torch.uint8, device=DEV).view(E4M3), torch.ones(3, 0, device=DEV)]
        for _ in range(mats):
            ops += [torch.zeros(200, 0, dtype=torch.uint8, device=DEV).view(E4M3), torch.ones(2, 0, device=DEV)]
        y = run(ops, torch.float16, out=torch.full((3, 200), 4.0, dtype=torch.float16, device=DEV))
        q, s = run(ops, E4M3)
        torch.cuda.synchronize()
        assert (y == 0).all() and (q.view(torch.uint8) == 0).all() and (s == ref.TINY).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_stream_and_graph(M):
    """Another stream, and captured calls replayed on new inputs between eager ones."""
    ops = operands(M, 640, 1024, 3, 2)
    down = operands(1, 300, 640, 4)[2:]

    def chain(**kw):
        a, s = glu.fp8_dual_glu(*ops, out_dtype=E4M3, **kw)
        return a, s, glu.fp8_linear(a, s, *down, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = chain(stream=side)
    side.synchronize()
    for a, b in zip(got, chain()):
        assert same_bits(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for seed in (11, 12, 13):
        for dst, src in zip(ops, operands(M, 640, 1024, seed, 2)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        want = chain()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert same_bits(a, b)


@pytest.mark.parametrize("M", [1, 5, 90, 600])
def test_mlp_block(M):
    """norm -> gate and up -> down in 8 bits against the 64-bit MLP on the converted weights, and the update
    of the weights in place."""
    K, N = 512, 1152
    g = gen(M)
    w = [torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16) * 0.05 for s in ((N, K), (N, K), (K, N))]
    nw = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    x, r = (torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    mlp = Fp8GluMlp(nw, *w)
    held = [t.data_ptr() for p in (mlp.gate, mlp.up, mlp.down) for t in p]
    mlp.update(*w)
    assert held == [t.data_ptr() for p in (mlp.gate, mlp.up, mlp.down) for t in p]
    y, h = mlp(x, r)
    torch.cuda.synchronize()
    hr, n, _, _ = ref.norm64(x, nw, 1e-6, r)
    assert torch.equal(h, hr)
    # each stage against the 64-bit stage on the stored 8-bit operands before it
    q, s, _ = glu.add_rms_norm_fp8(x, nw, 1e-6, residual=r)
    a, sa = glu.fp8_dual_glu(q, s, *mlp.gate, *mlp.up, out_dtype=E4M3)
    want, err = expected([q, s, *mlp.gate, *mlp.up])
    ref.check_e4m3("glu", a, sa, want, err)
    want, err = expected([a, sa, *mlp.down], M > 16)
    ref.check_store("down", y, want, err)
    # and the whole against the MLP on unrounded activations: two conversions of relative error 2^-4 at most per
    # element, independent, so far below 2^-4 of the root mean square of the result
    wd = [q.double() * ref.per_element(s.double(), *q.shape, True) for q, s in (mlp.gate, mlp.up, mlp.down)]
    gate, up = n @ wd[0].t(), n @ wd[1].t()
    full = (gate * torch.sigmoid(gate) * up) @ wd[2].t()
    assert float((y.double() - full).square().mean().sqrt()) < 2.0 ** -4 * float(full.square().mean().sqrt())


def test_python_refusals():
    x, sx, w, sw = operands(4, 256, 256, 1)
    bad = [
        (ValueError, lambda: glu.fp8_linear(x, sx[:3], w, sw)),
        (ValueError, lambda: glu.fp8_linear(x, sx, w, sw[:1])),
        (ValueError, lambda: glu.fp8_linear(x, sx, w[:, :128], sw)),
        (ValueError, lambda: glu.fp8_dual_glu(x, sx, w, sw, w[:128], sw[:1])),
        (TypeError, lambda: glu.fp8_linear(x.view(torch.uint8), sx, w, sw)),
        (TypeError, lambda: glu.fp8_linear(x, sx.half(), w, sw)),
        (TypeError, lambda: glu.fp8_linear(x, sx, w, sw, out_dtype=torch.float64)),
        (ValueError, lambda: glu.fp8_linear(x, sx, w.t(), sw)),
        (ValueError, lambda: glu.fp8_linear(x.cpu(), sx, w, sw)),
        (ValueError, lambda: glu.fp8_linear(x, sx, w, sw, scale_out=sx)),
        (ValueError, lambda: glu.fp8_linear(x, sx, w, sw, out=torch.empty(4, 255, dtype=torch.bfloat16, device=DEV))),
        (GluError, lambda: glu.fp8_linear(x, sx, w, sw, out_dtype=E4M3, out=x)),
        (GluError, lambda: glu.fp8_linear(x, sx, w, sw, plan=fp8.ProductPlan(3, 9, 0, 1))),
        (GluError, lambda: glu.fp8_linear(x, sx, w, sw, plan=fp8.ProductPlan(2, 16, 17, 1))),
        (GluError, lambda: glu.fp8_linear(x, sx, w, sw, plan=fp8.ProductPlan(3, 1, 0, 3))),
        (TypeError, lambda: glu.fp8_quantize(x)),
        (ValueError, lambda: glu.fp8_quantize(sx[0])),
        (ValueError, lambda: glu.fp8_quantize(sx, out=torch.empty(4, 3, dtype=torch.uint8, device=DEV).view(E4M3))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    torch.cuda.synchronize()
