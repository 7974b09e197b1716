"""The norm and e4m3 operators by their definitions in 64 bits, with error bounds, for the tests.

u = 2^-24 is the rounding of an fp32 operation; half(t) that of a store to type t.  A bound counts the
fp32 operations behind a value (the longest chain of a sum, in any order the kernels may take) and
the final store.
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
E4M3 = torch.float8_e4m3fn


def half(t):
    return torch.finfo(t).eps / 2


def floor_of(t):
    """Half the smallest subnormal of t: the absolute error of a store near zero."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150, E4M3: 2.0 ** -10}[t]


def groups(n):
    return -(-n // 128)


def per_element(s, rows, cols, block_rows):
    """Scales as one value per element of [rows, cols]."""
    if block_rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def group_amax(y):
    m, k = y.shape
    return torch.nn.functional.pad(y.abs(), (0, -k % 128)).view(m, groups(k), 128).amax(2)


def block_amax(y):
    n, k = y.shape
    return torch.nn.functional.pad(y.abs(), (0, -k % 128, 0, -n % 128)).view(groups(n), 128, groups(k), 128).amax((1, 3))


def scale_of(amax):
    return (amax / 448.0).clamp_min(TINY)


def quantize32(x, block):
    """The conversion in fp32 steps (IEEE divisions): the stored bits are determined."""
    f = x.float()
    s = scale_of(block_amax(f) if block else group_amax(f))
    return (f / per_element(s, *f.shape, block)).to(E4M3), s


def norm64(x, weight, eps, residual):
    """h in x's type, y and rstd in 64 bits, and y's bound before its store."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    d = h.double()
    r = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    y = d * r * weight.double()
    # sum of squares: at most 40 additions in a lane, 6 + 16 across lanes and waves, halved by the root; root, reciprocal,
    # mean, eps and two products
    return h, y, r[:, 0], 40 * U * y.abs()


def grad64(dy, h, weight, rstd, dres):
    d, g, w, r = h.double(), dy.double(), weight.double(), rstd.double()[:, None]
    xh, a = d * r, g * w
    K = d.shape[1]
    dx = r * (a - xh * (a * xh).mean(1, keepdim=True))
    # the mean's sum: up to 62 + 2 steps; then product, difference, product, addition
    edx = U * r * (4 * a.abs() + xh.abs() * 72 * (a * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        edx = edx + U * dx.abs()
    dw = (g * xh).sum(0)
    edw = U * (h.shape[0] + 40) * (g * xh).abs().sum(0)
    return dx, edx, dw, edw


def product64(x, sx, w, sw):
    """The product and a bound of its fp32 evaluation: 128 products inside a K-block (a tree, counted as 16
    with the matrix core's unspecified rounding), one fused addition per K-block, up to 16 + 64 joins, the scales' product."""
    m, k = x.shape
    n = w.shape[0]
    xd = x.double() * per_element(sx.double(), m, k, False)
    wd = w.double() * per_element(sw.double(), n, k, True)
    return xd @ wd.t(), U * (groups(k) + 100) * (xd.abs() @ wd.abs().t())


def matrix_unit(x, sx, w, sw):
    """What the 8-bit matrix path may lose on top: in every 8 neighbouring products each is cut below 2^-12 of
    the largest.  (worst case: all 8 the same way; root mean square: independent, evenly spread)"""
    m, k = x.shape
    n = w.shape[0]
    xa = x.float().abs() * per_element(sx, m, k, False)
    wa = w.float().abs() * per_element(sw, n, k, True)
    total = torch.zeros(m, n, dtype=torch.float64, device=x.device)
    square = torch.zeros_like(total)
    for k0 in range(0, k, 8):
        p = torch.zeros(m, n, device=x.device)
        for i in range(k0, min(k0 + 8, k)):
            p = torch.maximum(p, xa[:, i, None] * wa[None, :, i])
        total += p
        square += p.double() ** 2
    return 8 * 2.0 ** -12 * total, 2.0 ** -12 * (8 / 3 * square).sqrt()


def glu64(g, eg, u, eu):
    """silu(g) u and its bound: |silu'| <= 1.1, the evaluation itself a dozen fp32 steps."""
    s = g * torch.sigmoid(g)
    y = s * u
    return y, 1.1 * eg * u.abs() + s.abs() * eu + 1.1 * eg * eu + 16 * U * y.abs() + TINY * u.abs()


def check_store(name, got, ref, err):
    """got, stored in its type, against ref +- err."""
    t = got.dtype
    d = (got.double() - ref).abs()
    tol = err + half(t) * (ref.abs() + err) + floor_of(t)
    bad = ~(d <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside; worst excess "
                           f"{float((d - tol)[bad].max())} at ref {float(ref[bad].reshape(-1)[0])}")


def check_e4m3(name, q, s, ref, err):
    """(q, s) against ref +- err: the scales, and the values q stands for."""
    m, n = ref.shape
    want = scale_of(group_amax(ref))
    serr = group_amax(err) / 448 + 2 * U * want
    assert ((s.double() - want).abs() <= serr).all(), f"{name}: scales off by {float((s.double() - want).abs().max())}"
    se = per_element(s.double(), m, n, False)
    d = (q.double() * se - ref).abs()
    tol = err + half(E4M3) * (ref.abs() + err) + (floor_of(E4M3) + 448 * 4 * U) * se
    bad = ~(d <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside"


def rms(t):
    return float(t.double().square().mean().sqrt())


def check_unit_rms(name, got, ops):
    """A 16-bit result of the 8-bit matrix path, of one product or of the pair's GLU, in the root mean square over
    its outputs: the path cuts each product below 2^-13 of the largest of its 8 (half of what matrix_unit allows one
    output), independently, which goes through silu(g) u to first order; then the fp32 steps' bound and the store's."""
    y, e = product64(*ops[:4])
    loss = matrix_unit(*ops[:4])[1] / 2
    if len(ops) == 6:
        u, eu = product64(*ops[:2], *ops[4:])
        lu = matrix_unit(*ops[:2], *ops[4:])[1] / 2
        s = torch.sigmoid(y)
        loss = ((s * (1 + y * (1 - s)) * u * loss).square() + (y * s * lu).square()).sqrt()
        y, e = glu64(y, e, u, eu)
    off, most = rms(got.double() - y), rms(loss) + half(got.dtype) * rms(y) + rms(e) + floor_of(got.dtype)
    assert off <= most, f"{name}: off by {off} in the root mean square, at most {most}"
