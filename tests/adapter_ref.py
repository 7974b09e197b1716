"""Low-rank adapters by their definition in 64 bits, with error bounds, for the tests.

u = 2^-24 is the rounding of an fp32 operation (the matrix unit's sums are counted at twice that: its inner rounding is
not specified).
"""
import torch

from fp8_ref import U

# what two numbers of a type leave of one in fp32: each rounds by half a step of the type, relative to what it rounds
LEFT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}
# fp16: numbers are brought to 2^15 at most by a power of two of their row, and a second one below 2^-14 is rounded to
# multiples of 2^-24: relative to the row's largest, 2^-25 / 2^14
SUBNORMAL = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -39}


def adapters_of(index, L):
    return [(l, (index == l).nonzero()[:, 0]) for l in range(L)]


def left_of(z, t, dim):
    """Bound of what is lost when z goes into a product as two numbers of t (SUBNORMAL by the largest along dim)."""
    if not z.numel():
        return z.abs()
    return LEFT[t] * z.abs() + SUBNORMAL[t] * z.abs().amax(dim, keepdim=True)


def low64(x, a, index):
    """x a^T per row and its bound; zeros without an adapter."""
    x, n = x.double(), x.shape[1] / 16 + 40  # chain of a sum: 32 numbers an instruction, waves, parts
    t = x.new_zeros(x.shape[0], a.shape[1])
    err = t.clone()
    for l, rows in adapters_of(index, a.shape[0]):
        w = a[l].double()
        t[rows] = x[rows] @ w.t()
        err[rows] = 2 * U * n * (x[rows].abs() @ w.abs().t())
    return t, err


def add64(y, x, a, b, index, scale):
    """out before its rounding, and its bound."""
    t, err = low64(x, a, index)
    out = y.double().clone()
    bound = U * out.abs()
    R = a.shape[1]
    for l, rows in adapters_of(index, a.shape[0]):
        w, s = b[l].double(), 1.0 if scale is None else float(scale[l])
        delta = s * (t[rows] @ w.t())
        near = err[rows] + left_of(t[rows], y.dtype, 1) + 2 * U * (R / 8 + 8) * t[rows].abs()
        out[rows] += delta
        bound[rows] += abs(s) * (near @ w.abs().t()) * (1 + 1e-3) + 2 * U * delta.abs() + U * out[rows].abs()
    return out, bound


def glu64(gate, up, eg, eu):
    """silu(g) u and its bound from those of g and u: |silu'| <= 1.1, 8 fp32 roundings in the activation, and exp(-g) taken as
    2^t, where t = -g log2(e) is off by 1.6 units of its own: 1.6 |g| units of the exponential."""
    s = gate * torch.sigmoid(gate)
    out = s * up
    return out, 1.1 * eg * up.abs() + s.abs() * eu + 1.1 * eg * eu + (8 + 2 * gate.abs()) * U * out.abs()


def backward64(dout, x, a, b, index, low, scale):
    """((dx, bound), (da, bound), (db, bound)) before their rounding."""
    t = dout.dtype
    d, n = dout.double(), dout.shape[1] / 16 + 40
    dx = torch.zeros_like(x, dtype=torch.double)
    edx = dx.clone()
    da, db = torch.zeros_like(a, dtype=torch.double), torch.zeros_like(b, dtype=torch.double)
    eda, edb = da.clone(), db.clone()
    for l, rows in adapters_of(index, a.shape[0]):
        if not rows.numel():
            continue
        s = 1.0 if scale is None else float(scale[l])
        wa, wb, v, g, z = a[l].double(), b[l].double(), x[rows].double(), d[rows], low[rows].double()
        through = g @ wb
        err = 2 * U * n * (g.abs() @ wb.abs())
        R, m = a.shape[1], rows.numel() / 16 + 40
        dx[rows] = s * (through @ wa)
        edx[rows] = abs(s) * ((err + left_of(through, t, 1) + 2 * U * (R / 8 + 8) * through.abs()) @ wa.abs()) * 1.001 \
            + 2 * U * dx[rows].abs()
        da[l] = s * (through.t() @ v)
        eda[l] = abs(s) * ((err + left_of(through, t, 0) + 2 * U * m * through.abs()).t() @ v.abs()) * 1.001 \
            + 2 * U * da[l].abs()
        db[l] = s * (g.t() @ z)
        edb[l] = abs(s) * (g.abs().t() @ (left_of(z, t, 0) + 2 * U * m * z.abs())) * 1.001 + 2 * U * db[l].abs()
    return (dx, edx), (da, eda), (db, edb)

