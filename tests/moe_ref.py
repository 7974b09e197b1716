"""The expert layer by its definition in 64 bits, with an error bound, for the tests."""
import math

import torch

from fp8_ref import U, floor_of, half


def chosen(logits, top):
    """[M, E] which experts a row takes: fewer than ``top`` others come before them, and they are not masked."""
    l = logits.double()
    col = torch.arange(l.shape[1], device=l.device)
    key = torch.where(l.isnan(), math.inf, l)
    nan = l.isnan()
    gt = (key[:, None, :] > key[:, :, None]) | (nan[:, None, :] & ~nan[:, :, None])
    same = (key[:, None, :] == key[:, :, None]) & (nan[:, None, :] == nan[:, :, None])
    before = gt | (same & (col[None, :] < col[:, None]))
    return (before.sum(2) < top) & (l != -math.inf)


def weights(logits, take, normalize):
    l = logits.double()
    most = l.masked_fill(~take, -math.inf).amax(1, keepdim=True)
    e = torch.exp(l - torch.where(most == -math.inf, 0.0, most))
    return torch.where(take, e, 0.0) / torch.where(take, e, 0.0).sum(1, keepdim=True).clamp_min(1e-300) if normalize \
        else torch.where(take, e / e.sum(1, keepdim=True), 0.0)


def expert(w, scale, e):
    """One expert's matrix in 64 bits."""
    m = w[e].double()
    if scale is not None:
        rows, cols = m.shape
        m = m * scale[e].double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return m


def moe64(x, logits, gate, up, down, top, normalize=True, scales=(None, None, None)):
    """out before its rounding, and its bound."""
    t, (M, K), N = x.dtype, x.shape, gate.shape[1]
    take = chosen(logits, top)
    p = weights(logits, take, normalize)
    x = x.double()
    out = torch.zeros_like(x)
    err = out.clone()
    # chains of fp32 sums on the matrix unit (counted at twice their rounding): 32 numbers an instruction, a scale per 128,
    # 8 waves
    nk, nn = K / 16 + 40, N / 16 + 40
    for e in take.any(0).nonzero()[:, 0].tolist():
        rows = take[:, e].nonzero()[:, 0]
        wg, wu, wd = (expert(w, s, e) for w, s in zip((gate, up, down), scales))
        g, u = x[rows] @ wg.t(), x[rows] @ wu.t()
        eg, eu = (2 * U * nk * (x[rows].abs() @ w.abs().t()) for w in (wg, wu))
        a = g * torch.sigmoid(g) * u
        # |silu'| <= 1.1; 8 roundings in the activation; one to t
        ea = 1.1 * eg * (u.abs() + eu) + (g * torch.sigmoid(g)).abs() * eu + 8 * U * a.abs()
        ea = ea + half(t) * (a.abs() + ea) + floor_of(t)
        y = a @ wd.t()
        ey = ea @ wd.abs().t() + 2 * U * nn * (a.abs() @ wd.abs().t())
        pe = p[rows, e, None]
        out[rows] += pe * y
        # the weight: exp of a difference rounded by U (|l - most| <= 64 here), a sum of up to 1024, a division
        err[rows] += pe * ey + (80 + 20) * U * pe * y.abs()
    return out, err + 40 * U * out.abs() + (top + 8) * U * err
