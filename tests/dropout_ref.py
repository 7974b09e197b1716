"""Dropout's draws by the published generator, in whole numbers, for the tests."""
import torch


def philox4x32_10(counter, key):
    """Four 32-bit words of Python ints or int64 tensors."""
    low = 0xFFFFFFFF
    c, k = list(counter), list(key)
    for _ in range(10):
        # 32 x 32 bits in pieces of 16, so that signed 64-bit tensors hold every step
        h, l = zip(*(product(x, m) for x, m in ((c[0], 0xD2511F53), (c[2], 0xCD9E8D57))))
        c = [h[1] ^ c[1] ^ k[0], l[1], h[0] ^ c[3] ^ k[1], l[0]]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return c


def product(x, m):
    x0, x1, m0, m1 = x & 0xFFFF, x >> 16, m & 0xFFFF, m >> 16
    low = x0 * m0
    mid = x1 * m0 + (low >> 16)
    mid2 = x0 * m1 + (mid & 0xFFFF)
    return x1 * m1 + (mid >> 16) + (mid2 >> 16), (mid2 & 0xFFFF) << 16 | low & 0xFFFF


def draws(M, K, seed, offset, device="cpu"):
    """[M, K] draws of 16 bits."""
    low = 0xFFFFFFFF
    seed, offset = seed & (1 << 64) - 1, offset & (1 << 64) - 1
    m = torch.arange(M, device=device)[:, None].expand(M, -(-K // 8))
    b = torch.arange(-(-K // 8), device=device)[None].expand_as(m)
    o = [torch.full_like(m, w) for w in (offset & low, offset >> 32)]
    words = philox4x32_10((b, m, *o), (seed & low, seed >> 32))
    return torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 2).flatten(1)[:, :K]


def dropout32(x, p, seed, offset, residual=None):
    """The definition in fp32 steps: the stored bits are determined."""
    drop = round(65536 * p)
    kept = draws(*x.shape, seed, offset, x.device) >= drop
    scale = torch.tensor(65536.0 / (65536 - drop) if drop < 65536 else 0.0, dtype=torch.float32, device=x.device)
    y = torch.where(kept, x.float() * scale, 0.0)
    return (y if residual is None else residual.float() + y).to(x.dtype)
