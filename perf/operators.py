"""Measured cases of the RMS-norm and 8-bit (e4m3) operators around the GLU projection.

Each case is one call that a decoder layer makes: residual addition + RMS norm
(to e4m3 with a scale per 128 columns, or in the input's type), its backward,
quantisation of activations and of weights, the dual-weight GLU projection and
the plain projection on block-scaled e4m3 operands.  ``run`` computes a pass in
elementary torch operations in 32 bits, or with ``own`` through the framework's
entry points; ``exact`` is the definition in 64 bits.

Scales: an activation row has one fp32 scale per 128 columns (tensor [M, G],
stored group by group), a weight one per block of 128 x 128 ([N / 128, K / 128]).
A stored value q stands for q * scale.
"""
import math

import torch

own = False

GROUP = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale: an all-zero group keeps a finite quotient
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one token's residual stream on its way into a 2560-wide layer's MLP: latency alone
        {"name": "norm_token", "op": "norm", "M": 1, "K": 2560, "type": "bf16", "residual": True, "out": "fp8"},
        # a prefill of 8192 tokens at width 5120
        {"name": "norm_prefill", "op": "norm", "M": 8192, "K": 5120, "type": "bf16", "residual": True, "out": "fp8"},
        # a short ragged training batch
        {"name": "norm_grad_short", "op": "norm_grad", "M": 203, "K": 2560, "type": "bf16", "residual": True},
        # a training micro-batch of 16384 tokens at width 4096
        {"name": "norm_grad_long", "op": "norm_grad", "M": 16384, "K": 4096, "type": "bf16", "residual": True},
        # what attention gives back for 77 tokens, before an 8-bit output projection
        {"name": "quantize_rows", "op": "quantize", "M": 77, "K": 4096, "type": "bf16", "block": False},
        # a gate weight after an optimiser step, back to 8 bits for the rollout
        {"name": "quantize_weight", "op": "quantize", "M": 17408, "K": 5120, "type": "bf16", "block": True},
        # one token through gate and up, the product leaving in 8 bits
        {"name": "glu_token", "op": "glu", "M": 1, "K": 2560, "N": 9216, "out": "fp8"},
        # a decode batch with an odd number of sequences
        {"name": "glu_batch", "op": "glu", "M": 37, "K": 4096, "N": 12288, "out": "bf16"},
        # a prefill
        {"name": "glu_prefill", "op": "glu", "M": 4096, "K": 5120, "N": 17408, "out": "fp8"},
        # one token through the down projection
        {"name": "linear_token", "op": "linear", "M": 1, "K": 9216, "N": 2560, "out": "bf16"},
        # a short prompt through the down projection, rows that fill no tile
        {"name": "linear_prompt", "op": "linear", "M": 203, "K": 12288, "N": 4096, "out": "bf16"},
        # a prefill through the down projection
        {"name": "linear_prefill", "op": "linear", "M": 4096, "K": 17408, "N": 5120, "out": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "glu", "linear"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        case = {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 128, 8192), "type": kind, "residual": rng.random() < 0.7}
        if rng.random() < 0.6:
            case["K"] = max(128, case["K"] // 64 * 64)  # most widths are whole multiples; the others stay odd
        if op == "norm":
            case["out"] = rng.choice(["fp8", "fp8", "same"])
        return case
    if op == "quantize":
        block = rng.random() < 0.5
        return {"op": op, "M": _log(rng, 1, 16384), "K": 16 * _log(rng, 16, 320), "type": kind, "block": block}
    # the contraction is padded to 16 bytes of e4m3, as every 8-bit weight file has it; rows and outputs are not
    case = {"op": op, "M": _log(rng, 1, 4096), "K": 16 * _log(rng, 16, 640), "N": _log(rng, 256, 12288)}
    if rng.random() < 0.5:
        case["K"] = max(GROUP, case["K"] // GROUP * GROUP)
    if rng.random() < 0.6:
        case["N"] = max(GROUP, case["N"] // GROUP * GROUP)
    case["out"] = rng.choice(["bf16", "bf16", "fp16"]) if op == "linear" else rng.choice(["fp8", "fp8", "bf16"])
    return case


def _groups(n):
    return -(-n // GROUP)


def _spread(s, dim, n):
    """One value per 128 along ``dim`` as one per element, the first n."""
    return s.repeat_interleave(GROUP, dim).narrow(dim, 0, n)


def _scale_of(a):
    return (a / E4M3_MAX).clamp_min(TINY)


def _pad(x, rows):
    """x with its columns (and with ``rows`` its rows) filled up with zeros to whole groups."""
    m, k = x.shape
    return torch.nn.functional.pad(x, (0, -k % GROUP, 0, -m % GROUP if rows else 0))


def _row_scales(y):
    m, k = y.shape
    return _scale_of(_pad(y, False).view(m, _groups(k), GROUP).abs().amax(2))


def _block_scales(y):
    m, k = y.shape
    return _scale_of(_pad(y, True).view(_groups(m), GROUP, _groups(k), GROUP).abs().amax((1, 3)))


def _activations(g, M, K):
    """e4m3 rows and their scales, as the framework's norm leaves them: unit-variance values, some columns larger."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5)
    s = _row_scales(x)
    return (x / _spread(s, 1, K)).to(E4M3), s.t().contiguous().t()


def _weight(g, N, K):
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    s = _block_scales(w)
    return (w / _spread(_spread(s, 0, N), 1, K)).to(E4M3), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, M, K = case["op"], case["M"], case["K"]
    state = {"case": case}
    if op in ("norm", "norm_grad"):
        t = TYPES[case["type"]]
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        state["weight"] = (1.0 + 0.1 * rand(K)).to(t)
        if op == "norm":
            state["x"] = rand(M, K).to(t)
            state["residual"] = (3.0 * rand(M, K)).to(t) if case["residual"] else None
        else:
            h = (3.0 * rand(M, K)).to(t)
            state["h"] = h
            state["rstd"] = torch.rsqrt(h.double().square().mean(1) + EPS).float()
            state["dy"] = (0.1 * rand(M, K)).to(t)
            state["dresidual"] = (0.1 * rand(M, K)).to(t) if case["residual"] else None
    elif op == "quantize":
        t = TYPES[case["type"]]
        state["x"] = (torch.randn(M, K, generator=g, device="cuda") * (0.02 if case["block"] else 1.0)).to(t)
    else:
        state["x"], state["x_scale"] = _activations(g, M, K)
        state["w"], state["w_scale"] = _weight(g, case["N"], K)
        if op == "glu":
            state["up"], state["up_scale"] = _weight(g, case["N"], K)
    return state


def _quantized(y):
    s = _row_scales(y)
    return (y / _spread(s, 1, y.shape[1])).to(E4M3), s


def _product(s, w, w_scale):
    M, K = s["x"].shape
    x = s["x"].float() * _spread(s["x_scale"], 1, K)
    return x @ (w.float() * _spread(_spread(w_scale, 0, w.shape[0]), 1, K)).t()


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        t = s["x"].dtype
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(t)
        f = h.float()
        y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        out = list(_quantized(y)) if case["out"] == "fp8" else [y.to(t)]
        return out if s["residual"] is None else out + [h]
    if op == "norm_grad":
        t = s["h"].dtype
        h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
        xhat = h * r
        a = dy * s["weight"].float()
        dx = r * (a - xhat * (a * xhat).mean(1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        return [dx.to(t), (dy * xhat).sum(0).to(t)]
    if op == "quantize":
        y = s["x"].float()
        if not case["block"]:
            return list(_quantized(y))
        b = _block_scales(y)
        return [(y / _spread(_spread(b, 0, y.shape[0]), 1, y.shape[1])).to(E4M3), b]
    y = _product(s, s["w"], s["w_scale"])
    if op == "glu":
        y = y / (1.0 + torch.exp(-y)) * _product(s, s["up"], s["up_scale"])
    return list(_quantized(y)) if case["out"] == "fp8" else [y.to(TYPES[case["out"]])]


def _run_own(s):
    import glu_mlp_gemv_amd as glu

    case = s["case"]
    op = case["op"]
    if op == "norm":
        if case["out"] == "fp8":
            q, scale, h = glu.add_rms_norm_fp8(s["x"], s["weight"], EPS, residual=s["residual"])
            return [q, scale] if s["residual"] is None else [q, scale, h]
        y, h = glu.add_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
        return [y] if s["residual"] is None else [y, h]
    if op == "norm_grad":
        return list(glu.add_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dresidual=s["dresidual"]))
    if op == "quantize":
        return list((glu.fp8_quantize_weight if case["block"] else glu.fp8_quantize)(s["x"]))
    if op == "glu":
        out = glu.fp8_dual_glu(s["x"], s["x_scale"], s["w"], s["w_scale"], s["up"], s["up_scale"],
                               out_dtype=E4M3 if case["out"] == "fp8" else TYPES[case["out"]])
        return list(out) if case["out"] == "fp8" else [out]
    return [glu.fp8_linear(s["x"], s["x_scale"], s["w"], s["w_scale"], out_dtype=TYPES[case["out"]])]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op in ("norm", "norm_grad", "quantize"):
        e = TYPES[case["type"]].itemsize
        G = _groups(K)
    if op == "norm":
        out = M * K + 4 * M * G if case["out"] == "fp8" else M * K * e
        return {"bytes": M * K * e * (3 if case["residual"] else 1) + K * e + out, "flops": 6 * M * K}
    if op == "norm_grad":
        return {"bytes": M * K * e * (4 if case["residual"] else 3) + 4 * M + 2 * K * e, "flops": 10 * M * K}
    if op == "quantize":
        scales = _groups(M) * G if case["block"] else M * G
        return {"bytes": M * K * (e + 1) + 4 * scales, "flops": 3 * M * K}
    N, n = case["N"], 2 if op == "glu" else 1
    G = _groups(K)
    out = M * N + 4 * M * _groups(N) if case["out"] == "fp8" else 2 * M * N
    return {"bytes": M * K + 4 * M * G + n * (N * K + 4 * _groups(N) * G) + out, "flops": 2.0 * n * M * N * K}


def _exact_groups(y):
    """Scales by 128 columns and the quotients before they go to 8 bits."""
    scales = [y[:, c:c + GROUP].abs().max(1).values.div(E4M3_MAX).clamp_min(TINY) for c in range(0, y.shape[1], GROUP)]
    quotients = [y[:, GROUP * b:GROUP * (b + 1)] / sb[:, None] for b, sb in enumerate(scales)]
    return [torch.cat(quotients, 1), torch.stack(scales, 1)]


def _exact_product(x, sx, w, sw):
    """The sum over K-blocks of the unscaled 64-bit products, each scaled by its row's and its block's scale."""
    total = 0.0
    rows = torch.arange(w.shape[0], device=w.device) // GROUP
    for b in range(sx.shape[1]):
        k = slice(GROUP * b, GROUP * (b + 1))
        part = x[:, k].double() @ w[:, k].double().t()
        part *= sx[:, b, None].double()
        part *= sw[rows, b].double()
        total = part.add_(total)
    return total


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
        d = h.double()
        y = d / torch.sqrt((d * d).sum(1, keepdim=True) / d.shape[1] + EPS) * s["weight"].double()
        out = _exact_groups(y) if case["out"] == "fp8" else [y]
        return out if s["residual"] is None else out + [s["x"].double() + s["residual"].double()]
    if op == "norm_grad":
        # d/dh of w . dy . h * rstd(h), with rstd as it was saved: rstd a - h rstd^3 sum(a h) / K
        h, dy, r, w = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None], s["weight"].double()
        dx = r * dy * w - h * r ** 3 * ((dy * w * h).sum(1, keepdim=True) / h.shape[1])
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].double()
        return [dx, (dy * h * r).sum(0)]
    if op == "quantize":
        y = s["x"].double()
        if not case["block"]:
            return _exact_groups(y)
        scales = [[y[i:i + GROUP, j:j + GROUP].abs().max().div(E4M3_MAX).clamp_min(TINY) for j in range(0, y.shape[1], GROUP)]
                  for i in range(0, y.shape[0], GROUP)]
        b = torch.stack([torch.stack(row) for row in scales])
        i = torch.arange(y.shape[0], device=y.device) // GROUP
        j = torch.arange(y.shape[1], device=y.device) // GROUP
        return [y / b[i][:, j], b]
    y = _exact_product(s["x"], s["x_scale"], s["w"], s["w_scale"])
    if op == "glu":
        y = y * torch.sigmoid(y) * _exact_product(s["x"], s["x_scale"], s["up"], s["up_scale"])
    return _exact_groups(y) if case["out"] == "fp8" else [y]
