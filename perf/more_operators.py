"""Measured cases of the operators whose weights a token chooses, and of the dropout they are trained with.

Low-rank adapters beside a shared projection (each row of a batch names its adapter), alone and inside the GLU, with
their backward; a mixture-of-experts GLU layer for a few tokens, on 16-bit or block-scaled e4m3 weights; and
dropout whose mask is computed from a counter.  ``run`` computes a pass in elementary torch operations in 32 bits, or
with ``own`` through the framework's entry points; ``exact`` is the definition in 64 bits.

Dropout's random numbers: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
2011) with key (seed low, seed high) and counter (k // 8, m, offset low, offset high) for element (m, k); the four
words are eight draws of 16 bits, the low half of a word first, and draw k % 8 is the element's.  It is kept where the
draw is at least round(65536 p).
"""
import math

import torch

own = False

GROUP = 128
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one request, its adapter on an up projection: latency alone
        {"name": "adapter_token", "op": "adapter", "M": 1, "K": 2560, "N": 9216, "R": 16, "L": 8, "order": "mixed",
         "none": 0.0, "type": "bf16"},
        # a decode batch with an odd number of sequences, some of them without an adapter
        {"name": "adapter_batch", "op": "adapter", "M": 37, "K": 4096, "N": 12288, "R": 16, "L": 32, "order": "mixed",
         "none": 0.1, "type": "bf16"},
        # a prefill of four requests, adapters of rank 64
        {"name": "adapter_prefill", "op": "adapter", "M": 8192, "K": 5120, "N": 5120, "R": 64, "L": 4,
         "order": "segments", "none": 0.0, "type": "fp16"},
        # a decode batch through the GLU with adapters on gate and up
        {"name": "adapter_glu_batch", "op": "adapter_glu", "M": 64, "K": 2560, "N": 9216, "R": 32, "L": 16,
         "order": "mixed", "none": 0.0, "type": "bf16"},
        # a prefill of three requests through the same, lengths that fill no tile
        {"name": "adapter_glu_prefill", "op": "adapter_glu", "M": 2050, "K": 4096, "N": 12288, "R": 16, "L": 3,
         "order": "segments", "none": 0.0, "type": "bf16"},
        # a short ragged training batch
        {"name": "adapter_grad_short", "op": "adapter_grad", "M": 203, "K": 2560, "N": 2560, "R": 8, "L": 2,
         "order": "segments", "none": 0.0, "type": "fp16"},
        # a training micro-batch of 16384 tokens that tunes four adapters at once
        {"name": "adapter_grad_long", "op": "adapter_grad", "M": 16384, "K": 4096, "N": 4096, "R": 16, "L": 4,
         "order": "segments", "none": 0.0, "type": "bf16"},
        # one token through a layer of 64 experts
        {"name": "moe_token", "op": "moe", "M": 1, "K": 2560, "N": 1024, "E": 64, "top": 8, "type": "bf16", "e4m3": False},
        # a decode batch through a layer of 128 narrow experts, nearly all of which it needs
        {"name": "moe_batch", "op": "moe", "M": 37, "K": 4096, "N": 768, "E": 128, "top": 8, "type": "bf16", "e4m3": False},
        # a few tokens (of a draft, say) through 8-bit experts
        {"name": "moe_few_e4m3", "op": "moe", "M": 6, "K": 4096, "N": 1536, "E": 128, "top": 8, "type": "bf16",
         "e4m3": True},
        # the residual stream of a short ragged training batch
        {"name": "dropout_short", "op": "dropout", "M": 203, "K": 2560, "p": 0.1, "residual": True, "type": "bf16"},
        # the gradient of a micro-batch of 16384 tokens on its way back through the mask
        {"name": "dropout_long", "op": "dropout", "M": 16384, "K": 4096, "p": 0.05, "residual": False, "type": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """Most widths are whole multiples of 64; the others stay odd."""
    n = _log(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["adapter", "adapter", "adapter_glu", "adapter_grad", "moe", "moe", "dropout"])
    kind = rng.choice(["bf16", "bf16", "fp16"])
    if op == "moe":
        E = _log(rng, 4, 128)
        K = _width(rng, 256, 4096)
        N = max(64, min(_width(rng, 128, 2048), (1 << 28) // (E * K)))
        return {"op": op, "M": _log(rng, 1, 64), "K": K, "N": N, "E": E, "top": rng.randint(1, min(E, 8)), "type": kind,
                "e4m3": rng.random() < 0.4}
    if op == "dropout":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _width(rng, 128, 8192), "p": rng.choice([0.05, 0.1, 0.3, 0.5]),
                "residual": rng.random() < 0.5, "type": rng.choice(["bf16", "fp16", "fp32"])}
    M = _log(rng, 1, 8192 if op == "adapter" else 4096)
    return {"op": op, "M": M, "K": _width(rng, 128, 5120), "N": _width(rng, 128, 8192), "R": rng.choice([4, 8, 16, 16, 24, 32, 64]),
            "L": _log(rng, 1, 32), "order": "mixed" if M <= 256 and rng.random() < 0.7 else "segments",
            "none": rng.choice([0.0, 0.0, 0.2]), "type": kind}


def _groups(n):
    return -(-n // GROUP)


def _rows_without(case):
    return int(case["M"] * case["none"])


def _index(g, case):
    """The adapter of each row: as many adapters as there are (or rows), each in one run of rows or anywhere."""
    M, L = case["M"], case["L"]
    used = min(L, M - _rows_without(case))
    names = torch.randperm(L, generator=g, device="cuda")[:used]
    index = names[torch.arange(M, device="cuda") * used // M]
    if case["order"] == "mixed":
        index = names[torch.arange(M, device="cuda") % used]
        index[M - _rows_without(case):] = -1
        index = index[torch.randperm(M, generator=g, device="cuda")]
    else:
        index[M - _rows_without(case):] = -1
    return index.to(torch.int32)


def _blocks(s, rows, cols):
    """One value per block of 128 x 128 as one per element."""
    return s.repeat_interleave(GROUP, -2)[..., :rows, :].repeat_interleave(GROUP, -1)[..., :cols]


def _weight8(w):
    """A 16-bit expert's matrix [rows, cols] in e4m3 and its blocks' scales."""
    rows, cols = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -cols % GROUP, 0, -rows % GROUP))
    s = p.view(_groups(rows), GROUP, _groups(cols), GROUP).abs().amax((1, 3)).div(E4M3_MAX).clamp_min(2.0 ** -126)
    return (w.float() / _blocks(s, rows, cols)).to(E4M3), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, M, K, t = case["op"], case["M"], case["K"], TYPES[case["type"]]
    state = {"case": case}
    if op == "dropout":
        state["x"] = rand(M, K).to(t)
        state["residual"] = (3.0 * rand(M, K)).to(t) if case["residual"] else None
        state["seed"], state["offset"] = 0x9E3779B97F4A7C15 * (int(seed) + 1) % (1 << 64), 3
        return state
    N = case["N"]
    state["x"] = rand(M, K).to(t)
    if op == "moe":
        E = case["E"]
        state["logits"] = rand(M, E)  # uniform routing: the number of experts that a batch needs follows from M, E and top
        for name, rows, cols in (("gate", N, K), ("up", N, K), ("down", K, N)):
            w = torch.empty(E, rows, cols, dtype=E4M3 if case["e4m3"] else t, device="cuda")
            scales = []
            for e in range(E):
                one = (rand(rows, cols) * cols ** -0.5).to(t)
                if case["e4m3"]:
                    one, s = _weight8(one)
                    scales.append(s)
                w[e] = one
            state[name] = w
            state[name + "_scale"] = torch.stack(scales) if case["e4m3"] else None
        return state
    L, R = case["L"], case["R"]
    state["index"] = _index(g, case)
    state["scale"] = 2.0 * torch.rand(L, generator=g, device="cuda") + 0.5  # alpha / rank
    for i in range(2 if op == "adapter_glu" else 1):
        state["a%d" % i] = (rand(L, R, K) * K ** -0.5).to(t)
        state["b%d" % i] = (rand(L, N, R) * 0.5 * R ** -0.5).to(t)
        if op != "adapter_grad":
            state["y%d" % i] = rand(M, N).to(t)
    if op == "adapter_grad":
        state["dout"] = (0.1 * rand(M, N)).to(t)
        # what the forward keeps for the backward: x a^T in 32 bits, zeros where a row has no adapter
        rows = (state["index"] >= 0).nonzero()[:, 0]
        low = torch.zeros(M, R, device="cuda")
        for l in state["index"][rows].unique().tolist():
            mine = (state["index"] == l).nonzero()[:, 0]
            low[mine] = (state["x"][mine].double() @ state["a0"][l].double().t()).float()
        state["low"] = low
    return state


def _chosen(s):
    """[M, L, 1]: whether a row has that adapter."""
    return (s["index"][:, None] == torch.arange(s["case"]["L"], device="cuda")[None, :])[:, :, None]


def _delta(s, i, chosen):
    """The i-th adapters' part of the projection: the products of all adapters, of which a row keeps its own."""
    L, R = s["case"]["L"], s["case"]["R"]
    low = (s["x"].float() @ s["a%d" % i].float().flatten(0, 1).t()).unflatten(1, (L, R))
    low = torch.where(chosen, low * s["scale"][:, None], 0.0).flatten(1)
    return low @ s["b%d" % i].float().transpose(1, 2).reshape(L * R, -1)


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _route(logits, top):
    """Experts and weights [M, top]: the largest logits (of equal ones the lowest index), softmax over them."""
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    best = torch.exp(order.values[:, :top] - order.values[:, :1])
    return order.indices[:, :top], best / best.sum(1, keepdim=True)


def _expert(s, name, ids):
    w = s[name][ids].float()
    return w if s[name + "_scale"] is None else w * _blocks(s[name + "_scale"][ids], *w.shape[1:])


def _philox(c0, c1, c2, c3, key):
    """Ten rounds on tensors of 32-bit words, held in 64."""
    low = 0xFFFFFFFF
    k0, k1 = key & low, key >> 32
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64; the shift's sign bits are masked away
        c0, c1, c2, c3 = (q >> 32 & low) ^ c1 ^ k0, q & low, (p >> 32 & low) ^ c3 ^ k1, p & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return c0, c1, c2, c3


def _kept(s):
    M, K = s["x"].shape
    row = torch.arange(M, device="cuda")[:, None].expand(M, -(-K // 8))
    block = torch.arange(-(-K // 8), device="cuda")[None, :].expand_as(row)
    offset = s["offset"]
    words = _philox(block, row, torch.full_like(row, offset & 0xFFFFFFFF), torch.full_like(row, offset >> 32), s["seed"])
    draws = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 2).flatten(1)[:, :K]
    return draws >= round(65536 * s["case"]["p"])


def _run_plain(s):
    case = s["case"]
    op, t = case["op"], s["x"].dtype
    if op == "dropout":
        out = torch.where(_kept(s), s["x"].float() * (65536 / (65536 - round(65536 * case["p"]))), 0.0)
        return [(out if s["residual"] is None else s["residual"].float() + out).to(t)]
    if op == "moe":
        ids, weights = _route(s["logits"], case["top"])
        rows = []
        for m in range(case["M"]):
            x = s["x"][m].float()
            a = _silu(_expert(s, "gate", ids[m]) @ x) * (_expert(s, "up", ids[m]) @ x)
            rows.append(((_expert(s, "down", ids[m]) * a[:, None, :]).sum(2) * weights[m][:, None]).sum(0))
        return [torch.stack(rows).to(t)]
    chosen = _chosen(s)
    if op == "adapter":
        return [(s["y0"].float() + _delta(s, 0, chosen)).to(t)]
    if op == "adapter_glu":
        gate, up = (s["y%d" % i].float() + _delta(s, i, chosen) for i in (0, 1))
        return [(_silu(gate) * up).to(t)]
    L, R = case["L"], case["R"]
    a, b = s["a0"].float().flatten(0, 1), s["b0"].float().transpose(1, 2).reshape(L * R, -1)
    dout, x = s["dout"].float(), s["x"].float()
    dlow = torch.where(chosen, (dout @ b.t()).unflatten(1, (L, R)) * s["scale"][:, None], 0.0).flatten(1)
    low = torch.where(chosen, s["low"][:, None, :] * s["scale"][:, None], 0.0).flatten(1)
    db = (low.t() @ dout).unflatten(0, (L, R)).transpose(1, 2)
    return [(dlow @ a).to(t), (dlow.t() @ x).unflatten(0, (L, R)).to(t), db.to(t).contiguous()]


def _run_own(s):
    import glu_mlp_gemv_amd as glu

    case = s["case"]
    op = case["op"]
    if op == "dropout":
        return [glu.dropout(s["x"], case["p"], s["seed"], s["offset"], residual=s["residual"])]
    if op == "moe":
        return [glu.moe_glu(s["x"], s["logits"], s["gate"], s["up"], s["down"], case["top"], gate_scale=s["gate_scale"],
                            up_scale=s["up_scale"], down_scale=s["down_scale"])]
    if op == "adapter":
        return [glu.adapter_add(s["y0"], s["x"], s["a0"], s["b0"], s["index"], s["scale"])]
    if op == "adapter_glu":
        return [glu.adapter_glu(s["y0"], s["y1"], s["x"], s["a0"], s["b0"], s["a1"], s["b1"], s["index"], s["scale"])]
    return list(glu.adapter_backward(s["dout"], s["x"], s["a0"], s["b0"], s["index"], s["low"], s["scale"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    e = TYPES[case["type"]].itemsize
    if op == "dropout":
        return {"bytes": M * K * e * (3 if case["residual"] else 2), "flops": 2 * M * K}
    N = case["N"]
    if op == "moe":
        E, top = case["E"], case["top"]
        needed = E * (1.0 - (1.0 - top / E) ** M)  # experts that M tokens choose, each uniformly: the mean
        matrix = N * K + 4 * _groups(N) * _groups(K) if case["e4m3"] else N * K * e
        return {"bytes": int(3 * needed * matrix) + 2 * M * K * e + 4 * M * E, "flops": 6.0 * M * top * N * K}
    L, R, rows = case["L"], case["R"], M - _rows_without(case)
    used = min(L, rows)
    if op == "adapter_grad":
        return {"bytes": 2 * M * K * e + M * N * e + 4 * M * R + 4 * M + 2 * L * R * (K + N) * e,
                "flops": 4.0 * rows * R * (K + N)}
    n = 2 if op == "adapter_glu" else 1
    return {"bytes": M * K * e + n * used * R * (K + N) * e + (n + 1) * M * N * e + 4 * M,
            "flops": 2.0 * n * rows * R * (K + N)}


def _wide_product(x, y):
    """The 64-bit product of two 32-bit words as (high, low), from products of 16 bits."""
    x0, x1, y0, y1 = x & 0xFFFF, x >> 16, y & 0xFFFF, y >> 16
    mid = x1 * y0 + (x0 * y0 >> 16)
    mid2 = x0 * y1 + (mid & 0xFFFF)
    return x1 * y1 + (mid >> 16) + (mid2 >> 16), (mid2 & 0xFFFF) << 16 | x0 * y0 & 0xFFFF


def _exact_dropout(s):
    x = s["x"].double()
    M, K = x.shape
    drop = round(65536 * s["case"]["p"])
    k, m = torch.arange(K, device="cuda"), torch.arange(M, device="cuda")[:, None]
    word = [(k // 8).expand(M, K), m.expand(M, K), torch.tensor(s["offset"] % 2 ** 32, device="cuda"),
            torch.tensor(s["offset"] // 2 ** 32, device="cuda")]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for r in range(10):
        h0, l0 = _wide_product(word[0], 0xD2511F53)
        h2, l2 = _wide_product(word[2], 0xCD9E8D57)
        word = [h2 ^ word[1] ^ (key[0] + r * 0x9E3779B9) % 2 ** 32, l2, h0 ^ word[3] ^ (key[1] + r * 0xBB67AE85) % 2 ** 32, l0]
    half = k % 8
    mine = torch.where(half < 2, word[0], torch.where(half < 4, word[1], torch.where(half < 6, word[2], word[3])))
    draws = mine // torch.where(half % 2 == 1, 65536, 1) % 65536
    out = x * (draws >= drop) / (1.0 - drop / 65536.0)
    return [out if s["residual"] is None else out + s["residual"].double()]


def _exact_weight(s, name, e):
    w = s[name][e].double()
    if s[name + "_scale"] is not None:
        i, j = (torch.arange(n, device="cuda") // GROUP for n in w.shape)
        w = w * s[name + "_scale"][e].double()[i][:, j]
    return w


def _exact_moe(s):
    logits, x, top = s["logits"].double(), s["x"].double(), s["case"]["top"]
    out = torch.zeros_like(x)
    # an expert is chosen by a row where fewer than `top` others come before it
    col = torch.arange(logits.shape[1], device="cuda")
    before = (logits[:, None, :] > logits[:, :, None]) | ((logits[:, None, :] == logits[:, :, None]) & (col[None, :] < col[:, None]))
    chosen = before.sum(2) < top
    weights = torch.softmax(logits.masked_fill(~chosen, -math.inf), 1)
    for e in range(logits.shape[1]):
        rows = chosen[:, e].nonzero()[:, 0]
        if rows.numel():
            g = x[rows] @ _exact_weight(s, "gate", e).t()
            a = g * torch.sigmoid(g) * (x[rows] @ _exact_weight(s, "up", e).t())
            out[rows] += weights[rows, e, None] * (a @ _exact_weight(s, "down", e).t())
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        return _exact_dropout(s)
    if op == "moe":
        return _exact_moe(s)
    groups = [(l, (s["index"] == l).nonzero()[:, 0], float(s["scale"][l])) for l in range(case["L"])]
    x = s["x"].double()
    if op == "adapter_grad":
        dout = s["dout"].double()
        dx, da, db = torch.zeros_like(x), [], []
        for l, rows, scale in groups:
            a, b = s["a0"][l].double(), s["b0"][l].double()
            through = scale * (dout[rows] @ b)
            dx[rows] = through @ a
            da.append(through.t() @ x[rows])
            db.append(scale * (dout[rows].t() @ s["low"][rows].double()))
        return [dx, torch.stack(da), torch.stack(db)]
    y = []
    for i in range(2 if op == "adapter_glu" else 1):
        y.append(s["y%d" % i].double())
        for l, rows, scale in groups:
            y[i][rows] += scale * (x[rows] @ s["a%d" % i][l].double().t() @ s["b%d" % i][l].double().t())
    return [y[0] if len(y) == 1 else y[0] * torch.sigmoid(y[0]) * y[1]]
