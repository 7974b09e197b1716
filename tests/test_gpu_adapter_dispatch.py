"""Adapters at sizes that reach every kernel variant, each with several stages of its loop, tails and ranks that fill no tile."""
import pytest
import torch

import adapter_ref as ref
import glu_mlp_gemv_amd as glu
import test_gpu_adapter as base
from fp8_ref import check_store

T = {"bf16": torch.bfloat16, "fp16": torch.float16}
# M, K, N, R, L.  Widths that are multiples of 8 are whole 16-byte chunks a row
CASES = [(2050, 4120, 4104, 16, 3), (1100, 8200, 8216, 32, 3), (1100, 8198, 330, 24, 5), (4200, 2568, 2600, 64, 4),
         (4200, 1096, 328, 40, 3), (2050, 4104, 2056, 48, 3), (4200, 1030, 331, 64, 3), (1100, 8203, 130, 16, 2)]


def variants(M, C, N, R, L, mats, backward):
    """The two products' kernels and the stages of the first one's busiest wave, by the rules of glu_adapter.hip.  backward: C are
    dout's columns and b is read turned, in rows of whole chunks (past 512 rows)."""
    mixed = M <= 1024 and M < 16 * L
    few = M <= 256 or mixed
    by_columns = backward and M <= 512
    if few or by_columns:
        first, tm, rt = ("one" if not by_columns else "columns"), 1, 1
    else:
        tm, rt = (4, 1) if R <= 16 else (4, 2) if R <= 32 else (4, 4) if M > 4096 else (2, 4)
        if C % 8 == 0:
            first = f"tile {tm} {rt}"
        else:
            first = f"gather {min(tm, 8 // rt)} {rt}"
    rows = 16 * tm if tm > 1 else 64 if mixed else 16
    tiles = -(-M // rows)
    units = tiles if not mixed else min(tiles * L, M)
    groups = units * mats * -(-R // (16 * rt))
    parts = max(1, min((768 if tm == 1 else 256) // groups, -(-C // 256), 4 if tm == 1 else 16))
    stages = -(-(-(-C // 64)) // parts)
    s = 0 if R > 64 else 1 if R <= 16 else 2 if R <= 32 else 4
    out = 1 if few or R > 64 else 4 if mats == 1 else 2
    return first, -(-stages // 4), f"out {out} {mats} {s}" + (" columns" if backward else "")


def test_every_variant_is_reached():
    shapes = base.SHAPES + CASES
    seen = {}
    for M, K, N, R, L in shapes:
        for first, stages, second in (variants(M, K, N, R, L, 1, False), variants(M, K, N, R, L, 2, False),
                                      variants(M, N, K, R, L, 1, True)):
            seen[first] = max(seen.get(first, 0), stages)
            seen[second] = 0
    want = {"one", "columns", "tile 4 1", "tile 4 2", "tile 4 4", "tile 2 4", "gather 4 1", "gather 4 2", "gather 2 4"}
    assert all(seen[v] >= 3 for v in want), seen
    want |= {f"out 1 {mats} {s}{c}" for s in (0, 1, 2, 4) for mats, c in ((1, ""), (2, ""), (1, " columns"))}
    want |= {f"out {tm} {mats} {s}{c}" for s in (1, 2, 4) for tm, mats, c in ((4, 1, ""), (2, 2, ""), (4, 1, " columns"))}
    assert want == set(seen), want ^ set(seen)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["mixed", "segments"])
@pytest.mark.parametrize("M,K,N,R,L", CASES)
def test_add_and_glu(M, K, N, R, L, order, kind):
    print(f"[adapter variants] {M=} {K=} {N=} {R=} {L=} {order} {kind}", flush=True)
    (y, u), x, ((a, b), (ua, ub)), index, scale = base.operands(M, K, N, R, L, T[kind], order, M + K, 2)
    g64 = ref.add64(y, x, a, b, index, scale)
    out, low = glu.adapter_add(y, x, a, b, index, scale, return_low=True)
    torch.cuda.synchronize()
    check_store("out", out, *g64)
    check_store("low", low, *ref.low64(x, a, index))
    assert torch.equal(out, glu.adapter_add(y, x, a, b, index, scale)), "the same bits without low, and again"
    u64 = ref.add64(u, x, ua, ub, index, scale)
    act = glu.adapter_glu(y, u, x, a, b, ua, ub, index, scale)
    torch.cuda.synchronize()
    check_store("glu", act, *ref.glu64(g64[0], u64[0], g64[1], u64[1]))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["mixed", "segments"])
@pytest.mark.parametrize("M,K,N,R,L", CASES)
def test_backward(M, K, N, R, L, order, kind):
    print(f"[adapter variants, backward] {M=} {K=} {N=} {R=} {L=} {order} {kind}", flush=True)
    (dout,), x, ((a, b),), index, scale = base.operands(M, K, N, R, L, T[kind], order, M + R)
    dout *= 0.1
    low = ref.low64(x, a, index)[0].float()
    got = glu.adapter_backward(dout, x, a, b, index, low, scale)
    torch.cuda.synchronize()
    for name, v, (w, bound) in zip(("dx", "da", "db"), got, ref.backward64(dout, x, a, b, index, low, scale)):
        check_store(name, v, w, bound)
    again = glu.adapter_backward(dout, x, a, b, index, low, scale)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "a second call gives the same bits"
