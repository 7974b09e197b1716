"""The C ABI of include/glu_moe.h on the host: refusals before any HIP call, and workspaces (CPU only).

The addresses are made up: a call that got past its checks would launch, so every call here must be
refused or be empty."""
import ctypes

import pytest

from glu_mlp_gemv_amd import api, moe

OK, NULLP, SHAPE, ALIGN, ALIAS, LAUNCH, UNSUP, STRIDE, WORKSPACE = range(9)
ARG = 10
BF16, FP16, FP32, E4M3 = range(4)
P = [0x100000000 + i * 0x10000000 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    return api.library()


def call(lib, **kw):
    k = dict(x=P[0], ldx=256, logits=P[1], ldl=8, lt=FP32, gate=P[2], gs=P[3], up=P[4], us=P[5], down=P[6], ds=P[7], stack=32768,
             ld=256, dstack=32768, dld=128, sstack=2, sld=2, out=P[8], ldo=256, M=4, K=256, N=128, E=8, top=2, dtype=BF16,
             wt=E4M3, ws=P[9], short=0, mats=7, sizes=1)
    k.update(kw)
    n = ctypes.c_int64()
    assert lib.glu_moe_workspace(moe.Sizes(4, 256, 128, 8, 2), ctypes.byref(n)) == OK
    g, u = (moe.Matrix(d, s, k["stack"], k["ld"], k["sstack"], k["sld"]) for d, s in ((k["gate"], k["gs"]), (k["up"], k["us"])))
    d = moe.Matrix(k["down"], k["ds"], k["dstack"], k["dld"], k["sstack"], 1)
    g, u, d = (m if k["mats"] >> i & 1 else None for i, m in enumerate((g, u, d)))
    sizes = moe.Sizes(k["M"], k["K"], k["N"], k["E"], k["top"]) if k["sizes"] else None
    return lib.glu_moe_glu(k["x"], k["ldx"], k["logits"], k["ldl"], k["lt"], g, u, d, k["out"], k["ldo"], sizes, 1, k["dtype"],
                           k["wt"], k["ws"], n.value - k["short"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=FP32), ARG), (dict(dtype=E4M3), ARG), (dict(lt=FP16), ARG), (dict(wt=FP16), ARG), (dict(wt=FP32), ARG),
    (dict(M=-1), SHAPE), (dict(K=-1), SHAPE), (dict(N=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, top=1), SHAPE),
    (dict(top=0), SHAPE), (dict(top=9), SHAPE), (dict(E=64, top=33), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=(1 << 24) + 1), SHAPE),
    (dict(M=64, E=1024, top=32, N=1 << 24), SHAPE), (dict(sizes=0), NULLP), (dict(mats=3), NULLP), (dict(mats=6), NULLP),
    (dict(x=None), NULLP), (dict(logits=None), NULLP), (dict(gate=None), NULLP), (dict(ds=None), NULLP), (dict(out=None), NULLP),
    (dict(ldx=255), STRIDE), (dict(ldl=7), STRIDE), (dict(ld=255), STRIDE), (dict(stack=32767), STRIDE), (dict(dld=127), STRIDE),
    (dict(sstack=1), STRIDE), (dict(ldo=255), STRIDE), (dict(stack=1 << 62), STRIDE), (dict(ld=1 << 61), STRIDE),
    (dict(x=P[0] + 1), ALIGN), (dict(logits=P[1] + 2), ALIGN), (dict(gs=P[3] + 2), ALIGN), (dict(wt=BF16, gate=P[2] + 1), ALIGN),
    (dict(out=P[0]), ALIAS), (dict(out=P[1]), ALIAS), (dict(out=P[2] + 512), ALIAS), (dict(out=P[7]), ALIAS), (dict(ws=P[0]), ALIAS),
    (dict(ws=P[8]), ALIAS), (dict(ws=None), WORKSPACE), (dict(ws=P[9] + 8), WORKSPACE), (dict(short=1), WORKSPACE),
    (dict(M=0), OK), (dict(K=0), OK), (dict(M=0, x=None, logits=None, gate=None, out=None, ws=None), OK),
])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_workspaces(lib):
    n = ctypes.c_int64()
    r = ctypes.byref(n)
    seen = {}
    for M in (0, 1, 8, 63, 64, 65, 200, 5000):
        assert lib.glu_moe_workspace(moe.Sizes(M, 2560, 1024, 64, 8), r) == OK
        seen[M] = n.value
        assert n.value % 16 == 0
    assert seen[0] == 0 and seen[1] >= 8 * 1024 * 2 and seen[64] >= 64 * 8 * 1024 * 2
    assert seen[64] <= seen[65] <= seen[5000] + 0 <= seen[64] + seen[65], "64 rows at a time"
    assert lib.glu_moe_workspace(moe.Sizes(1, 64, 64, 4, 5), r) == SHAPE and n.value == 0
    assert lib.glu_moe_workspace(None, r) == NULLP and lib.glu_moe_workspace(moe.Sizes(1, 64, 64, 4, 4), None) == NULLP
