"""The C ABI of include/glu_adapter.h on the host: refusals before any HIP call, and workspaces (CPU only).

The addresses are made up: a call that got past its checks would launch, so every call here must be
refused or be empty."""
import ctypes

import pytest

from glu_mlp_gemv_amd import adapters, api

OK, NULLP, SHAPE, ALIGN, ALIAS, LAUNCH, UNSUP, STRIDE, WORKSPACE = range(9)
ARG = 10
BF16, FP16, FP32, E4M3 = range(4)
# disjoint made-up arrays, 256 MiB apart
P = [0x100000000 + i * 0x10000000 for i in range(14)]


@pytest.fixture(scope="module")
def lib():
    return api.library()


def sizes(M=4, N=256, K=128, R=16, L=3):
    return adapters.Sizes(M, N, K, R, L)


def need_of(lib, query, *args):
    n = ctypes.c_int64()
    assert getattr(lib, query)(*args, ctypes.byref(n)) == OK
    return n.value


COMMON = [
    (dict(dtype=FP32), ARG), (dict(dtype=E4M3), ARG), (dict(dtype=-1), ARG),
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(L=0), SHAPE), (dict(R=0), SHAPE), (dict(R=257), SHAPE),
    (dict(K=(1 << 23) + 1), SHAPE), (dict(N=(1 << 23) + 1), SHAPE), (dict(ldx=(1 << 23) + 1), STRIDE),
    (dict(a_row=(1 << 23) + 1, a_stack=1 << 30), STRIDE),
    (dict(x=None), NULLP), (dict(a=None), NULLP), (dict(b=None), NULLP), (dict(index=None), NULLP), (dict(ab=None), NULLP),
    (dict(sizes=None), NULLP), (dict(ldx=127), STRIDE), (dict(a_row=127), STRIDE), (dict(a_stack=2047), STRIDE),
    (dict(b_row=15), STRIDE), (dict(b_stack=4095), STRIDE), (dict(a_stack=1 << 62), STRIDE), (dict(b_row=1 << 60), STRIDE),
    (dict(x=P[1] + 1), ALIGN), (dict(a=P[2] + 1), ALIGN), (dict(index=P[4] + 2), ALIGN), (dict(scale=P[5] + 1), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=P[8] + 8), WORKSPACE), (dict(short=1), WORKSPACE),
    (dict(ws=P[1]), ALIAS), (dict(ws=P[4]), ALIAS),
]


def pair(k):
    return None if k["ab"] is None else adapters.Adapter(k["a"], k["b"], k["a_stack"], k["a_row"], k["b_stack"], k["b_row"])


def defaults(kw):
    k = dict(x=P[1], ldx=128, a=P[2], b=P[3], index=P[4], scale=P[5], out=P[6], ldo=256, low=P[7], ws=P[8], short=0, ab=1,
             a_stack=2048, a_row=128, b_stack=4096, b_row=16, dtype=BF16, M=4, N=256, K=128, R=16, L=3, sizes=1)
    k.update(kw)
    k["s"] = sizes(k["M"], k["N"], k["K"], k["R"], k["L"]) if k["sizes"] else None
    return k


def add(lib, y=P[0], ldy=256, **kw):
    k = defaults(kw)
    n = need_of(lib, "glu_adapter_workspace", 1, sizes()) - k["short"]
    return lib.glu_adapter_add(y, ldy, k["x"], k["ldx"], pair(k), k["index"], k["scale"], k["out"], k["ldo"], k["low"],
                               k["s"], k["dtype"], k["ws"], n, None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(y=None), NULLP), (dict(out=None), NULLP), (dict(ldy=255), STRIDE), (dict(ldo=255), STRIDE), (dict(out=P[6] + 1), ALIGN),
    (dict(low=P[7] + 2), ALIGN), (dict(out=P[1]), ALIAS), (dict(out=P[0] + 2), ALIAS), (dict(out=P[0], ldo=300), ALIAS),
    (dict(out=P[2]), ALIAS), (dict(out=P[4]), ALIAS), (dict(low=P[0]), ALIAS), (dict(low=P[6]), ALIAS), (dict(low=P[8]), ALIAS),
    (dict(M=0), OK), (dict(N=0, low=None), OK), (dict(M=0, x=None, y=None, out=None, ws=None), OK), (dict(M=1 << 31), SHAPE),
])
def test_add_refusals(lib, kw, status):
    assert add(lib, **kw) == status


def glu(lib, gate=P[0], up=P[9], ldg=256, ldu=256, **kw):
    k = defaults(kw)
    uab = adapters.Adapter(P[10], P[11], 2048, 128, 4096, 16) if k.get("uab", 1) else None
    n = need_of(lib, "glu_adapter_workspace", 2, sizes()) - k["short"]
    return lib.glu_adapter_glu(gate, ldg, up, ldu, k["x"], k["ldx"], pair(k), uab, k["index"], k["scale"], k["out"], k["ldo"],
                               k["s"], k["dtype"], k["ws"], n, None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(gate=None), NULLP), (dict(up=None), NULLP), (dict(uab=None), NULLP), (dict(ldu=255), STRIDE), (dict(out=P[10]), ALIAS),
    (dict(out=P[9] + 512), ALIAS), (dict(M=0), OK), (dict(N=0), OK),
])
def test_glu_refusals(lib, kw, status):
    assert glu(lib, **kw) == status


def backward(lib, dout=P[0], ldd=256, dx=P[9], lddx=128, da=P[10], db=P[11], **kw):
    k = defaults(kw)
    n = need_of(lib, "glu_adapter_backward_workspace", sizes()) - k["short"]
    return lib.glu_adapter_backward(dout, ldd, k["x"], k["ldx"], pair(k), k["index"], k["scale"], k["low"], dx, lddx, da, db,
                                    k["s"], k["dtype"], k["ws"], n, None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dout=None), NULLP), (dict(low=None), NULLP), (dict(ldd=255), STRIDE), (dict(lddx=127), STRIDE),
    (dict(dx=P[0]), ALIAS), (dict(da=P[2]), ALIAS), (dict(db=P[10]), ALIAS), (dict(dx=P[7]), ALIAS), (dict(da=P[8]), ALIAS),
    (dict(dx=None, da=None, db=None), OK), (dict(M=(1 << 24) + 1), SHAPE), (dict(N=(1 << 23) + 1), SHAPE),
    (dict(L=65537), SHAPE), (dict(ldd=(1 << 23) + 1), STRIDE), (dict(lddx=(1 << 23) + 1), STRIDE),
])
def test_backward_refusals(lib, kw, status):
    assert backward(lib, **kw) == status


def test_workspaces(lib):
    need = lambda *a: need_of(lib, "glu_adapter_workspace", *a)  # noqa: E731
    assert need(1, sizes(M=0)) == 0
    for M in (1, 16, 17, 256, 257, 5000):
        for K in (0, 1, 64, 4096, 17408):
            for R in (1, 16, 65, 256):
                one, two = need(1, sizes(M=M, K=K, R=R)), need(2, sizes(M=M, K=K, R=R))
                assert one % 16 == 0 and one >= M * R * 4 and (one % (M * R * 4)) < 16 and two >= 2 * M * R * 4
                assert one <= 16 * M * R * 4 + 16
    n = ctypes.c_int64()
    r = ctypes.byref(n)
    assert lib.glu_adapter_workspace(3, sizes(), r) == ARG and lib.glu_adapter_workspace(1, sizes(R=0), r) == SHAPE
    assert lib.glu_adapter_workspace(1, None, r) == NULLP and lib.glu_adapter_workspace(1, sizes(), None) == NULLP
    assert lib.glu_adapter_backward_workspace(sizes(L=0), r) == SHAPE
    assert lib.glu_adapter_backward_workspace(sizes(), None) == NULLP
    assert need_of(lib, "glu_adapter_backward_workspace", sizes(M=0)) == 0
    # past one item per adapter: the order, the table of items and their sums
    small = need_of(lib, "glu_adapter_backward_workspace", sizes(M=512))
    large = need_of(lib, "glu_adapter_backward_workspace", sizes(M=513))
    assert large > small + 513 * 4 + 3 * 16 * (256 + 128) * 4
