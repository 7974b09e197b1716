"""The C ABI of include/glu_fp8.h on the host: refusals before any HIP call, and launch plans (CPU only).

The addresses are made up: a call that got past its checks would launch, so every call here must be
refused or be empty."""
import ctypes

import pytest

from glu_mlp_gemv_amd import api, fp8

OK, NULLP, SHAPE, ALIGN, ALIAS, LAUNCH, UNSUP, STRIDE, WORKSPACE = range(9)
ARG = 10
BF16, FP16, FP32, E4M3 = range(4)
# disjoint made-up arrays, 256 MiB apart
P = [0x100000000 + i * 0x10000000 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    return api.library()


def norm(lib, **kw):
    a = dict(x=P[0], ldx=256, res=P[1], ldr=256, w=P[2], sum=P[3], lds=256, out=P[4], ldo=256, rstd=P[5], M=4, K=256,
             eps=1e-6, dtype=BF16)
    a.update(kw)
    return lib.glu_add_rms_norm(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["sum"], a["lds"], a["out"], a["ldo"],
                                a["rstd"], a["M"], a["K"], a["eps"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(dtype=7), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(M=-1), SHAPE), (dict(K=-1), SHAPE), (dict(K=0), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=1 << 31), SHAPE),
    (dict(M=0), OK), (dict(M=0, x=None, w=None, out=None), OK),
    (dict(sum=None), NULLP), (dict(res=None), NULLP), (dict(x=None), NULLP), (dict(w=None), NULLP), (dict(out=None), NULLP),
    (dict(ldx=255), STRIDE), (dict(ldr=0), STRIDE), (dict(lds=-256), STRIDE), (dict(ldo=255), STRIDE),
    (dict(ldx=1 << 62), STRIDE),
    (dict(x=P[0] + 1), ALIGN), (dict(out=P[4] + 1), ALIGN), (dict(rstd=P[5] + 2), ALIGN),
    (dict(dtype=FP32, w=P[2] + 2), ALIGN),
    (dict(out=P[0]), ALIAS), (dict(out=P[1] + 512), ALIAS), (dict(out=P[2]), ALIAS), (dict(out=P[3]), ALIAS),
    (dict(sum=P[1] + 2), ALIAS), (dict(sum=P[1], lds=300), ALIAS), (dict(sum=P[2]), ALIAS), (dict(rstd=P[4]), ALIAS),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def test_norm_fp8_refusals(lib):
    def call(q=P[4], ldq=256, scale=P[5], lds=4, M=4):
        return lib.glu_add_rms_norm_fp8(P[0], 256, None, 0, P[2], None, 0, q, ldq, scale, lds, None, M, 256, 1e-6, BF16,
                                        None)
    assert call(q=None) == NULLP and call(scale=None) == NULLP
    assert call(ldq=255) == STRIDE and call(lds=3) == STRIDE
    assert call(scale=P[5] + 2) == ALIGN
    assert call(q=P[5]) == ALIAS and call(scale=P[0]) == ALIAS
    assert call(M=0) == OK


def test_norm_backward_refusals(lib):
    need = ctypes.c_int64()
    assert lib.glu_add_rms_norm_backward_workspace(100, 512, ctypes.byref(need)) == OK
    assert need.value % 4 == 0 and need.value >= 2 * 512 * 4
    assert lib.glu_add_rms_norm_backward_workspace(1, 512, ctypes.byref(need)) == OK and need.value == 0
    assert lib.glu_add_rms_norm_backward_workspace(0, 512, ctypes.byref(need)) == OK and need.value == 0
    assert lib.glu_add_rms_norm_backward_workspace(5, 0, ctypes.byref(need)) == SHAPE
    assert lib.glu_add_rms_norm_backward_workspace(5, 5, None) == NULLP
    lib.glu_add_rms_norm_backward_workspace(100, 512, ctypes.byref(need))

    def call(dy=P[0], lddy=512, h=P[1], w=P[2], rstd=P[3], dr=P[4], dx=P[5], dw=P[6], M=100, K=512, dtype=BF16,
             ws=P[7], n=need.value):
        return lib.glu_add_rms_norm_backward(dy, lddy, h, 512, w, rstd, dr, 512, dx, 512, dw, M, K, dtype, ws, n, None)
    for name in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert call(**{name: None}) == NULLP
    assert call(dtype=E4M3) == ARG and call(M=-1) == SHAPE and call(K=0) == SHAPE
    assert call(lddy=511) == STRIDE and call(dx=P[5] + 1) == ALIGN
    assert call(dx=P[0]) == ALIAS and call(dx=P[4] + 2) == ALIAS and call(dw=P[2]) == ALIAS and call(dw=P[5]) == ALIAS
    assert call(ws=P[1]) == ALIAS
    assert call(ws=None) == WORKSPACE and call(ws=P[7] + 4) == WORKSPACE and call(n=need.value - 1) == WORKSPACE


def test_quantize_refusals(lib):
    for f, scale_ld in ((lib.glu_fp8_quantize, 4), (lib.glu_fp8_quantize_weight, 2)):
        def call(x=P[0], ldx=256, q=P[1], ldq=256, s=P[2], lds=scale_ld, M=4, K=256, dtype=BF16):
            return f(x, ldx, q, ldq, s, lds, M, K, dtype, None)
        assert call(dtype=E4M3) == ARG and call(M=-1) == SHAPE and call(K=1 << 31) == SHAPE
        assert call(M=0) == OK and call(K=0) == OK
        assert call(x=None) == NULLP and call(q=None) == NULLP and call(s=None) == NULLP
        assert call(ldx=255) == STRIDE and call(ldq=255) == STRIDE and call(M=400, lds=1) == STRIDE
        assert call(x=P[0] + 1) == ALIGN and call(s=P[2] + 1) == ALIGN
        assert call(q=P[0]) == ALIAS and call(s=P[1]) == ALIAS


def product(lib, mats=1, x=P[0], sx=P[1], ldx=256, sxr=1, sxb=4, w=P[2], sw=P[3], ldw=256, swr=2, swb=1, up=P[4],
            su=P[5], out=P[6], ldo=256, os=None, lds=0, M=4, N=256, K=256, dtype=BF16, ws=P[8], n=1 << 20, plan=None):
    xm, wm = fp8.Matrix(x, sx, ldx, sxr, sxb), fp8.Matrix(w, sw, ldw, swr, swb)
    um = fp8.Matrix(up, su, ldw, swr, swb)
    r = ctypes.byref
    if plan is not None:
        return lib.glu_fp8_product_tuned(r(xm), r(wm), r(um) if mats == 2 else None, out, ldo, os, lds, M, N, K, dtype,
                                         r(plan), ws, n, None)
    if mats == 2:
        return lib.glu_fp8_dual_glu(r(xm), r(wm), r(um), out, ldo, os, lds, M, N, K, dtype, ws, n, None)
    return lib.glu_fp8_linear(r(xm), r(wm), out, ldo, os, lds, M, N, K, dtype, ws, n, None)


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=4), ARG), (dict(dtype=-1), ARG),
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=None, w=None, out=None), OK),
    (dict(x=None), NULLP), (dict(sx=None), NULLP), (dict(w=None), NULLP), (dict(sw=None), NULLP), (dict(out=None), NULLP),
    (dict(dtype=E4M3, os=None, lds=4), NULLP),
    (dict(ldx=255), STRIDE), (dict(ldw=0), STRIDE), (dict(ldo=255), STRIDE), (dict(swr=1), STRIDE), (dict(swb=2), STRIDE),
    (dict(sxr=-1), STRIDE), (dict(sxb=-4), STRIDE), (dict(sxr=1 << 62), STRIDE), (dict(dtype=E4M3, os=P[7], lds=3), STRIDE),
    (dict(sx=P[1] + 1), ALIGN), (dict(sw=P[3] + 2), ALIGN), (dict(out=P[6] + 1), ALIGN),
    (dict(out=P[0]), ALIAS), (dict(out=P[1]), ALIAS), (dict(out=P[2] + 1024), ALIAS), (dict(out=P[3]), ALIAS),
    (dict(dtype=E4M3, os=P[6], lds=4), ALIAS),
    (dict(dtype=E4M3, os=P[7], lds=4, ws=P[0]), ALIAS),
    (dict(dtype=E4M3, os=P[7], lds=4, ws=None), WORKSPACE), (dict(dtype=E4M3, os=P[7], lds=4, n=16), WORKSPACE),
    (dict(dtype=E4M3, os=P[7], lds=4, ws=P[8] + 8), WORKSPACE),
])
def test_product_refusals(lib, kw, status, mats):
    assert product(lib, mats, **kw) == status


def test_dual_refusals(lib):
    assert product(lib, 2, up=None) == NULLP and product(lib, 2, su=None) == NULLP
    assert product(lib, 2, out=P[4]) == ALIAS and product(lib, 2, out=P[5]) == ALIAS
    assert lib.glu_fp8_linear(None, None, P[0], 256, None, 0, 4, 256, 256, BF16, None, 0, None) == NULLP


@pytest.mark.parametrize("plan", [(0, 0, 0, 1), (5, 0, 0, 1), (3, -1, 0, 1), (3, 99, 0, 1), (3, 0, 0, 0), (3, 0, 0, 3),
                                  (2, 5, 4, 1), (2, 8, 4, 1), (2, 16, 0, 1), (2, 16, 9, 1), (2, 16, 4, -1), (2, 32, 4, 1), (4, 8, 4, 1)])
def test_unsupported_plans(lib, plan):
    assert product(lib, plan=fp8.ProductPlan(*plan)) == UNSUP


def test_unsupported_columns(lib):
    for columns in (-128, 100, 256, 384):
        assert product(lib, plan=fp8.ProductPlan(3, 1, 0, 1, 0, 0, columns)) == UNSUP
    assert product(lib, plan=fp8.ProductPlan(2, 16, 4, 1, 0, 0, 128)) == UNSUP


def test_layouts_that_are_not_fast_refuse_the_fast_kernels(lib):
    for kw in (dict(x=P[0] + 1), dict(ldx=264), dict(w=P[2] + 8), dict(K=250, ldw=256)):
        for kernel, tile in ((2, 16), (3, 1)):
            assert product(lib, plan=fp8.ProductPlan(kernel, tile, 4, 1), **kw) == UNSUP
    assert product(lib, plan=fp8.ProductPlan(2, 4, 4, 1), M=5, sxb=5) == UNSUP, "4 rows of weights serve 4 rows of x"


def test_plans_cover_every_size():
    """Every size gets a plan whose parts fit it; e4m3 output and split sums ask for the workspace they use."""
    import torch
    for mats in (1, 2):
        for M in (1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 203, 257, 1024, 1025, 4096, 8192, 70000):
            for N in (1, 100, 256, 2560, 17408, 100000):
                for K in (1, 16, 128, 144, 2560, 9216, 17408):
                    for t in (torch.bfloat16, fp8.E4M3):
                        for fast in (True, False):
                            p = fp8.product_plan(mats, M, N, K, t, fast)
                            blocks = -(-K // 128)
                            assert p["kernel_name"] in (("stream", "tile") if fast else ("any",))
                            assert 1 <= p["splits"] <= blocks
                            if p["columns"]:
                                assert fast and 0 < p["columns"] < N and p["columns"] % 128 == 0 and M > 16
                                assert 2 <= p["launches"] <= 4
                                continue
                            want = p["splits"] * mats * M * N * 4 if p["launches"] == 2 else 0
                            assert p["workspace_bytes"] == want and p["launches"] in (1, 2)
                            assert p["splits"] == 1 or p["launches"] == 2
    assert fp8.product_plan(1, 0, 5, 5)["kernel_name"] == "none"
    assert fp8.product_plan(1, 5, 5, 0)["kernel_name"] == "zero"


def test_few_rows_take_the_narrow_form_where_the_other_leaves_cus_idle():
    """3 or 4 rows of one matrix: 4 weight rows a workgroup where 16 would have work for two thirds of 256 CUs or less."""
    for K in (1024, 9216):
        for M in (1, 2, 3, 4, 5):
            for N in (16, 2560, 2561, 2720, 2721, 2816, 4096):
                p = fp8.product_plan(1, M, N, K)
                narrow = M <= 2 or M <= 4 and 3 * -(-N // 16) <= 512
                assert p["kernel_name"] == "tile" or p["tile"] == (4 if narrow else 16)
                assert p["kernel_name"] == "stream" or M > 2 and not narrow


def test_workspace_covers_either_layout(lib):
    import torch
    need = ctypes.c_int64()
    for mats in (1, 2):
        for M, N, K in ((1, 9216, 2560), (37, 12288, 4096), (203, 4096, 12288), (4096, 17408, 5120)):
            for t in (torch.bfloat16, fp8.E4M3):
                assert lib.glu_fp8_workspace(mats, M, N, K, fp8.DTYPES[t], ctypes.byref(need)) == OK
                for fast in (True, False):
                    assert need.value >= fp8.product_plan(mats, M, N, K, t, fast)["workspace_bytes"]
    assert lib.glu_fp8_workspace(3, 1, 1, 1, BF16, ctypes.byref(need)) == ARG
    assert lib.glu_fp8_workspace(1, 1, 1, 1, BF16, None) == NULLP
    assert lib.glu_fp8_product_plan(1, 1, 1, 1, BF16, 1, None) == NULLP


def test_copy_workspace(lib):
    def need(query, mats, M, N, K, dt=BF16):
        b = ctypes.c_int64(-1)
        return getattr(lib, query)(mats, M, N, K, dt, ctypes.byref(b)), b.value
    for mats in (1, 2):
        for M, N, K in ((17, 1, 1), (40, 300, 129), (300, 4096, 4100), (5000, 12288, 4096)):
            plan = fp8.ProductPlan()
            assert lib.glu_fp8_product_plan(mats, M, N, (K + 15) // 16 * 16, BF16, 1, ctypes.byref(plan)) == OK
            copies = (M + mats * N) * ((K + 15) // 16 * 16)
            assert need("glu_fp8_copy_workspace", mats, M, N, K) == (OK, (plan.workspace_bytes + 15) // 16 * 16 + copies)
    assert need("glu_fp8_copy_workspace", 1, 16, 300, 129) == (OK, 0)
    assert need("glu_fp8_copy_workspace", 1, 40, 300, 0) == (OK, 0)
    assert need("glu_fp8_copy_workspace", 3, 40, 300, 128)[0] == ARG
    assert need("glu_fp8_copy_workspace", 1, 40, 300, 128, 9)[0] == ARG
    assert need("glu_fp8_copy_workspace", 1, 40, -1, 128)[0] == SHAPE
    assert lib.glu_fp8_copy_workspace(1, 40, 300, 128, BF16, None) == NULLP
    # sizes whose workspace would not fit 63 bits
    assert need("glu_fp8_workspace", 2, 1 << 30, 1 << 30, 128)[0] == SHAPE


def test_copy_workspace_serves_a_call_in_place(lib):
    """Where copies do not pay a call of the same workspace is read in place."""
    b, plan = ctypes.c_int64(), fp8.ProductPlan()
    for mats in (1, 2):
        for M, N, K in ((17, 1, 1), (300, 4096, 100), (40, 5000, 17), (5000, 12288, 40)):
            for t in (BF16, E4M3):
                assert lib.glu_fp8_copy_workspace(mats, M, N, K, t, ctypes.byref(b)) == OK
                assert lib.glu_fp8_product_plan(mats, M, N, K, t, 0, ctypes.byref(plan)) == OK
                assert b.value >= plan.workspace_bytes and (t == BF16 or plan.workspace_bytes == mats * M * N * 4)


def test_no_copies_past_the_tile_kernels_strides(lib):
    """The tile kernel's row offsets are 32 bits wide: a row longer than the fast layout's longest stride is never
    copied for it, and a call from Python brings the workspace of the kernel that reads in place."""
    def need(query, *size):
        b = ctypes.c_int64(-1)
        return getattr(lib, query)(*size, ctypes.byref(b)), b.value
    longest = 1 << 23
    for mats in (1, 2):
        for t in (BF16, FP32, E4M3):
            assert need("glu_fp8_copy_workspace", mats, 17, 5, longest - 1, t)[1] >= (17 + mats * 5) * longest
            assert need("glu_fp8_copy_workspace", mats, 17, 5, longest, t)[1] >= (17 + mats * 5) * longest
            for M, N, K in ((17, 5, longest + 1), (17, 5, longest + 16), (40, 200, 1 << 26), (17, 32, 1 << 28),
                            (4096, 256, (1 << 24) + (1 << 18)), (17, 256, (1 << 25) + (1 << 20))):
                assert need("glu_fp8_copy_workspace", mats, M, N, K, t) == (OK, 0)
                plan = fp8.ProductPlan()
                assert lib.glu_fp8_product_plan(mats, M, N, K, t, 0, ctypes.byref(plan)) == OK
                assert fp8.KERNEL_NAMES[plan.kernel] == "any"
                assert fp8._product_workspace(mats, M, N, K, t, False) >= plan.workspace_bytes


def test_workspace_of_the_fast_layout(lib):
    """A prefill that ends in e4m3 by itself needs none on the fast layout."""
    need = ctypes.c_int64(-1)
    for mats, M, N, K, t in ((2, 4096, 17408, 5120, E4M3), (1, 203, 4096, 12288, BF16), (2, 1, 9216, 2560, E4M3)):
        plan = fp8.ProductPlan()
        assert lib.glu_fp8_product_plan(mats, M, N, K, t, 1, ctypes.byref(plan)) == OK
        assert lib.glu_fp8_product_workspace(mats, M, N, K, t, None, ctypes.byref(need)) == OK
        assert need.value == plan.workspace_bytes
        assert (need.value == 0) == (M == 4096)


def test_python_refuses_cpu_tensors():
    import torch

    import glu_mlp_gemv_amd as glu
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        glu.add_rms_norm(x, x[0], 1e-6)
    with pytest.raises(ValueError):
        glu.fp8_quantize(x)
    with pytest.raises(ValueError):
        glu.fp8_linear(x.to(fp8.E4M3), torch.ones(2, 1), x.to(fp8.E4M3), torch.ones(1, 1))
    with pytest.raises(TypeError):
        glu.add_rms_norm([1.0], x[0], 1e-6)


def test_forms_without_a_gradient_refuse_operands_that_require_one():
    import torch

    import glu_mlp_gemv_amd as glu
    for which in range(3):
        x, w, r = torch.zeros(2, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16), torch.zeros(2, 128).bfloat16()
        (x, w, r)[which].requires_grad_()
        for call in (lambda: glu.add_rms_norm_fp8(x, w, 1e-6, residual=r),
                     lambda: glu.add_rms_norm_fp8(x, w, 1e-6, residual=r, return_rstd=True),
                     lambda: glu.add_rms_norm(x, w, 1e-6, residual=r, out=torch.zeros_like(x)),
                     lambda: glu.add_rms_norm(x, w, 1e-6, residual=r, residual_out=torch.zeros_like(x)),
                     lambda: glu.add_rms_norm(x, w, 1e-6, residual=r, return_rstd=True)):
            with pytest.raises(RuntimeError, match="gradient"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # as far as a host goes
                call()


def test_mlp_refuses_inputs_that_require_a_gradient():
    import torch

    from glu_mlp_gemv_amd.mlp import Fp8GluMlp
    mlp = Fp8GluMlp.__new__(Fp8GluMlp)  # what __call__ reads before its first kernel
    mlp.eps, mlp.norm_weight = 1e-6, torch.ones(128, dtype=torch.bfloat16)
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for a, b in ((x.clone().requires_grad_(), None), (x, x.clone().requires_grad_())):
        with pytest.raises(RuntimeError, match="gradient"):
            mlp(a, b)


def test_host_calls_load_on_a_torch_without_a_gpu_backend():
    """The library and its planners are loaded where torch has no GPU backend's names."""
    import subprocess
    import sys
    code = ("import torch\nfor n in [n for n in dir(torch._C) if n.startswith('_cuda_') or n.startswith('_hip_')]: delattr(torch._C, n)\n"
            "from glu_mlp_gemv_amd import api, fp8\napi.library()\nprint(api.plan(1, 64, 64)['kernel'], fp8.product_plan(1, 1, 64, 64)['kernel'])")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=api.__file__.rsplit("/", 2)[0])
    assert res.returncode == 0, res.stderr


def test_the_library_is_built_without_the_binding(monkeypatch, tmp_path):
    """A torch binding that does not compile is an error, after the library has been linked."""
    from glu_mlp_gemv_amd import build

    def no_binding(verbose=False):
        raise RuntimeError("no torch headers")

    def link(cmd, check):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("library")
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIBRARY", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src + ".o")
    monkeypatch.setattr(build, "build_binding", no_binding)
    monkeypatch.setattr(build.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="torch headers"):
        build.build()
    assert (tmp_path / "lib.so").read_text() == "library"


def test_sanitizers_cover_every_c_entry():
    import os

    from glu_mlp_gemv_amd import build, sanitize
    for src in build.sources():
        with open(src) as f:
            if 'extern "C"' in f.read():
                assert os.path.basename(src) in sanitize.SAN_SOURCES
    assert "tests/" + os.path.basename(__file__) in sanitize.TESTS
