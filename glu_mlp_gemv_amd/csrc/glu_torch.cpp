// The short way from torch tensors to the C ABI, for the calls of fp8.py, adapters.py, moe.py and counter_dropout.py in
// their usual form: every operand of
// the expected type, shape and layout on the current device, outputs to be allocated, the current
// stream.  Checking, allocating and calling take 1.5 to 2 us here against 8 in Python, which shows where a kernel
// takes 3 us.  Whatever is not in that form returns None before anything is allocated, and the Python takes the call
// and says what is wrong. A status other than GLU_OK is returned as an int.
#include <Python.h>

#include <stdint.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/glu_adapter.h"
#include "../../include/glu_dropout.h"
#include "../../include/glu_fp8.h"
#include "../../include/glu_moe.h"

namespace {

// the library that fp8.py has loaded
struct Api {
    decltype(&glu_add_rms_norm) norm;
    decltype(&glu_add_rms_norm_fp8) norm_fp8;
    decltype(&glu_add_rms_norm_backward) norm_grad;
    decltype(&glu_add_rms_norm_backward_workspace) norm_grad_workspace;
    decltype(&glu_fp8_quantize) quantize;
    decltype(&glu_fp8_quantize_weight) quantize_weight;
    decltype(&glu_fp8_linear) linear;
    decltype(&glu_fp8_dual_glu) dual_glu;
    decltype(&glu_fp8_workspace) workspace;
    decltype(&glu_fp8_product_workspace) fast_workspace;
    decltype(&glu_adapter_add) adapter_add;
    decltype(&glu_adapter_glu) adapter_glu;
    decltype(&glu_adapter_workspace) adapter_workspace;
    decltype(&glu_adapter_backward) adapter_backward;
    decltype(&glu_adapter_backward_workspace) adapter_backward_workspace;
    decltype(&glu_moe_glu) moe;
    decltype(&glu_moe_workspace) moe_workspace;
    decltype(&glu_dropout) dropout;
};
Api api;

constexpr auto kE4m3 = c10::ScalarType::Float8_e4m3fn;

int64_t groups(int64_t n) { return (n + 127) / 128; }

int dtype_code(c10::ScalarType t)
{
    switch (t) {
    case c10::ScalarType::BFloat16: return GLU_DTYPE_BF16;
    case c10::ScalarType::Half: return GLU_DTYPE_FP16;
    case c10::ScalarType::Float: return GLU_DTYPE_FP32;
    case kE4m3: return GLU_DTYPE_E4M3;
    default: return -1;
    }
}

// What a call's operands have to agree on, taken from its first
struct Place {
    c10::Device device{c10::DeviceType::CPU};
    bool ok = false;
    void* stream = nullptr;
    explicit Place(PyObject* first)
    {
        if (!THPVariable_Check(first)) return;
        device = THPVariable_Unpack(first).device();
        if (!device.is_cuda() || device.index() != c10::hip::current_device()) return;
        ok = true;
        stream = (void*)c10::hip::getCurrentHIPStream(device.index()).stream();
    }
    // torch's own allocation on the device, without the dispatcher on the way
    at::Tensor empty(int64_t rows, int64_t cols, int64_t row_stride, int64_t col_stride, c10::ScalarType t) const
    {
        return at::detail::empty_strided_cuda({rows, cols}, {row_stride, col_stride}, t, device);
    }
    at::Tensor empty(int64_t n, int64_t rows, int64_t cols, c10::ScalarType t) const
    {
        return at::detail::empty_strided_cuda({n, rows, cols}, {rows * cols, cols, 1}, t, device);
    }
    at::Tensor empty(int64_t n, c10::ScalarType t) const { return at::detail::empty_strided_cuda({n}, {1}, t, device); }
    at::Tensor workspace(int64_t bytes) const
    {
        return bytes ? empty(bytes / 4, c10::ScalarType::Float) : at::Tensor();
    }
};

// [rows, cols] of type t with contiguous rows that do not overlap; rows or cols < 0: any (returned)
struct Rows {
    bool ok = false;
    int64_t rows = 0, cols = 0, ld = 0;
    void* p = nullptr;
    c10::ScalarType type = c10::ScalarType::Undefined;
    Rows(PyObject* o, const Place& at, int64_t want_rows, int64_t want_cols, c10::ScalarType want)
    {
        if (!THPVariable_Check(o)) return;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != c10::kStrided || t.dim() != 2 || t.device() != at.device) return;
        type = t.scalar_type();
        rows = t.size(0);
        cols = t.size(1);
        if (rows < 1 || cols < 1) return;  // empty calls are for the long way
        if (want != c10::ScalarType::Undefined && type != want) return;
        if ((want_rows >= 0 && rows != want_rows) || (want_cols >= 0 && cols != want_cols)) return;
        if (cols > 1 && t.stride(1) != 1) return;
        ld = rows > 1 ? t.stride(0) : cols;
        p = t.data_ptr();
        ok = ld >= cols;
    }
};

void* vector(PyObject* o, const Place& at, int64_t n, c10::ScalarType want)
{
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != c10::kStrided || t.dim() != 1 || t.device() != at.device || t.scalar_type() != want ||
        t.size(0) != n || (n > 1 && t.stride(0) != 1)) {
        return nullptr;
    }
    return t.data_ptr();
}

PyObject* pack(int n, const at::Tensor* t)
{
    PyObject* out = PyTuple_New(n);
    for (int i = 0; out && i < n; ++i) PyTuple_SET_ITEM(out, i, THPVariable_Wrap(t[i]));
    return out;
}

PyObject* status_int(glu_status st) { return PyLong_FromLong(st); }

// torch's allocator and checks throw: out of memory and the like become Python's exceptions here
template <class F>
PyObject* guarded(F&& f)
{
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// Whether autograd follows any of these: they require a gradient where it records, or carry a tangent of forward mode,
// which no_grad does not switch off
bool recorded(PyObject* const* a, Py_ssize_t n)
{
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPVariable_Check(a[i])) continue;
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if ((t.requires_grad() && c10::GradMode::is_enabled()) || t._fw_grad(0).defined()) return true;
    }
    return false;
}

// (x, weight, eps, residual or None, e4m3) -> (out, h or None[, scale])
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 5) Py_RETURN_NONE;
        const Place at(a[0]);
        if (!at.ok) Py_RETURN_NONE;
        const Rows x(a[0], at, -1, -1, c10::ScalarType::Undefined);
        const int dt = x.ok ? dtype_code(x.type) : -1;
        if (dt < 0 || dt == GLU_DTYPE_E4M3) Py_RETURN_NONE;
        void* w = vector(a[1], at, x.cols, x.type);
        const double eps = PyFloat_Check(a[2]) ? PyFloat_AS_DOUBLE(a[2]) : -1.0;
        if (!w || eps < 0.0) Py_RETURN_NONE;
        const bool has = a[3] != Py_None, e4m3 = a[4] == Py_True;
        if (recorded(a, 4)) Py_RETURN_NONE;  // fp8.py has them differentiated, or refuses
        void* res = nullptr;
        int64_t ldr = 0;
        if (has) {
            const Rows r(a[3], at, x.rows, x.cols, x.type);
            if (!r.ok) Py_RETURN_NONE;
            res = r.p;
            ldr = r.ld;
        }
        at::Tensor t[3];
        t[0] = at.empty(x.rows, x.cols, x.cols, 1, e4m3 ? kE4m3 : x.type);
        if (has) t[1] = at.empty(x.rows, x.cols, x.cols, 1, x.type);
        void* sum = has ? t[1].data_ptr() : nullptr;
        glu_status st;
        if (e4m3) {
            t[2] = at.empty(x.rows, groups(x.cols), 1, x.rows, c10::ScalarType::Float);
            st = api.norm_fp8(x.p, x.ld, res, ldr, w, sum, x.cols, (uint8_t*)t[0].data_ptr(), x.cols,
                              (float*)t[2].data_ptr(), x.rows, nullptr, x.rows, x.cols, (float)eps, dt, at.stream);
        } else {
            st = api.norm(x.p, x.ld, res, ldr, w, sum, x.cols, t[0].data_ptr(), x.cols, nullptr, x.rows, x.cols,
                          (float)eps, dt, at.stream);
        }
        return st == GLU_OK ? pack(e4m3 ? 3 : 2, t) : status_int(st);
    });
}

// (dy, h, weight, rstd, dresidual or None) -> (dx, dweight)
PyObject* norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 5) Py_RETURN_NONE;
        const Place at(a[0]);
        if (!at.ok) Py_RETURN_NONE;
        const Rows h(a[1], at, -1, -1, c10::ScalarType::Undefined);
        const int dt = h.ok ? dtype_code(h.type) : -1;
        if (dt < 0 || dt == GLU_DTYPE_E4M3) Py_RETURN_NONE;
        const Rows dy(a[0], at, h.rows, h.cols, h.type);
        void* w = vector(a[2], at, h.cols, h.type);
        void* rstd = vector(a[3], at, h.rows, c10::ScalarType::Float);
        if (!dy.ok || !w || !rstd) Py_RETURN_NONE;
        void* dres = nullptr;
        int64_t ldr = 0, bytes = 0;
        if (a[4] != Py_None) {
            const Rows r(a[4], at, h.rows, h.cols, h.type);
            if (!r.ok) Py_RETURN_NONE;
            dres = r.p;
            ldr = r.ld;
        }
        glu_status st = api.norm_grad_workspace(h.rows, h.cols, &bytes);
        if (st != GLU_OK) return status_int(st);
        const at::Tensor t[2] = {at.empty(h.rows, h.cols, h.cols, 1, h.type), at.empty(h.cols, h.type)};
        const at::Tensor ws = at.workspace(bytes);
        st = api.norm_grad(dy.p, dy.ld, h.p, h.ld, w, (const float*)rstd, dres, ldr, t[0].data_ptr(), h.cols,
                           t[1].data_ptr(), h.rows, h.cols, dt, bytes ? ws.data_ptr() : nullptr, bytes, at.stream);
        return st == GLU_OK ? pack(2, t) : status_int(st);
    });
}

// (x, blocks) -> (q, scale)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 2) Py_RETURN_NONE;
        const Place at(a[0]);
        if (!at.ok) Py_RETURN_NONE;
        const Rows x(a[0], at, -1, -1, c10::ScalarType::Undefined);
        const int dt = x.ok ? dtype_code(x.type) : -1;
        if (dt < 0 || dt == GLU_DTYPE_E4M3) Py_RETURN_NONE;
        const bool blocks = a[1] == Py_True;
        const int64_t G = groups(x.cols);
        const at::Tensor t[2] = {at.empty(x.rows, x.cols, x.cols, 1, kE4m3),
                                 blocks ? at.empty(groups(x.rows), G, G, 1, c10::ScalarType::Float)
                                        : at.empty(x.rows, G, 1, x.rows, c10::ScalarType::Float)};
        const glu_status st = (blocks ? api.quantize_weight : api.quantize)(
            x.p, x.ld, (uint8_t*)t[0].data_ptr(), x.cols, (float*)t[1].data_ptr(), blocks ? G : x.rows, x.rows, x.cols,
            dt, at.stream);
        return st == GLU_OK ? pack(2, t) : status_int(st);
    });
}

// (dtype code, x, x_scale, weight, weight_scale[, up, up_scale]) -> (out[, scale])
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 5 && n != 7) Py_RETURN_NONE;
        const Place at(a[1]);
        if (!at.ok) Py_RETURN_NONE;
        const int mats = n == 7 ? 2 : 1;
        const long dt = PyLong_AsLong(a[0]);
        const c10::ScalarType types[4] = {c10::ScalarType::BFloat16, c10::ScalarType::Half, c10::ScalarType::Float,
                                          kE4m3};
        if (dt < 0 || dt > 3) Py_RETURN_NONE;
        const Rows x(a[1], at, -1, -1, kE4m3);
        if (!x.ok || !THPVariable_Check(a[2])) Py_RETURN_NONE;
        const at::Tensor& sx = THPVariable_Unpack(a[2]);
        const int64_t M = x.rows, K = x.cols, G = groups(K);
        if (sx.layout() != c10::kStrided || sx.dim() != 2 || sx.device() != at.device ||
            sx.scalar_type() != c10::ScalarType::Float || sx.size(0) != M || sx.size(1) != G) {
            Py_RETURN_NONE;
        }
        const glu_fp8_matrix xm{(const uint8_t*)x.p, (const float*)sx.data_ptr(), x.ld, sx.stride(0), sx.stride(1)};
        glu_fp8_matrix wm[2];
        int64_t N = -1;
        for (int i = 0; i < mats; ++i) {
            const Rows w(a[3 + 2 * i], at, N, K, kE4m3);
            if (!w.ok) Py_RETURN_NONE;
            N = w.rows;
            const Rows s(a[4 + 2 * i], at, groups(N), G, c10::ScalarType::Float);
            if (!s.ok) Py_RETURN_NONE;
            wm[i] = glu_fp8_matrix{(const uint8_t*)w.p, (const float*)s.p, w.ld, s.ld, 1};
        }
        // a layout that the library copies first takes another workspace
        uintptr_t bits = (uintptr_t)K | (uintptr_t)x.p | (uintptr_t)x.ld;
        int64_t widest = x.ld;
        for (int i = 0; i < mats; ++i) {
            bits |= (uintptr_t)wm[i].data | (uintptr_t)wm[i].ld;
            if (wm[i].ld > widest) widest = wm[i].ld;
        }
        const bool fast = (bits & 15) == 0 && widest <= 1 << 23;
        if (M > 16 && !fast) Py_RETURN_NONE;
        int64_t bytes = 0;
        glu_status st = fast ? api.fast_workspace(mats, M, N, K, (int)dt, nullptr, &bytes)
                             : api.workspace(mats, M, N, K, (int)dt, &bytes);
        if (st != GLU_OK) return status_int(st);
        const bool e4m3 = dt == GLU_DTYPE_E4M3;
        at::Tensor t[2];
        t[0] = at.empty(M, N, N, 1, types[dt]);
        if (e4m3) t[1] = at.empty(M, groups(N), 1, M, c10::ScalarType::Float);
        const at::Tensor ws = at.workspace(bytes);
        float* scale = e4m3 ? (float*)t[1].data_ptr() : nullptr;
        void* wsp = bytes ? ws.data_ptr() : nullptr;
        st = mats == 2 ? api.dual_glu(&xm, &wm[0], &wm[1], t[0].data_ptr(), N, scale, M, M, N, K, (int)dt, wsp, bytes,
                                      at.stream)
                       : api.linear(&xm, &wm[0], t[0].data_ptr(), N, scale, M, M, N, K, (int)dt, wsp, bytes, at.stream);
        return st == GLU_OK ? pack(e4m3 ? 2 : 1, t) : status_int(st);
    });
}

// [n, rows, cols] of type t with contiguous rows; rows and matrices do not overlap
struct Matrices {
    bool ok = false;
    int64_t n = 0, rows = 0, cols = 0, stack = 0, ld = 0;
    void* p = nullptr;
    c10::ScalarType type = c10::ScalarType::Undefined;
    Matrices(PyObject* o, const Place& at, int64_t want_n, int64_t want_rows, int64_t want_cols)
    {
        if (!THPVariable_Check(o)) return;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != c10::kStrided || t.dim() != 3 || t.device() != at.device) return;
        type = t.scalar_type();
        n = t.size(0);
        rows = t.size(1);
        cols = t.size(2);
        if (n < 1 || rows < 1 || cols < 1) return;
        if ((want_n >= 0 && n != want_n) || (want_rows >= 0 && rows != want_rows) || (want_cols >= 0 && cols != want_cols)) return;
        if (cols > 1 && t.stride(2) != 1) return;
        ld = rows > 1 ? t.stride(1) : cols;
        stack = n > 1 ? t.stride(0) : rows * ld;
        p = t.data_ptr();
        ok = ld >= cols && stack >= (rows - 1) * ld + cols;
    }
};

bool half_type(c10::ScalarType t) { return t == c10::ScalarType::BFloat16 || t == c10::ScalarType::Half; }

// an optional vector: false where it is there and not as wanted
bool optional_vector(PyObject* o, const Place& at, int64_t n, c10::ScalarType want, void** p)
{
    *p = nullptr;
    return o == Py_None || (*p = vector(o, at, n, want)) != nullptr;
}

// (y, x, a, b, index, scale or None) or (gate, up, x, gate_a, gate_b, up_a, up_b, index, scale or None) -> out
PyObject* adapter(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 6 && n != 9) Py_RETURN_NONE;
        const int mats = n == 9 ? 2 : 1;
        const Place at(a[0]);
        if (!at.ok || recorded(a, n)) Py_RETURN_NONE;
        const Rows y(a[0], at, -1, -1, c10::ScalarType::Undefined);
        if (!y.ok || !half_type(y.type)) Py_RETURN_NONE;
        const Rows y2(a[mats - 1], at, y.rows, y.cols, y.type), x(a[mats], at, y.rows, -1, y.type);
        if (!y2.ok || !x.ok) Py_RETURN_NONE;
        glu_adapter ab[2];
        int64_t L = -1, R = -1;
        for (int i = 0; i < mats; ++i) {
            const Matrices wa(a[mats + 1 + 2 * i], at, L, R, x.cols);
            if (!wa.ok || wa.type != y.type) Py_RETURN_NONE;
            L = wa.n;
            R = wa.rows;
            const Matrices wb(a[mats + 2 + 2 * i], at, L, y.cols, R);
            if (!wb.ok || wb.type != y.type || R > GLU_ADAPTER_MAX_RANK) Py_RETURN_NONE;
            ab[i] = glu_adapter{wa.p, wb.p, wa.stack, wa.ld, wb.stack, wb.ld};
        }
        void *index = vector(a[n - 2], at, y.rows, c10::ScalarType::Int), *scale;
        if (!index || !optional_vector(a[n - 1], at, L, c10::ScalarType::Float, &scale)) Py_RETURN_NONE;
        const glu_adapter_sizes sizes{y.rows, y.cols, x.cols, R, L};
        int64_t bytes = 0;
        glu_status st = api.adapter_workspace(mats, &sizes, &bytes);
        if (st != GLU_OK) return status_int(st);
        const at::Tensor out = at.empty(y.rows, y.cols, y.cols, 1, y.type), ws = at.workspace(bytes);
        void* wsp = bytes ? ws.data_ptr() : nullptr;
        const int dt = dtype_code(y.type);
        st = mats == 2 ? api.adapter_glu(y.p, y.ld, y2.p, y2.ld, x.p, x.ld, &ab[0], &ab[1], (const int32_t*)index,
                                         (const float*)scale, out.data_ptr(), y.cols, &sizes, dt, wsp, bytes, at.stream)
                       : api.adapter_add(y.p, y.ld, x.p, x.ld, &ab[0], (const int32_t*)index, (const float*)scale,
                                         out.data_ptr(), y.cols, nullptr, &sizes, dt, wsp, bytes, at.stream);
        return st == GLU_OK ? THPVariable_Wrap(out) : status_int(st);
    });
}

// (dout, x, a, b, index, low, scale or None) -> (dx, da, db)
PyObject* adapter_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 7) Py_RETURN_NONE;
        const Place at(a[0]);
        if (!at.ok) Py_RETURN_NONE;
        const Rows d(a[0], at, -1, -1, c10::ScalarType::Undefined);
        if (!d.ok || !half_type(d.type)) Py_RETURN_NONE;
        const Rows x(a[1], at, d.rows, -1, d.type);
        if (!x.ok) Py_RETURN_NONE;
        const Matrices wa(a[2], at, -1, -1, x.cols);
        if (!wa.ok || wa.type != d.type) Py_RETURN_NONE;
        const int64_t L = wa.n, R = wa.rows;
        const Matrices wb(a[3], at, L, d.cols, R);
        if (!wb.ok || wb.type != d.type || R > GLU_ADAPTER_MAX_RANK) Py_RETURN_NONE;
        const Rows low(a[5], at, d.rows, R, c10::ScalarType::Float);
        void *index = vector(a[4], at, d.rows, c10::ScalarType::Int), *scale;
        if (!index || !low.ok || low.ld != R || !optional_vector(a[6], at, L, c10::ScalarType::Float, &scale)) Py_RETURN_NONE;
        const glu_adapter_sizes sizes{d.rows, d.cols, x.cols, R, L};
        int64_t bytes = 0;
        glu_status st = api.adapter_backward_workspace(&sizes, &bytes);
        if (st != GLU_OK) return status_int(st);
        const at::Tensor t[3] = {at.empty(d.rows, x.cols, x.cols, 1, d.type), at.empty(L, R, x.cols, d.type),
                                 at.empty(L, d.cols, R, d.type)};
        const at::Tensor ws = at.workspace(bytes);
        const glu_adapter ab{wa.p, wb.p, wa.stack, wa.ld, wb.stack, wb.ld};
        st = api.adapter_backward(d.p, d.ld, x.p, x.ld, &ab, (const int32_t*)index, (const float*)scale, (const float*)low.p,
                                  t[0].data_ptr(), x.cols, t[1].data_ptr(), t[2].data_ptr(), &sizes, dtype_code(d.type),
                                  bytes ? ws.data_ptr() : nullptr, bytes, at.stream);
        return st == GLU_OK ? pack(3, t) : status_int(st);
    });
}

// (x, logits, gate, up, down, top, normalize, gate_scale, up_scale, down_scale: three or None) -> out
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 10) Py_RETURN_NONE;
        const Place at(a[0]);
        if (!at.ok || recorded(a, n)) Py_RETURN_NONE;
        const Rows x(a[0], at, -1, -1, c10::ScalarType::Undefined);
        if (!x.ok || !half_type(x.type) || !PyLong_Check(a[5])) Py_RETURN_NONE;
        const Rows logits(a[1], at, x.rows, -1, c10::ScalarType::Undefined);
        if (!logits.ok || (logits.type != x.type && logits.type != c10::ScalarType::Float)) Py_RETURN_NONE;
        const int64_t E = logits.cols, K = x.cols;
        const long top = PyLong_AsLong(a[5]);
        if (top < 1 || top > E || top > GLU_MOE_MAX_TOP || E > GLU_MOE_MAX_EXPERTS) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        glu_expert_matrix w[3];
        c10::ScalarType wt = c10::ScalarType::Undefined;
        int64_t N = -1;
        for (int i = 0; i < 3; ++i) {
            const Matrices m(a[2 + i], at, E, i < 2 ? N : K, i < 2 ? K : N);
            if (!m.ok || (i && m.type != wt) || (m.type != x.type && m.type != kE4m3)) Py_RETURN_NONE;
            wt = m.type;
            if (i == 0) N = m.rows;
            w[i] = glu_expert_matrix{m.p, nullptr, m.stack, m.ld, 0, 0};
            if (wt != kE4m3) {
                if (a[7 + i] != Py_None) Py_RETURN_NONE;
                continue;
            }
            const Matrices s(a[7 + i], at, E, groups(m.rows), groups(m.cols));
            if (!s.ok || s.type != c10::ScalarType::Float) Py_RETURN_NONE;
            w[i].scale = (const float*)s.p;
            w[i].scale_stack = s.stack;
            w[i].scale_ld = s.ld;
        }
        const glu_moe_sizes sizes{x.rows, K, N, E, top};
        int64_t bytes = 0;
        glu_status st = api.moe_workspace(&sizes, &bytes);
        if (st != GLU_OK) return status_int(st);
        const at::Tensor out = at.empty(x.rows, K, K, 1, x.type), ws = at.workspace(bytes);
        st = api.moe(x.p, x.ld, logits.p, logits.ld, dtype_code(logits.type), &w[0], &w[1], &w[2], out.data_ptr(), K, &sizes,
                     a[6] == Py_True, dtype_code(x.type), dtype_code(wt), bytes ? ws.data_ptr() : nullptr, bytes, at.stream);
        return st == GLU_OK ? THPVariable_Wrap(out) : status_int(st);
    });
}

// (x, drop of 65536, seed below 2^64 or tensor, offset below 2^64, residual or None) -> out
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 5 || !PyLong_Check(a[1]) || !PyLong_Check(a[3])) Py_RETURN_NONE;
        const Place at(a[0]);
        if (!at.ok || recorded(a, 1) || recorded(a + 4, 1)) Py_RETURN_NONE;
        const Rows x(a[0], at, -1, -1, c10::ScalarType::Undefined);
        const int dt = x.ok ? dtype_code(x.type) : -1;
        if (dt < 0 || dt == GLU_DTYPE_E4M3) Py_RETURN_NONE;
        void *seed_at = nullptr, *res = nullptr;
        uint64_t seed = 0;
        if (PyLong_Check(a[2])) seed = PyLong_AsUnsignedLongLongMask(a[2]);
        else if (!(seed_at = vector(a[2], at, 1, c10::ScalarType::Long))) Py_RETURN_NONE;
        int64_t ldr = 0;
        if (a[4] != Py_None) {
            const Rows r(a[4], at, x.rows, x.cols, x.type);
            if (!r.ok) Py_RETURN_NONE;
            res = r.p;
            ldr = r.ld;
        }
        const at::Tensor out = at.empty(x.rows, x.cols, x.cols, 1, x.type);
        const glu_status st = api.dropout(x.p, x.ld, res, ldr, out.data_ptr(), x.cols, x.rows, x.cols, PyLong_AsLong(a[1]), seed,
                                          (const uint64_t*)seed_at, PyLong_AsUnsignedLongLongMask(a[3]), dt, at.stream);
        return st == GLU_OK ? THPVariable_Wrap(out) : status_int(st);
    });
}

// the addresses of the C functions, in the order of Api
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    constexpr Py_ssize_t count = sizeof(Api) / sizeof(void*);
    void* f[count];
    if (n != count) {
        PyErr_SetString(PyExc_TypeError, "one address per function");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < count; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL address");
            return nullptr;
        }
    }
    static_assert(sizeof(f) == sizeof(api), "function pointers only");
    __builtin_memcpy(&api, f, sizeof(f));
    Py_RETURN_NONE;
}

#define GLU_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GLU_METHOD(norm),    GLU_METHOD(norm_grad), GLU_METHOD(quantize),
                         GLU_METHOD(product), GLU_METHOD(adapter), GLU_METHOD(adapter_grad), GLU_METHOD(moe),
                         GLU_METHOD(dropout), GLU_METHOD(bind),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) { return PyModule_Create(&module); }
