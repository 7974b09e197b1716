// C ABI of the low-rank adapters (include/glu_adapter.h): argument validation, workspace and launches.  Validation
// happens before any HIP call; nothing is allocated or cached.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/glu_adapter.h"
#include "glu_adapter.h"
#include "glu_check.h"
#include "glu_status.h"

namespace {

using glu::Array;
using glu::bad_dim;
using glu::check_arrays;

constexpr int64_t kMaxGradRows = 1 << 24, kMaxGradAdapters = 1 << 16;

glu_status launched(hipError_t e) { return e == hipSuccess ? GLU_OK : glu::fail_launch(e); }

glu_status check_sizes(const glu_adapter_sizes* s)
{
    if (!s) return GLU_ERR_NULL_POINTER;
    if (bad_dim(s->M) || bad_dim(s->N) || bad_dim(s->K) || bad_dim(s->L) || s->L == 0) return GLU_ERR_BAD_SHAPE;
    if (s->N > glu::kMaxAdapterRow || s->K > glu::kMaxAdapterRow) return GLU_ERR_BAD_SHAPE;
    if (s->R < 1 || s->R > GLU_ADAPTER_MAX_RANK) return GLU_ERR_BAD_SHAPE;
    return GLU_OK;
}

glu_status check_grad_sizes(const glu_adapter_sizes* s)
{
    const glu_status st = check_sizes(s);
    if (st != GLU_OK) return st;
    return s->M > kMaxGradRows || s->L > kMaxGradAdapters ? GLU_ERR_BAD_SHAPE : GLU_OK;
}

// whether a row stride that is used is past what a tile's offsets hold
bool too_wide(int64_t rows, int64_t ld) { return rows > 1 && ld > glu::kMaxAdapterRow; }

// L matrices of `rows` rows of `len` elements as one array: rows and matrices may lie apart, but not overlap
glu_status stack_array(const void* p, int64_t L, int64_t rows, int64_t len, int64_t stack, int64_t row, Array* out)
{
    *out = Array{p, 0, 0, 0, 2, false};
    if (rows == 0 || len == 0) return GLU_OK;
    const Array one{p, rows, len, row, 2, false};
    if ((rows > 1 && row < len) || too_wide(rows, row)) return GLU_ERR_BAD_STRIDE;
    const int64_t bytes = glu::extent(one);
    if (bytes < 0) return GLU_ERR_BAD_STRIDE;
    *out = Array{p, L, bytes / 2, stack, 2, false};
    return GLU_OK;
}

glu_status stack_arrays(const glu_adapter* ab, const glu_adapter_sizes& s, Array* out)
{
    const glu_status st = stack_array(ab->a, s.L, s.R, s.K, ab->a_stack, ab->a_row, out);
    return st != GLU_OK ? st : stack_array(ab->b, s.L, s.N, s.R, ab->b_stack, ab->b_row, out + 1);
}

int64_t align16(int64_t n) { return (n + 15) & ~(int64_t)15; }

int low_splits(int mats, const glu_adapter_sizes& s, int64_t columns, bool down = false)
{
    return glu::adapter_low_splits((int)s.M, (int)columns, (int)s.R, (int)s.L, mats, down);
}

// t of every row, in its parts
int64_t low_bytes(int mats, const glu_adapter_sizes& s, int64_t columns)
{
    return align16((int64_t)low_splits(mats, s, columns) * mats * s.M * s.R * 4);
}

bool bad_workspace(const void* p, int64_t given, int64_t need)
{
    return need > 0 && (!p || ((uintptr_t)p & 15) || given < need);
}

glu_status apply(int mats, const void* const* y, const int64_t* ldy, const void* x, int64_t ldx,
                 const glu_adapter* const* ab, const int32_t* index, const float* scale, void* out, int64_t ldo,
                 float* low, const glu_adapter_sizes* sizes, int dtype, void* workspace, int64_t workspace_bytes,
                 void* stream)
{
    if (dtype != GLU_DTYPE_BF16 && dtype != GLU_DTYPE_FP16) return GLU_ERR_BAD_ARGUMENT;
    glu_status st = check_sizes(sizes);
    if (st != GLU_OK) return st;
    const glu_adapter_sizes s = *sizes;
    if (s.M == 0 || (s.N == 0 && !low)) return GLU_OK;
    for (int i = 0; i < mats; ++i) {
        if (!ab[i]) return GLU_ERR_NULL_POINTER;
    }
    if (too_wide(s.M, ldx) || too_wide(s.M, ldo) || too_wide(s.M, ldy[0]) || (mats == 2 && too_wide(s.M, ldy[1]))) {
        return GLU_ERR_BAD_STRIDE;
    }
    const int64_t need = low_bytes(mats, s, s.K);
    Array arrays[12];
    int n = 0;
    arrays[n++] = {y[0], s.M, s.N, ldy[0], 2, false};
    if (mats == 2) arrays[n++] = {y[1], s.M, s.N, ldy[1], 2, false};
    arrays[n++] = {out, s.M, s.N, ldo, 2, true};
    const unsigned shared_out = 1u << mats, shared_in = mats == 2 ? 3u : 1u;
    arrays[n++] = {x, s.M, s.K, ldx, 2, false};
    for (int i = 0; i < mats; ++i, n += 2) {
        st = stack_arrays(ab[i], s, arrays + n);
        if (st != GLU_OK) return st;
    }
    arrays[n++] = {index, 1, s.M, s.M, 4, false};
    arrays[n++] = {scale, scale ? 1 : 0, s.L, s.L, 4, false};
    arrays[n++] = {low, low ? s.M : 0, s.R, s.R, 4, true};
    if (bad_workspace(workspace, workspace_bytes, need)) {
        st = check_arrays(arrays, n, shared_out, shared_in);
        return st != GLU_OK ? st : GLU_ERR_WORKSPACE;
    }
    arrays[n++] = {workspace, 1, need, need, 1, true};
    st = check_arrays(arrays, n, shared_out, shared_in);
    if (st != GLU_OK) return st;

    glu::LowArgs la{};
    glu::OutArgs oa{};
    for (int i = 0; i < mats; ++i) {
        la.w[i] = {ab[i]->a, ab[i]->a_stack, ab[i]->a_row};
        oa.w[i] = {ab[i]->b, ab[i]->b_stack, ab[i]->b_row};
        oa.y[i] = y[i];
        oa.ldy[i] = ldy[i];
    }
    la.v = x;
    la.ldv = ldx;
    la.index = oa.index = index;
    la.splits = oa.splits = low_splits(mats, s, s.K);
    const bool straight = low && la.splits == 1;  // one part of t is t
    la.z = straight ? low : (float*)workspace;
    oa.z = la.z;
    oa.low = straight ? nullptr : low;
    la.M = oa.M = (int)s.M;
    la.C = (int)s.K;
    la.R = oa.R = (int)s.R;
    la.L = oa.L = (int)s.L;
    la.mats = oa.mats = mats;
    oa.scale = scale;
    oa.out = out;
    oa.ldo = ldo;
    oa.N = (int)s.N;
    const hipError_t e = glu::adapter_low_launch(dtype, false, la, (hipStream_t)stream);
    if (e != hipSuccess || (s.N == 0 && !oa.low)) return launched(e);
    return launched(glu::adapter_out_launch(dtype, false, oa, (hipStream_t)stream));
}

// The backward's workspace: d in its parts and, where there are several, their sum, the rows' order, the items, b turned, the
// items' sums.
struct GradPlan {
    bool direct;
    int splits, rows;
    int64_t items, sum, order, table, turned, pitch, part, bytes;  // offsets; turned: rows of `pitch`
};
GradPlan grad_plan(const glu_adapter_sizes& s)
{
    GradPlan p{};
    p.rows = glu::adapter_grad_rows((int)s.M, s.K + s.N);
    p.direct = glu::adapter_grad_direct((int)s.M, p.rows);
    p.splits = low_splits(1, s, s.N, p.direct);
    p.sum = align16(p.splits * s.M * s.R * 4);
    p.order = p.sum + (p.splits > 1 ? align16(s.M * s.R * 4) : 0);
    p.bytes = p.order;
    if (!p.direct) {
        p.items = glu::adapter_grad_items((int)s.M, (int)s.L, p.rows);
        p.table = p.order + align16(s.M * 4);
        p.turned = p.table + align16(p.items * 16 + s.L * 8);
        p.pitch = (s.N + 7) / 8 * 8;
        p.part = p.turned + align16(s.L * s.R * p.pitch * 2);
        p.bytes = p.part + p.items * s.R * (s.K + s.N) * 4;
    }
    return p;
}

}  // namespace

extern "C" {

glu_status glu_adapter_add(const void* y, int64_t ldy, const void* x, int64_t ldx, const glu_adapter* ab,
                           const int32_t* index, const float* scale, void* out, int64_t ldo, float* low,
                           const glu_adapter_sizes* sizes, int dtype, void* workspace, int64_t workspace_bytes,
                           void* stream)
{
    return apply(1, &y, &ldy, x, ldx, &ab, index, scale, out, ldo, low, sizes, dtype, workspace, workspace_bytes, stream);
}

glu_status glu_adapter_glu(const void* gate, int64_t ldg, const void* up, int64_t ldu, const void* x, int64_t ldx,
                           const glu_adapter* gate_ab, const glu_adapter* up_ab, const int32_t* index,
                           const float* scale, void* out, int64_t ldo, const glu_adapter_sizes* sizes, int dtype,
                           void* workspace, int64_t workspace_bytes, void* stream)
{
    const void* y[2] = {gate, up};
    const int64_t ldy[2] = {ldg, ldu};
    const glu_adapter* ab[2] = {gate_ab, up_ab};
    return apply(2, y, ldy, x, ldx, ab, index, scale, out, ldo, nullptr, sizes, dtype, workspace, workspace_bytes, stream);
}

glu_status glu_adapter_workspace(int mats, const glu_adapter_sizes* sizes, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    if (mats != 1 && mats != 2) return GLU_ERR_BAD_ARGUMENT;
    const glu_status st = check_sizes(sizes);
    if (st == GLU_OK) *bytes = low_bytes(mats, *sizes, sizes->K);
    return st;
}

glu_status glu_adapter_backward_workspace(const glu_adapter_sizes* sizes, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    const glu_status st = check_grad_sizes(sizes);
    if (st == GLU_OK) *bytes = grad_plan(*sizes).bytes;
    return st;
}

glu_status glu_adapter_backward(const void* dout, int64_t ldd, const void* x, int64_t ldx, const glu_adapter* ab,
                                const int32_t* index, const float* scale, const float* low, void* dx, int64_t lddx,
                                void* da, void* db, const glu_adapter_sizes* sizes, int dtype, void* workspace,
                                int64_t workspace_bytes, void* stream)
{
    if (dtype != GLU_DTYPE_BF16 && dtype != GLU_DTYPE_FP16) return GLU_ERR_BAD_ARGUMENT;
    glu_status st = check_grad_sizes(sizes);
    if (st != GLU_OK) return st;
    const glu_adapter_sizes s = *sizes;
    if (!dx && !da && !db) return GLU_OK;
    if (!ab) return GLU_ERR_NULL_POINTER;
    if (too_wide(s.M, ldd) || (da && too_wide(s.M, ldx)) || (dx && too_wide(s.M, lddx))) return GLU_ERR_BAD_STRIDE;
    const GradPlan p = grad_plan(s);
    Array arrays[12];
    int n = 0;
    arrays[n++] = {dout, s.M, s.N, ldd, 2, false};
    arrays[n++] = {x, da ? s.M : 0, s.K, ldx, 2, false};
    st = stack_arrays(ab, s, arrays + n);
    if (st != GLU_OK) return st;
    if (!dx) arrays[n].rows = 0;  // a is read for dx alone
    if (!dx && !da) arrays[n + 1].rows = 0;
    n += 2;
    arrays[n++] = {index, 1, s.M, s.M, 4, false};
    arrays[n++] = {scale, scale ? 1 : 0, s.L, s.L, 4, false};
    arrays[n++] = {low, db ? s.M : 0, s.R, s.R, 4, false};
    arrays[n++] = {dx, dx ? s.M : 0, s.K, lddx, 2, true};
    arrays[n++] = {da, da ? s.L : 0, s.R * s.K, s.R * s.K, 2, true};
    arrays[n++] = {db, db ? s.L : 0, s.N * s.R, s.N * s.R, 2, true};
    if (bad_workspace(workspace, workspace_bytes, p.bytes)) {
        st = check_arrays(arrays, n);
        return st != GLU_OK ? st : GLU_ERR_WORKSPACE;
    }
    arrays[n++] = {workspace, 1, p.bytes, p.bytes, 1, true};
    st = check_arrays(arrays, n);
    if (st != GLU_OK) return st;

    char* ws = (char*)workspace;
    float* d = (float*)ws;
    const hipStream_t hs = (hipStream_t)stream;
    glu::GradArgs g{};
    // the second product adds d's parts up and leaves the sum for the gradient
    float* const sum = p.splits > 1 && dx && s.K > 0 ? (float*)(ws + p.sum) : nullptr;
    g.side[0] = {x, sum ? sum : d, s.K > 0 ? da : nullptr, ldx, (int)s.K, sum ? 1 : p.splits, false};
    g.side[1] = {dout, low, s.N > 0 ? db : nullptr, ldd, (int)s.N, 1, true};
    g.index = index;
    g.scale = scale;
    g.order = (int32_t*)(ws + p.order);
    g.items = (int32_t*)(ws + p.table);
    g.part = (float*)(ws + p.part);
    g.M = (int)s.M;
    g.R = (int)s.R;
    g.L = (int)s.L;
    g.rows = p.rows;
    const bool any_grad = g.side[0].grad || g.side[1].grad, through = s.M > 0 && (dx || da);
    const glu::Stack b{ab->b, ab->b_stack, ab->b_row};
    hipError_t e = hipSuccess;
    if (!p.direct) {
        const glu::Turn turn{b, (uint16_t*)(ws + p.turned), through ? (int)s.N : 0, p.pitch};
        e = glu::adapter_prepare_launch(g, any_grad, turn, hs);
    }
    if (e == hipSuccess && through) {
        glu::LowArgs la{};
        la.v = dout;
        la.ldv = ldd;
        la.w[0] = p.direct ? b : glu::Stack{ws + p.turned, s.R * p.pitch, p.pitch};
        la.index = index;
        la.z = d;
        la.M = (int)s.M;
        la.C = (int)s.N;
        la.R = (int)s.R;
        la.L = (int)s.L;
        la.mats = 1;
        la.splits = p.splits;
        e = glu::adapter_low_launch(dtype, p.direct, la, hs);
    }
    if (e == hipSuccess && dx && s.M > 0 && s.K > 0) {
        glu::OutArgs oa{};
        oa.z = d;
        oa.w[0] = {ab->a, ab->a_stack, ab->a_row};
        oa.index = index;
        oa.scale = scale;
        oa.out = dx;
        oa.ldo = lddx;
        oa.low = da ? sum : nullptr;
        oa.M = (int)s.M;
        oa.N = (int)s.K;
        oa.R = (int)s.R;
        oa.L = (int)s.L;
        oa.mats = 1;
        oa.splits = p.splits;
        e = glu::adapter_out_launch(dtype, true, oa, hs);
    }
    if (e == hipSuccess && any_grad) e = glu::adapter_grad_launch(dtype, g, hs);
    return launched(e);
}

}  // extern "C"
