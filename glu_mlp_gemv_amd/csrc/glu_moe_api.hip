// C ABI of the expert layer (include/glu_moe.h): argument validation, workspace and launches, 64 rows at a time.
// Validation happens before any HIP call; nothing is allocated or cached.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/glu_moe.h"
#include "glu_check.h"
#include "glu_moe.h"
#include "glu_status.h"

namespace {

using glu::Array;
using glu::bad_dim;
using glu::ceil_div;

constexpr int64_t kMaxInner = 1 << 24;  // widths of an expert: its workgroups fit one launch

int64_t align16(int64_t n) { return (n + 15) & ~(int64_t)15; }

glu_status check_sizes(const glu_moe_sizes* s)
{
    if (!s) return GLU_ERR_NULL_POINTER;
    if (bad_dim(s->M) || s->K < 0 || s->K > kMaxInner || s->N < 0 || s->N > kMaxInner) return GLU_ERR_BAD_SHAPE;
    if (s->E < 1 || s->E > GLU_MOE_MAX_EXPERTS) return GLU_ERR_BAD_SHAPE;
    if (s->top < 1 || s->top > s->E || s->top > GLU_MOE_MAX_TOP) return GLU_ERR_BAD_SHAPE;
    // workgroups of the first product below 2^32 threads
    const int64_t rows = s->M < glu::kMoeRows ? s->M : glu::kMoeRows;
    const int64_t most = rows * s->top < s->E ? rows * s->top : s->E;
    return most * ceil_div(s->N, 32) >= (int64_t)1 << 23 ? GLU_ERR_BAD_SHAPE : GLU_OK;
}

struct Layout {
    glu::MoePlan plan;
    int64_t active, row, weight, act, factor, part, bytes, ld_act, ld_factor;  // offsets; how many experts are active is at 0
};
Layout layout(const glu_moe_sizes& s, int rows, bool e4m3)
{
    Layout l{};
    l.plan = glu::moe_plan(rows, (int)s.K, (int)s.N, (int)s.E, (int)s.top, e4m3);
    l.ld_act = (s.N + 7) / 8 * 8;
    l.ld_factor = ceil_div(s.N, 64) * 4;  // the second product reads four at a time
    l.active = 16;
    l.row = l.active + align16(s.E * (int64_t)sizeof(glu::Active));
    l.weight = l.row + align16(rows * s.top * 4);
    l.act = l.weight + align16(rows * s.top * 4);
    l.factor = l.act + align16(rows * s.top * l.ld_act * 4);
    l.part = l.factor + rows * s.top * l.ld_factor * 4;
    l.bytes = l.part + (l.plan.splits > 1 ? align16((int64_t)l.plan.splits * rows * s.K * 4) : 0);
    return l;
}

// E matrices of rows x cols as one array, and their scales as another
glu_status expert_arrays(const glu_expert_matrix* w, int64_t E, int64_t rows, int64_t cols, bool e4m3, Array* out)
{
    const int es = e4m3 ? 1 : 2;
    out[0] = Array{w->data, 0, 0, 0, es, false};
    out[1] = Array{w->scale, 0, 0, 0, 4, false};
    if (rows == 0 || cols == 0) return GLU_OK;
    if (rows > 1 && w->ld < cols) return GLU_ERR_BAD_STRIDE;
    const int64_t bytes = glu::extent(Array{w->data, rows, cols, w->ld, es, false});
    if (bytes < 0) return GLU_ERR_BAD_STRIDE;
    out[0] = Array{w->data, E, bytes / es, w->stack, es, false};
    if (!e4m3) return GLU_OK;
    const int64_t r = ceil_div(rows, 128), c = ceil_div(cols, 128);
    if (r > 1 && w->scale_ld < c) return GLU_ERR_BAD_STRIDE;
    const int64_t sb = glu::extent(Array{w->scale, r, c, w->scale_ld, 4, false});
    if (sb < 0) return GLU_ERR_BAD_STRIDE;
    out[1] = Array{w->scale, E, sb / 4, w->scale_stack, 4, false};
    return GLU_OK;
}

}  // namespace

extern "C" {

glu_status glu_moe_workspace(const glu_moe_sizes* sizes, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    const glu_status st = check_sizes(sizes);
    if (st != GLU_OK || sizes->M == 0 || sizes->K == 0) return st;
    // enough for both types of weights, and for the last rows of a call, which are fewer and cut otherwise
    const int64_t most = sizes->M < glu::kMoeRows ? sizes->M : glu::kMoeRows, last = sizes->M % glu::kMoeRows;
    for (const bool e4m3 : {false, true}) {
        for (const int64_t rows : {most, last ? last : most}) {
            const int64_t n = layout(*sizes, (int)rows, e4m3).bytes;
            if (n > *bytes) *bytes = n;
        }
    }
    return GLU_OK;
}

glu_status glu_moe_glu(const void* x, int64_t ldx, const void* logits, int64_t ldl, int logits_dtype,
                       const glu_expert_matrix* gate, const glu_expert_matrix* up, const glu_expert_matrix* down,
                       void* out, int64_t ldo, const glu_moe_sizes* sizes, int normalize, int dtype, int weight_dtype,
                       void* workspace, int64_t workspace_bytes, void* stream)
{
    if (dtype != GLU_DTYPE_BF16 && dtype != GLU_DTYPE_FP16) return GLU_ERR_BAD_ARGUMENT;
    if (logits_dtype != GLU_DTYPE_FP32 && logits_dtype != dtype) return GLU_ERR_BAD_ARGUMENT;
    if (weight_dtype != GLU_DTYPE_E4M3 && weight_dtype != dtype) return GLU_ERR_BAD_ARGUMENT;
    glu_status st = check_sizes(sizes);
    if (st != GLU_OK) return st;
    const glu_moe_sizes s = *sizes;
    if (s.M == 0 || s.K == 0) return GLU_OK;
    if (!gate || !up || !down) return GLU_ERR_NULL_POINTER;
    const bool e4m3 = weight_dtype == GLU_DTYPE_E4M3;
    const int ls = logits_dtype == GLU_DTYPE_FP32 ? 4 : 2;
    int64_t need = 0;
    glu_moe_workspace(&s, &need);
    Array arrays[10];
    arrays[0] = {x, s.M, s.K, ldx, 2, false};
    arrays[1] = {logits, s.M, s.E, ldl, ls, false};
    const glu_expert_matrix* w[3] = {gate, up, down};
    for (int i = 0; i < 3; ++i) {
        st = expert_arrays(w[i], s.E, i < 2 ? s.N : s.K, i < 2 ? s.K : s.N, e4m3, arrays + 2 + 2 * i);
        if (st != GLU_OK) return st;
    }
    arrays[8] = {out, s.M, s.K, ldo, 2, true};
    if (!workspace || ((uintptr_t)workspace & 15) || workspace_bytes < need) {
        st = glu::check_arrays(arrays, 9);
        return st != GLU_OK ? st : GLU_ERR_WORKSPACE;
    }
    arrays[9] = {workspace, 1, need, need, 1, true};
    st = glu::check_arrays(arrays, 10);
    if (st != GLU_OK) return st;

    for (int64_t m = 0; m < s.M; m += glu::kMoeRows) {
        const int rows = (int)(s.M - m < glu::kMoeRows ? s.M - m : glu::kMoeRows);
        const Layout l = layout(s, rows, e4m3);
        char* ws = (char*)workspace;
        glu::MoeArgs a{};
        a.x = (const char*)x + m * ldx * 2;
        a.logits = (const char*)logits + m * ldl * ls;
        a.out = (char*)out + m * ldo * 2;
        for (int i = 0; i < 3; ++i) {
            a.w[i] = {(const uint8_t*)w[i]->data, w[i]->scale, w[i]->stack, w[i]->ld, w[i]->scale_stack, w[i]->scale_ld};
        }
        a.ldx = ldx;
        a.ldl = ldl;
        a.ldo = ldo;
        a.M = rows;
        a.K = (int)s.K;
        a.N = (int)s.N;
        a.E = (int)s.E;
        a.top = (int)s.top;
        a.normalize = normalize != 0;
        a.actives = (int*)ws;
        a.active = (glu::Active*)(ws + l.active);
        a.row = (int*)(ws + l.row);
        a.weight = (float*)(ws + l.weight);
        a.act = (uint16_t*)(ws + l.act);
        a.factor = (float*)(ws + l.factor);
        a.part = (float*)(ws + l.part);
        a.ld_act = l.ld_act;
        a.ld_factor = l.ld_factor;
        const hipError_t e = glu::moe_launch(dtype, logits_dtype, e4m3, a, l.plan, (hipStream_t)stream);
        if (e != hipSuccess) return glu::fail_launch(e);
    }
    return GLU_OK;
}

glu_status glu_moe_logits(const void* x, int64_t ldx, const void* router, int64_t ldr, float* logits, int64_t M, int64_t K,
                          int64_t E, int dtype, void* stream)
{
    if (dtype != GLU_DTYPE_BF16 && dtype != GLU_DTYPE_FP16) return GLU_ERR_BAD_ARGUMENT;
    if (bad_dim(M) || K < 0 || K > kMaxInner || E < 1 || E > GLU_MOE_MAX_EXPERTS) return GLU_ERR_BAD_SHAPE;
    if (M == 0) return GLU_OK;
    const Array arrays[] = {
        {x, M, K, ldx, 2, false},
        {router, E, K, ldr, 2, false},
        {logits, M, E, E, 4, true},
    };
    const glu_status st = glu::check_arrays(arrays, 3);
    if (st != GLU_OK) return st;
    const hipError_t e = glu::moe_logits_launch(dtype, {x, router, logits, ldx, ldr, (int)M, (int)K, (int)E}, (hipStream_t)stream);
    return e == hipSuccess ? GLU_OK : glu::fail_launch(e);
}

}  // extern "C"
