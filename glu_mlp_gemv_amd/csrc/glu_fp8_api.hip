// C ABI of the 8-bit decoder-MLP path (include/glu_fp8.h): argument
// validation, the choice of kernel, and launch.  Validation happens before any
// HIP call; nothing is allocated or cached.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/glu_fp8.h"
#include "glu_check.h"
#include "glu_fp8.h"
#include "glu_norm.h"
#include "glu_quantize.h"
#include "glu_status.h"

namespace {

using glu::Array;
using glu::bad_dim;
using glu::ceil_div;
using glu::check_arrays;
using glu::extent;
using glu::kMaxDim;

constexpr int64_t kMaxFastLd = 1 << 23;        // the tile kernel's row offsets: 256 rows * stride < 2^32
constexpr int kGroup = 128;
constexpr int kCUs = 256;

int type_size(int dtype) { return dtype == GLU_DTYPE_E4M3 ? 1 : dtype == GLU_DTYPE_FP32 ? 4 : 2; }
bool input_type(int dtype) { return dtype == GLU_DTYPE_BF16 || dtype == GLU_DTYPE_FP16 || dtype == GLU_DTYPE_FP32; }

glu_status launched(hipError_t e) { return e == hipSuccess ? GLU_OK : glu::fail_launch(e); }

glu_status norm_call(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* sum,
                     int64_t lds, void* out, int64_t ldo, float* scale, int64_t ld_scale, float* rstd, int64_t M,
                     int64_t K, float eps, int dtype, bool e4m3, void* stream)
{
    if (!input_type(dtype) || !(eps >= 0.0f) || !(eps <= 3.4028234e38f)) return GLU_ERR_BAD_ARGUMENT;
    if (bad_dim(M) || bad_dim(K) || K == 0) return GLU_ERR_BAD_SHAPE;
    if (M == 0) return GLU_OK;
    if ((residual == nullptr) != (sum == nullptr)) return GLU_ERR_NULL_POINTER;
    const int es = type_size(dtype);
    const int64_t with = residual ? M : 0;
    const Array arrays[] = {
        {x, M, K, ldx, es, false},
        {residual, with, K, ldr, es, false},
        {weight, 1, K, K, es, false},
        {sum, with, K, lds, es, true},
        {out, M, K, ldo, e4m3 ? 1 : es, true},
        {scale, e4m3 ? ceil_div(K, kGroup) : 0, M, ld_scale, 4, true},
        {rstd, rstd ? 1 : 0, M, M, 4, true},
    };
    const glu_status st = check_arrays(arrays, 7, 1u << 3, 1u << 0 | 1u << 1);
    if (st != GLU_OK) return st;
    const glu::NormArgs a{x,   residual, weight, sum,      out,    scale,  rstd, ldx,
                          ldr, lds,      ldo,    ld_scale, (int)M, (int)K, eps};
    return launched(glu::norm_launch(dtype, e4m3, a, (hipStream_t)stream));
}

// ---- products ----------------------------------------------------------------------

// outputs that show more than the 8-bit matrix unit's sums hold (glu_fp8_mfma.h), and up to 16 rows, where the other
// unit has the time, all of them
bool needs_wide(int64_t M, int out_dtype)
{
    return M <= 16 || out_dtype == GLU_DTYPE_FP32 || out_dtype == GLU_DTYPE_E4M3;
}

// Microseconds that a tiled product is expected to take.  A workgroup takes a constant time per stage (one
// K-block of its tile), each round of 256 workgroups (one per CU) has a start and an end, and sums that leave
// the kernel cost their way to memory and back; that and the time to read the operands join as a fourth-power
// mean.  The constants are fitted to timings.  Over 98 other sizes (M = 17 to 4096, K = 128 to 17408, N = 256 to 17408;
// 1978 timings, profiles/glu_fp8_tile_shapes.json) the plan of least expected time is 0.7 % slower than the best in the
// mean, 23 % at most (270 rows, K = 11008 N = 2944), then 10 and 4.  By whole rounds of one shape alone it is 1.1 %, and
// leaving out one shape makes that 2.7 to 9.3 % in the mean, 32 to 57 % at most.
constexpr double kStage[2][glu::kTileShapeCount] = {{1.7, 0.98, 0.74, 0.44, 0.27}, {3.3, 1.8, 1.3, 0.8, 0.51}};
constexpr double kRound = 2.4, kLaunch = 2.8, kJoinSplit = 0.41;
constexpr double kJoin = 2.5;                              // 1.2 of it the kernel, the rest the host's launch
constexpr double kPlaneBytes = 3.3e6, kReadBytes = 4.5e6;  // per microsecond

bool has_planes(int mats, int out_dtype, int shape, int64_t splits)
{
    return splits > 1 || (out_dtype == GLU_DTYPE_E4M3 && !glu::fp8_tile_owns_groups(mats, shape));
}

double tile_cost(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int shape, int splits)
{
    const glu::TileShape& t = glu::kTileShapes[shape];
    const int64_t tiles = ceil_div(M, t.bm) * ceil_div(N, t.br / mats);
    const int stages = ((int)ceil_div(K, kGroup) + splits - 1) / splits;
    const double round = stages * kStage[needs_wide(M, out_dtype)][shape] + kRound;
    double us = kLaunch + (double)ceil_div(tiles * splits, kCUs) * round;
    if (has_planes(mats, out_dtype, shape, splits)) {
        us += kJoin + kJoinSplit * splits + (double)(splits * mats * 4) * (double)M * (double)N / kPlaneBytes;
    }
    const double read = kLaunch + ((double)M + (double)mats * (double)N) * (double)K / kReadBytes;
    return sqrt(sqrt(us * us * us * us + read * read * read * read));
}

// The same of the streaming kernel with 16 weight rows per workgroup: a CU with one workgroup more than the others is
// waited for, which the tiled kernel avoids by splitting K (5 rows, K = 17408 N = 5120, 320 workgroups: 29.0 us
// against 20.8; 16 rows 38.5 against 21.6).  A fit to 7 sizes at 5, 8 and 16 rows, all within 9 %.
double stream_cost(int mats, int64_t M, int64_t N, int64_t K, int out_dtype)
{
    const double block = mats == 1 ? 0.0945 + 0.0027 * (double)M : 0.1575 + 0.0039 * (double)M;
    double us = kLaunch + (double)(ceil_div(ceil_div(N, 16), kCUs) * ceil_div(K, kGroup)) * block;
    if (out_dtype == GLU_DTYPE_E4M3) us += kJoin + kJoinSplit + (double)(mats * 4) * (double)M * (double)N / kPlaneBytes;
    return us;
}

double best_tile(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, glu_fp8_plan* p)
{
    double best = 0.0;
    p->kernel = GLU_FP8_KERNEL_TILE;
    p->splits = 0;
    for (int shape = 0; shape < glu::kTileShapeCount; ++shape) {
        for (const int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (splits > ceil_div(K, kGroup)) break;
            const double us = tile_cost(mats, M, N, K, out_dtype, shape, splits);
            if (p->splits == 0 || us < best) {
                best = us;
                p->tile = shape;
                p->width = glu::kTileShapes[shape].threads;
                p->splits = splits;
            }
        }
    }
    return best;
}

// Fills the launch shape for sizes >= 1.
void choose(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, bool fast, glu_fp8_plan* p)
{
    const int64_t KB = ceil_div(K, kGroup);
    p->splits = 1;
    if (!fast) {
        p->kernel = GLU_FP8_KERNEL_ANY;
        p->tile = 16;
        p->width = 4;
        return;
    }
    if (M <= 16) {
        // 4 weight rows a workgroup for one or two rows of x, and up to 4 for two matrices or where 16 would leave a
        // third of the CUs idle; else 16.  4 rows, in 4 and in 16: K = 9216 N = 2048 7.2 and 9.1 us, N = 2560 (160 of 256
        // CUs) 9.9 and 10.0, N = 2816 (176) 10.9 and 10.1, N = 3328 13.1 and 10.2; K = 17408 N = 2560 17.1 and 17.2, N =
        // 2816 17.2 and 16.8, N = 4096 21.6 and 16.8.  Dual, which goes up and down with N: K = 9216 N = 512 8.0 and 12.9,
        // N = 2048 11.2 and 14.6, N = 4096 19.4 and 17.1, N = 6144 25.7 and 28.2, N = 9216 38.0 and 39.2, N = 12288 47.1
        // and 42.9
        const bool few = M <= 2 || (M <= 4 && (mats == 2 || 3 * ceil_div(N, 16) <= 2 * kCUs));
        if (!few && best_tile(mats, M, N, K, out_dtype, p) < stream_cost(mats, M, N, K, out_dtype)) return;
        p->kernel = GLU_FP8_KERNEL_STREAM;
        p->tile = few ? 4 : 16;
        p->splits = 1;
        // Waves that keep enough loads in flight; more only lengthen the join (one row, K = 9216 N = 2560: 8.1 us
        // with 3, 8.4 with 8; 8 rows, K = 12288 N = 4096: 13.9 with 6, 14.1 with 8; dual K = 2560 N = 9216: 14.8 with 6,
        // 14.0 with 8)
        const int64_t steps = ceil_div(KB, 16 / p->tile), most = few ? 3 : mats == 1 ? 6 : 8;
        p->width = (int)(steps < most ? steps : most);
        return;
    }
    double best = best_tile(mats, M, N, K, out_dtype, p);
    // Whole rounds of the largest tile in one launch and the columns left over in another, shaped for
    // themselves, where a last round would leave most CUs idle
    const glu::TileShape& t = glu::kTileShapes[0];
    const int64_t bn = t.br / mats, high = ceil_div(M, t.bm);
    const int64_t rounds = high * (N / bn) / kCUs, columns = rounds * kCUs / high * bn;
    if (columns > 0 && columns < N) {
        glu_fp8_plan rest{};
        const double us = tile_cost(mats, M, columns, K, out_dtype, 0, 1) +
                          best_tile(mats, M, N - columns, K, out_dtype, &rest);
        if (us < best) {
            best = us;
            p->tile = 0;
            p->width = t.threads;
            p->splits = 1;
            p->columns = columns;
        }
    }
}

// what follows from a launch shape
void complete(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, glu_fp8_plan* p)
{
    if (p->columns > 0) {  // the first columns by this shape, the others by their own
        glu_fp8_plan first = *p, rest{};
        first.columns = 0;
        complete(mats, M, p->columns, K, out_dtype, &first);
        best_tile(mats, M, N - p->columns, K, out_dtype, &rest);
        complete(mats, M, N - p->columns, K, out_dtype, &rest);
        p->launches = first.launches + rest.launches;
        p->workspace_bytes = first.workspace_bytes;
        if (rest.workspace_bytes > p->workspace_bytes) p->workspace_bytes = rest.workspace_bytes;
        return;
    }
    const bool planes = p->kernel == GLU_FP8_KERNEL_TILE
                            ? has_planes(mats, out_dtype, p->tile, p->splits)
                            : p->splits > 1 || out_dtype == GLU_DTYPE_E4M3;
    p->launches = planes ? 2 : 1;
    p->workspace_bytes = planes ? (int64_t)p->splits * mats * M * N * 4 : 0;
}

glu_status check_sizes(int mats, int64_t M, int64_t N, int64_t K, int out_dtype)
{
    if (mats != 1 && mats != 2) return GLU_ERR_BAD_ARGUMENT;
    if (out_dtype < GLU_DTYPE_BF16 || out_dtype > GLU_DTYPE_E4M3) return GLU_ERR_BAD_ARGUMENT;
    if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return GLU_ERR_BAD_SHAPE;
    if (M > 0 && N > ((int64_t)1 << 50) / M) return GLU_ERR_BAD_SHAPE;  // bytes of any workspace fit 63 bits
    return GLU_OK;
}

glu_status product_plan(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, bool fast,
                        const glu_fp8_plan* asked, glu_fp8_plan* p)
{
    *p = glu_fp8_plan{};
    const glu_status st = check_sizes(mats, M, N, K, out_dtype);
    if (st != GLU_OK) return st;
    if (M == 0 || N == 0) {
        p->kernel = GLU_FP8_KERNEL_NONE;
        return GLU_OK;
    }
    if (K == 0) {
        p->kernel = GLU_FP8_KERNEL_ZERO;
        p->launches = 1;
        return GLU_OK;
    }
    if (asked) {
        p->kernel = asked->kernel;
        p->tile = asked->tile;
        p->width = asked->width;
        p->splits = asked->splits;
        p->columns = asked->columns;
        if (p->columns != 0 && (p->kernel != GLU_FP8_KERNEL_TILE || p->columns < 0 || p->columns >= N ||
                                p->columns % kGroup != 0)) {
            return GLU_ERR_UNSUPPORTED;
        }
        if (p->splits < 1 || p->splits > ceil_div(K, kGroup) || p->splits > 64) return GLU_ERR_UNSUPPORTED;
        if (p->kernel == GLU_FP8_KERNEL_TILE) {
            if (!fast || p->tile < 0 || p->tile >= glu::kTileShapeCount) return GLU_ERR_UNSUPPORTED;
            p->width = glu::kTileShapes[p->tile].threads;
        } else if (p->kernel == GLU_FP8_KERNEL_STREAM || p->kernel == GLU_FP8_KERNEL_ANY) {
            const bool any = p->kernel == GLU_FP8_KERNEL_ANY;
            if (!any && !fast) return GLU_ERR_UNSUPPORTED;
            const glu::StreamConfig c{p->tile, p->width, p->splits, any};
            if (!glu::fp8_stream_supported(c, (int)M)) return GLU_ERR_UNSUPPORTED;
        } else {
            return GLU_ERR_UNSUPPORTED;
        }
    } else {
        choose(mats, M, N, K, out_dtype, fast, p);
    }
    // the streaming grid: one row tile's threads below 2^32
    if (p->kernel != GLU_FP8_KERNEL_TILE && ceil_div(N, p->tile) * p->splits > 0xffffffffLL / (64 * p->width)) {
        return GLU_ERR_UNSUPPORTED;
    }
    complete(mats, M, N, K, out_dtype, p);
    return GLU_OK;
}

// One launch shape on checked operands: the product, and the join of its parts
hipError_t run_product(int mats, const glu_fp8_plan& p, glu::Fp8Args a, int out_dtype, bool wide, hipStream_t s)
{
    a.out_dtype = p.launches == 2 ? glu::kPartial : out_dtype;
    hipError_t e;
    if (p.kernel == GLU_FP8_KERNEL_TILE) {
        e = glu::fp8_tile_launch(mats, glu::TileConfig{p.tile, p.splits, wide}, a, s);
    } else {
        const glu::StreamConfig c{p.tile, p.width, p.splits, p.kernel == GLU_FP8_KERNEL_ANY};
        e = glu::fp8_stream_launch(mats, c, a, s);
    }
    if (e != hipSuccess || p.launches == 1) return e;
    const glu::FinishArgs fin{a.part, a.out, a.scale, a.ldo, a.lds, a.M, a.N, p.splits, mats};
    return glu::finish_launch(out_dtype, fin, s);
}

// A layout that is not fast, above 16 rows: where the workspace has room for them the operands may be copied to the
// fast layout first, behind the product's own part of it.  The copies run on the bf16 unit, as the kernel in place
// does.  A row too long for the fast layout's strides stays in place, whose kernel counts in 64 bits.
int64_t padded(int64_t K) { return (K + 15) / 16 * 16; }
bool may_copy(int64_t M, int64_t K) { return M > 16 && padded(K) <= kMaxFastLd; }

// Whether copies are expected to pay.  In place 16 rows of x pass over the weights at a time, more than twice as slowly
// where addresses are no multiples of 4 bytes; a copy costs its launch and its bytes there and back.  Over 107 sizes of
// 17 to 512 rows the choice is 11 % slower than the better at most.  Copied and in place, us: K = 4100 N = 4096 17 rows
// 29.3 and 12.9, 64 rows 30.6 and 19.8, 128 rows 39.3 and 37.6, 256 rows 39.7 and 65.6, 2048 rows 95 and 470; K = 12290
// N = 4096 17 rows 40.6 and 61.2; K = 1030 N = 1024 256 rows 19.8 and 12.5, 512 rows 19.9 and 24.3; dual K = 2561 N =
// 9216 17 rows 43 and 63; dual K = 5125 N = 17408 4096 rows 1290 and 21000.
constexpr double kPlaceAligned = 1.3e-7, kPlace = 3.6e-7, kCopy = 6.0, kCopyBytes = 3e6;
bool copies_pay(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, bool aligned)
{
    glu_fp8_plan p{};
    const double copied = best_tile(mats, M, N, padded(K), out_dtype, &p) + kCopy * (mats + 1) +
                          ((double)M + (double)mats * (double)N) * (double)K / kCopyBytes;
    const double k = (double)(K < 2 * kGroup ? 2 * kGroup : K);  // fewer K-blocks leave waves idle
    const double place = kLaunch + (double)ceil_div(M, 16) * (double)N * k * (mats + 1) * (aligned ? kPlaceAligned : kPlace);
    return copied < place;
}

glu_status copy_plan(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, glu_fp8_plan* p, int64_t* bytes)
{
    const glu_status st = product_plan(mats, M, N, padded(K), out_dtype, true, nullptr, p);
    *bytes = padded(p->workspace_bytes) + (M + mats * N) * padded(K);
    return st;
}

glu_status product_call(const glu_fp8_matrix* x, const glu_fp8_matrix* w0, const glu_fp8_matrix* w1, int mats,
                        void* out, int64_t ldo, float* out_scale, int64_t ld_scale, int64_t M, int64_t N, int64_t K,
                        int out_dtype, const glu_fp8_plan* asked, void* ws, int64_t ws_bytes, void* stream)
{
    glu_status st = check_sizes(mats, M, N, K, out_dtype);
    if (st != GLU_OK) return st;
    if (M == 0 || N == 0) return GLU_OK;
    if (!x || !w0 || (mats == 2 && !w1)) return GLU_ERR_NULL_POINTER;
    const glu_fp8_matrix* w[2] = {w0, w1};
    const int64_t KB = ceil_div(K, kGroup), NB = ceil_div(N, kGroup);
    // scales: x's by two strides of any order, a weight's rows contiguous
    if (KB > 0 && (x->scale_row < 0 || x->scale_block < 0)) return GLU_ERR_BAD_STRIDE;
    if (KB > 0 && ((M > 1 && x->scale_row > INT64_MAX / 8 / M) || (KB > 1 && x->scale_block > INT64_MAX / 8 / KB))) {
        return GLU_ERR_BAD_STRIDE;
    }
    for (int i = 0; i < mats; ++i) {
        if (KB > 1 && w[i]->scale_block != 1) return GLU_ERR_BAD_STRIDE;
    }
    const int64_t sx_span = KB > 0 ? (M - 1) * x->scale_row + (KB - 1) * x->scale_block + 1 : 0;
    const int64_t on = K > 0 ? 1 : 0;  // with K == 0 no operand is read
    const bool e4m3 = out_dtype == GLU_DTYPE_E4M3;
    uintptr_t bits = 0;
    bool fast = K % 16 == 0;
    if (on) {
        bits = (uintptr_t)x->data | (M > 1 ? (uintptr_t)x->ld : 0);
        fast = fast && (M <= 1 || x->ld <= kMaxFastLd);
        for (int i = 0; i < mats; ++i) {
            bits |= (uintptr_t)w[i]->data | (N > 1 ? (uintptr_t)w[i]->ld : 0);
            fast = fast && (N <= 1 || w[i]->ld <= kMaxFastLd);
        }
        fast = fast && (bits & 15) == 0;
    }
    glu_fp8_plan p;
    bool copied = false;
    int64_t need = 0;
    if (on && !fast && !asked && may_copy(M, K) &&
        (product_plan(mats, M, N, K, out_dtype, false, nullptr, &p) != GLU_OK ||
         copies_pay(mats, M, N, K, out_dtype, (bits & 3) == 0))) {
        st = copy_plan(mats, M, N, K, out_dtype, &p, &need);
        copied = st == GLU_OK && ws && ((uintptr_t)ws & 15) == 0 && ws_bytes >= need;
    }
    if (!copied) {
        st = product_plan(mats, M, N, K, out_dtype, fast, asked, &p);
        need = p.workspace_bytes;
    }
    if (st != GLU_OK) return st;
    const Array arrays[] = {
        {x->data, M * on, K, x->ld, 1, false},
        {x->scale, on, sx_span, sx_span, 4, false},
        {w0->data, N * on, K, w0->ld, 1, false},
        {w0->scale, NB * on, KB, w0->scale_row, 4, false},
        {w1 ? w1->data : nullptr, mats == 2 ? N * on : 0, K, w1 ? w1->ld : K, 1, false},
        {w1 ? w1->scale : nullptr, mats == 2 ? NB * on : 0, KB, w1 ? w1->scale_row : KB, 4, false},
        {out, M, N, ldo, type_size(out_dtype), true},
        {out_scale, e4m3 ? NB : 0, M, ld_scale, 4, true},
        {ws, need && ws ? 1 : 0, need, need, 1, true},
    };
    st = check_arrays(arrays, 9);
    if (st != GLU_OK) return st;
    if (need > 0 && (!ws || ((uintptr_t)ws & 15) || ws_bytes < need)) return GLU_ERR_WORKSPACE;

    hipStream_t s = (hipStream_t)stream;
    if (p.kernel == GLU_FP8_KERNEL_ZERO) {
        const glu::FinishArgs zero{nullptr, out, out_scale, ldo, ld_scale, (int)M, (int)N, 0, mats};
        return launched(glu::finish_launch(out_dtype, zero, s));
    }
    glu::Fp8Args a{};
    a.x = x->data;
    a.sx = x->scale;
    a.ldx = x->ld;
    a.sxm = x->scale_row;
    a.sxg = x->scale_block;
    for (int i = 0; i < mats; ++i) {
        a.w[i] = w[i]->data;
        a.sw[i] = w[i]->scale;
        a.ldw[i] = w[i]->ld;
        a.ldsw[i] = w[i]->scale_row;
    }
    a.out = out;
    a.scale = out_scale;
    a.ldo = ldo;
    a.lds = ld_scale;
    a.part = static_cast<float*>(ws);
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    const bool wide = copied || needs_wide(M, out_dtype);
    if (copied) {
        const int kp = (int)padded(K);
        uint8_t* to = static_cast<uint8_t*>(ws) + padded(p.workspace_bytes);
        hipError_t e = glu::copy_rows_launch(a.x, a.ldx, to, kp, a.M, a.K, s);
        a.x = to;
        a.ldx = kp;
        to += (int64_t)M * kp;
        for (int i = 0; i < mats && e == hipSuccess; ++i) {
            e = glu::copy_rows_launch(a.w[i], a.ldw[i], to, kp, a.N, a.K, s);
            a.w[i] = to;
            a.ldw[i] = kp;
            to += (int64_t)N * kp;
        }
        if (e != hipSuccess) return launched(e);
        a.K = kp;
        K = kp;
    }
    if (p.columns > 0) {
        glu_fp8_plan rest{};
        best_tile(mats, M, N - p.columns, K, out_dtype, &rest);
        complete(mats, M, N - p.columns, K, out_dtype, &rest);
        glu_fp8_plan first = p;
        first.columns = 0;
        complete(mats, M, p.columns, K, out_dtype, &first);
        a.N = (int)p.columns;
        const hipError_t e = run_product(mats, first, a, out_dtype, wide, s);
        if (e != hipSuccess) return launched(e);
        for (int i = 0; i < mats; ++i) {
            a.w[i] += p.columns * a.ldw[i];
            a.sw[i] += p.columns / kGroup * a.ldsw[i];
        }
        a.out = static_cast<char*>(a.out) + p.columns * type_size(out_dtype);
        if (a.scale) a.scale += p.columns / kGroup * a.lds;
        a.N = (int)(N - p.columns);
        return launched(run_product(mats, rest, a, out_dtype, wide, s));
    }
    return launched(run_product(mats, p, a, out_dtype, wide, s));
}

}  // namespace

extern "C" {

glu_status glu_add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                            void* sum, int64_t lds, void* out, int64_t ldo, float* rstd, int64_t M, int64_t K,
                            float eps, int dtype, void* stream)
{
    return norm_call(x, ldx, residual, ldr, weight, sum, lds, out, ldo, nullptr, 0, rstd, M, K, eps, dtype, false,
                     stream);
}

glu_status glu_add_rms_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                void* sum, int64_t lds, uint8_t* q, int64_t ldq, float* scale, int64_t ld_scale,
                                float* rstd, int64_t M, int64_t K, float eps, int dtype, void* stream)
{
    return norm_call(x, ldx, residual, ldr, weight, sum, lds, q, ldq, scale, ld_scale, rstd, M, K, eps, dtype, true,
                     stream);
}

glu_status glu_add_rms_norm_backward_workspace(int64_t M, int64_t K, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    if (bad_dim(M) || bad_dim(K) || K == 0) return GLU_ERR_BAD_SHAPE;
    for (int dtype = GLU_DTYPE_BF16; dtype <= GLU_DTYPE_FP32; ++dtype) {  // what serves any of the types
        const int64_t need = glu::norm_grad_part_floats(dtype, (int)M, (int)K) * 4;
        if (need > *bytes) *bytes = need;
    }
    return GLU_OK;
}

glu_status glu_add_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                                     const float* rstd, const void* dresidual, int64_t lddr, void* dx, int64_t lddx,
                                     void* dweight, int64_t M, int64_t K, int dtype, void* workspace,
                                     int64_t workspace_bytes, void* stream)
{
    if (!input_type(dtype)) return GLU_ERR_BAD_ARGUMENT;
    int64_t need = 0;
    const glu_status size = glu_add_rms_norm_backward_workspace(M, K, &need);
    if (size != GLU_OK) return size;
    const int es = type_size(dtype);
    const Array arrays[] = {
        {dy, M, K, lddy, es, false},
        {h, M, K, ldh, es, false},
        {weight, M > 0 ? 1 : 0, K, K, es, false},
        {rstd, M > 0 ? 1 : 0, M, M, 4, false},
        {dresidual, dresidual ? M : 0, K, lddr, es, false},
        {dx, M, K, lddx, es, true},
        {dweight, 1, K, K, es, true},
        {workspace, need && workspace ? 1 : 0, need, need, 1, true},
    };
    const glu_status st = check_arrays(arrays, 8, 1u << 5, 1u << 4);
    if (st != GLU_OK) return st;
    if (need > 0 && (!workspace || ((uintptr_t)workspace & 15) || workspace_bytes < need)) return GLU_ERR_WORKSPACE;
    const glu::NormGradArgs a{dy, h, dresidual, weight, rstd, dx, dweight, static_cast<float*>(workspace),
                              lddy, ldh, lddr, lddx, (int)M, (int)K};
    return launched(glu::norm_grad_launch(dtype, a, (hipStream_t)stream));
}

glu_status glu_fp8_quantize(const void* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, int64_t ld_scale,
                            int64_t M, int64_t K, int dtype, void* stream)
{
    if (!input_type(dtype)) return GLU_ERR_BAD_ARGUMENT;
    if (bad_dim(M) || bad_dim(K)) return GLU_ERR_BAD_SHAPE;
    if (M == 0 || K == 0) return GLU_OK;
    const Array arrays[] = {
        {x, M, K, ldx, type_size(dtype), false},
        {q, M, K, ldq, 1, true},
        {scale, ceil_div(K, kGroup), M, ld_scale, 4, true},
    };
    const glu_status st = check_arrays(arrays, 3);
    if (st != GLU_OK) return st;
    return launched(glu::quantize_rows_launch(dtype, x, ldx, q, ldq, scale, ld_scale, (int)M, (int)K,
                                              (hipStream_t)stream));
}

glu_status glu_fp8_quantize_weight(const void* w, int64_t ldw, uint8_t* q, int64_t ldq, float* scale,
                                   int64_t ld_scale, int64_t N, int64_t K, int dtype, void* stream)
{
    if (!input_type(dtype)) return GLU_ERR_BAD_ARGUMENT;
    if (bad_dim(N) || bad_dim(K)) return GLU_ERR_BAD_SHAPE;
    if (N == 0 || K == 0) return GLU_OK;
    const Array arrays[] = {
        {w, N, K, ldw, type_size(dtype), false},
        {q, N, K, ldq, 1, true},
        {scale, ceil_div(N, kGroup), ceil_div(K, kGroup), ld_scale, 4, true},
    };
    const glu_status st = check_arrays(arrays, 3);
    if (st != GLU_OK) return st;
    return launched(glu::quantize_blocks_launch(dtype, w, ldw, q, ldq, scale, ld_scale, (int)N, (int)K,
                                                (hipStream_t)stream));
}

glu_status glu_fp8_linear(const glu_fp8_matrix* x, const glu_fp8_matrix* w, void* out, int64_t ldo, float* out_scale,
                          int64_t ld_scale, int64_t M, int64_t N, int64_t K, int out_dtype, void* workspace,
                          int64_t workspace_bytes, void* stream)
{
    return product_call(x, w, nullptr, 1, out, ldo, out_scale, ld_scale, M, N, K, out_dtype, nullptr, workspace,
                        workspace_bytes, stream);
}

glu_status glu_fp8_dual_glu(const glu_fp8_matrix* x, const glu_fp8_matrix* gate, const glu_fp8_matrix* up, void* out,
                            int64_t ldo, float* out_scale, int64_t ld_scale, int64_t M, int64_t N, int64_t K,
                            int out_dtype, void* workspace, int64_t workspace_bytes, void* stream)
{
    return product_call(x, gate, up, 2, out, ldo, out_scale, ld_scale, M, N, K, out_dtype, nullptr, workspace,
                        workspace_bytes, stream);
}

glu_status glu_fp8_product_tuned(const glu_fp8_matrix* x, const glu_fp8_matrix* w, const glu_fp8_matrix* up,
                                 void* out, int64_t ldo, float* out_scale, int64_t ld_scale, int64_t M, int64_t N,
                                 int64_t K, int out_dtype, const glu_fp8_plan* plan, void* workspace,
                                 int64_t workspace_bytes, void* stream)
{
    return product_call(x, w, up, up ? 2 : 1, out, ldo, out_scale, ld_scale, M, N, K, out_dtype, plan, workspace,
                        workspace_bytes, stream);
}

glu_status glu_fp8_product_plan(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int fast,
                                glu_fp8_plan* plan)
{
    if (!plan) return GLU_ERR_NULL_POINTER;
    return product_plan(mats, M, N, K, out_dtype, fast != 0, nullptr, plan);
}

glu_status glu_fp8_product_workspace(int mats, int64_t M, int64_t N, int64_t K, int out_dtype,
                                     const glu_fp8_plan* plan, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    glu_fp8_plan p;
    const glu_status st = product_plan(mats, M, N, K, out_dtype, true, plan, &p);
    if (st == GLU_OK) *bytes = p.workspace_bytes;
    return st;
}

glu_status glu_fp8_copy_workspace(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    const glu_status size = check_sizes(mats, M, N, K, out_dtype);
    if (size != GLU_OK || !may_copy(M, K) || N == 0 || K == 0) return size;
    glu_fp8_plan p;
    const glu_status st = copy_plan(mats, M, N, K, out_dtype, &p, bytes);
    if (st != GLU_OK) {
        *bytes = 0;
    } else if (product_plan(mats, M, N, K, out_dtype, false, nullptr, &p) == GLU_OK && p.workspace_bytes > *bytes) {
        *bytes = p.workspace_bytes;  // a call that is not copied after all
    }
    return st;
}

glu_status glu_fp8_workspace(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int64_t* bytes)
{
    if (!bytes) return GLU_ERR_NULL_POINTER;
    *bytes = 0;
    for (int fast = 0; fast < 2; ++fast) {
        glu_fp8_plan p;
        const glu_status st = product_plan(mats, M, N, K, out_dtype, fast != 0, nullptr, &p);
        if (fast == 0 && st == GLU_ERR_UNSUPPORTED) continue;  // too large for the other layouts' kernel
        if (st != GLU_OK) return st;
        if (p.workspace_bytes > *bytes) *bytes = p.workspace_bytes;
    }
    return GLU_OK;
}

}  // extern "C"
