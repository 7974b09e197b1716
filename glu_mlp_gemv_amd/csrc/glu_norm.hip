// Residual addition + RMS norm, to the input's type or to e4m3 with a scale
// per 128 columns, and its backward.
//
//   h = T(x + residual)      r = 1 / sqrt(mean(h^2) + eps)      y = h r w
//
// Bound by memory: every value is read once and written once, so a row stays
// in registers between its sum of squares and its scaled store.  A row is held by `wpr` waves,
// C chunks of 8 values per lane; chunk c = lane + 64 (wave + wpr i), so that 16 neighbouring lanes hold one
// group of 128 columns and its maximum is a 4-step DPP reduction without LDS.
#include "../../include/glu_fp8.h"
#include "glu_fp8_device.h"
#include "glu_norm.h"

namespace glu {

namespace {

constexpr int kNormMaxWaves = 16;
constexpr int kNormMaxChunks = 4;  // per lane

// sum over a team of `waves` waves, in wave order; every lane gets it.  `slot` is the team's LDS row.
__device__ __forceinline__ float team_sum(float v, float* slot, int wave, int lane, int waves)
{
    v = wave_sum(v);
    if (waves == 1) return v;
    if (lane == 0) slot[wave] = v;
    __syncthreads();
    float s = slot[0];
    for (int w = 1; w < waves; ++w) s += slot[w];
    return s;
}

template <class T, bool E4M3>
__device__ __forceinline__ void norm_store(const NormArgs& a, int row, int c, const float (&y)[8], int n)
{
    if constexpr (E4M3) {
        const Scale s = scale_of(max16(abs_max8(y)));
        if (n > 0) {
            store_e4m3x8(static_cast<uint8_t*>(a.out) + row * a.ldo + 8 * (int64_t)c, e4m3x8(y, s), n);
            if ((c & 15) == 0) a.scale[(c >> 4) * a.lds + row] = s.s;
        }
    } else {
        if (n > 0) store_chunk(static_cast<T*>(a.out) + row * a.ldo + 8 * (int64_t)c, narrow8<T>(y), n);
    }
}

// h of one chunk: the sum rounded to T, and stored, where there is a residual
template <class T>
__device__ __forceinline__ void norm_input(const NormArgs& a, int row, int c, int n, float (&h)[8])
{
    if (n <= 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = 0.0f;
        return;
    }
    const Chunk<T> x = load_chunk(static_cast<const T*>(a.x) + row * a.ldx + 8 * (int64_t)c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = widen(x.e[e]);
    if (a.res) {
        const Chunk<T> r = load_chunk(static_cast<const T*>(a.res) + row * a.ldr + 8 * (int64_t)c, n);
        Chunk<T> s;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s.e[e] = narrow<T>(h[e] + widen(r.e[e]));
            h[e] = widen(s.e[e]);
        }
        store_chunk(static_cast<T*>(a.sum) + row * a.ldsum + 8 * (int64_t)c, s, n);
    }
}

}  // namespace

// One row per team of wpr waves; with wpr == 1 a workgroup holds several rows.
template <class T, bool E4M3, int C>
__global__ void __launch_bounds__(64 * kNormMaxWaves)
norm_kernel(NormArgs a, int wpr, int rows_per_wg)
{
    __shared__ float red[kNormMaxWaves];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = rows_per_wg > 1 ? 0 : wv;
    // consecutive rows on one XCD: their scales, 4 bytes apart, then meet in its L2
    const int row = xcd_run(blockIdx.x, gridDim.x) * rows_per_wg + (rows_per_wg > 1 ? wv : 0);
    if (row >= a.M) return;  // whole waves, and only where no barrier follows (rows_per_wg > 1)

    float h[C][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + 64 * (wave + wpr * i);
        norm_input<T>(a, row, c, a.K - 8 * c, h[i]);
    }
    Chunk<T> w[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + 64 * (wave + wpr * i);
        if (8 * c < a.K) w[i] = load_chunk(static_cast<const T*>(a.weight) + 8 * c, a.K - 8 * c);
        else w[i] = Chunk<T>{};
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    }
    ss = team_sum(ss, red, wave, lane, wpr);
    const float r = 1.0f / sqrtf(ss / (float)a.K + a.eps);
    if (a.rstd && wave == 0 && lane == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + 64 * (wave + wpr * i);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[i][e] * r * widen(w[i].e[e]);
        norm_store<T, E4M3>(a, row, c, y, a.K - 8 * c);
    }
}

// Rows longer than a workgroup's registers (K > 32768): the row is read again, from the sum that
// this thread stored itself, or from x.
template <class T, bool E4M3>
__global__ void __launch_bounds__(64 * kNormMaxWaves)
norm_long_kernel(NormArgs a)
{
    __shared__ float red[kNormMaxWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = xcd_run(blockIdx.x, gridDim.x);
    const int chunks = (a.K + 7) >> 3;
    float ss = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += 64 * kNormMaxWaves) {
        float h[8];
        norm_input<T>(a, row, c, a.K - 8 * c, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(h[e], h[e], ss);
    }
    ss = team_sum(ss, red, wave, lane, kNormMaxWaves);
    const float r = 1.0f / sqrtf(ss / (float)a.K + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    const T* src = a.res ? static_cast<const T*>(a.sum) + row * a.ldsum : static_cast<const T*>(a.x) + row * a.ldx;
    // whole waves of chunks: every lane takes part in a group's maximum
    for (int c = threadIdx.x; c - lane < chunks; c += 64 * kNormMaxWaves) {
        const int n = a.K - 8 * c;
        float y[8];
        if (n > 0) {
            const Chunk<T> h = load_chunk(src + 8 * (int64_t)c, n);
            const Chunk<T> w = load_chunk(static_cast<const T*>(a.weight) + 8 * (int64_t)c, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = widen(h.e[e]) * r * widen(w.e[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.0f;
        }
        norm_store<T, E4M3>(a, row, c, y, n);
    }
}

// ---- backward ----------------------------------------------------------------
//
//   xhat = h r,  a = dy w,  dx = r (a - xhat mean(a xhat)) + dres,  dw = sum over rows of dy xhat
//
// One pass: a team of waves walks a run of rows, keeps w and its columns' dw in registers and loads the next
// row while the current one's mean is being reduced.  dw's partial sums, one per workgroup, are joined in a fixed order
// by a second kernel, so the result does not change from run to run; a single workgroup writes dw itself.  K past a
// team's registers walks column slices in a first pass for the mean.

namespace {

template <class T>
struct GradRow {
    Chunk<T> h, dy, dr;
};

}  // namespace

template <class T, int C, int WAVES, bool ONCE>
__global__ void __launch_bounds__(64 * WAVES)
norm_grad_kernel(NormGradArgs a, int wpr, int teams_per_wg)
{
    __shared__ float red[2][kNormMaxWaves];
    extern __shared__ float sum[];  // [teams_per_wg][K], with more than one
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int own = wv / wpr, wave = wv - own * wpr;
    const int team = blockIdx.x * teams_per_wg + own, teams = gridDim.x * teams_per_wg;
    const int per = a.M / teams, rem = a.M % teams;
    const int row0 = team * per + min(team, rem);
    const int row1 = row0 + per + (team < rem ? 1 : 0);
    const int last = row0 + per + (rem > 0 ? 1 : 0);  // teams that share barriers take as many turns

    Chunk<T> w[C];
    float dw[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + 64 * (wave + wpr * i);
        if (8 * c < a.K) w[i] = load_chunk(static_cast<const T*>(a.weight) + 8 * c, a.K - 8 * c);
        else w[i] = Chunk<T>{};
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    }
    auto fetch = [&](int row, GradRow<T> (&g)[C]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = lane + 64 * (wave + wpr * i);
            const int n = a.K - 8 * c;
            if (n > 0) {
                g[i].h = load_chunk<ONCE>(static_cast<const T*>(a.h) + row * a.ldh + 8 * c, n);
                g[i].dy = load_chunk<ONCE>(static_cast<const T*>(a.dy) + row * a.lddy + 8 * c, n);
                if (a.dres) g[i].dr = load_chunk<ONCE>(static_cast<const T*>(a.dres) + row * a.lddr + 8 * c, n);
            } else {
                g[i] = GradRow<T>{};
            }
        }
    };
    GradRow<T> cur[C], nxt[C];
    float r = 0.0f, rn = 0.0f;
    if (row0 < row1) {
        fetch(row0, cur);
        r = a.rstd[row0];
    }
    for (int row = row0; row < last; ++row) {
        if (row + 1 < row1) {
            fetch(row + 1, nxt);
            rn = a.rstd[row + 1];
        }
        float s = 0.0f;
        if (row < row1) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float dy = widen(cur[i].dy.e[e]);
                    const float xh = widen(cur[i].h.e[e]) * r;
                    s = fmaf(dy * widen(w[i].e[e]), xh, s);
                    dw[i][e] = fmaf(dy, xh, dw[i][e]);
                }
            }
        }
        // the two LDS rows alternate: a wave writes one only after the barrier of the row between
        const float mean = team_sum(s, &red[(row - row0) & 1][own * wpr], wave, lane, wpr) / (float)a.K;
        if (row >= row1) break;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = lane + 64 * (wave + wpr * i);
            const int n = a.K - 8 * c;
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = widen(cur[i].h.e[e]) * r;
                d[e] = r * (widen(cur[i].dy.e[e]) * widen(w[i].e[e]) - xh * mean);
                if (a.dres) d[e] += widen(cur[i].dr.e[e]);
            }
            if (n > 0) store_chunk(static_cast<T*>(a.dx) + row * a.lddx + 8 * c, narrow8<T>(d), n);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) cur[i] = nxt[i];
        r = rn;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + 64 * (wave + wpr * i);
        const int n = a.K - 8 * c;
        if (n <= 0) continue;
        if (teams_per_wg > 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e < n) sum[own * a.K + 8 * c + e] = dw[i][e];
            }
        } else if (teams == 1) {
            store_chunk(static_cast<T*>(a.dw) + 8 * c, narrow8<T>(dw[i]), n);
        } else {
            store_chunk(reinterpret_cast<Fp32*>(a.part) + (int64_t)team * a.K + 8 * c, narrow8<Fp32>(dw[i]), n);
        }
    }
    if (teams_per_wg == 1) return;
    __syncthreads();
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
        float s = sum[k];
        for (int t = 1; t < teams_per_wg; ++t) s += sum[t * a.K + k];
        if (gridDim.x == 1) static_cast<T*>(a.dw)[k] = narrow<T>(s);
        else a.part[(int64_t)blockIdx.x * a.K + k] = s;
    }
}

// K past a team's registers: dx row by row (the row read twice) ...
template <class T>
__global__ void __launch_bounds__(64 * kNormMaxWaves)
norm_grad_long_kernel(NormGradArgs a, int row_base)
{
    __shared__ float red[kNormMaxWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = row_base + blockIdx.x;
    const int chunks = (a.K + 7) >> 3;
    const T* h = static_cast<const T*>(a.h) + row * a.ldh;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* w = static_cast<const T*>(a.weight);
    const float r = a.rstd[row];
    float s = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += 64 * kNormMaxWaves) {
        const int n = a.K - 8 * c;
        const Chunk<T> ch = load_chunk(h + 8 * (int64_t)c, n), cy = load_chunk(dy + 8 * (int64_t)c, n),
                       cw = load_chunk(w + 8 * (int64_t)c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(widen(cy.e[e]) * widen(cw.e[e]), widen(ch.e[e]) * r, s);
    }
    const float mean = team_sum(s, red, wave, lane, kNormMaxWaves) / (float)a.K;
    for (int c = threadIdx.x; c < chunks; c += 64 * kNormMaxWaves) {
        const int n = a.K - 8 * c;
        const Chunk<T> ch = load_chunk(h + 8 * (int64_t)c, n), cy = load_chunk(dy + 8 * (int64_t)c, n),
                       cw = load_chunk(w + 8 * (int64_t)c, n);
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = r * (widen(cy.e[e]) * widen(cw.e[e]) - widen(ch.e[e]) * r * mean);
        if (a.dres) {
            const Chunk<T> cr = load_chunk(static_cast<const T*>(a.dres) + row * a.lddr + 8 * (int64_t)c, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] += widen(cr.e[e]);
        }
        store_chunk(static_cast<T*>(a.dx) + row * a.lddx + 8 * (int64_t)c, narrow8<T>(d), n);
    }
}

// ... and dw's partial sums by 2048 columns x a team's rows
template <class T>
__global__ void __launch_bounds__(256)
norm_grad_long_dw_kernel(NormGradArgs a, int teams)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    const int n = a.K - 8 * c;
    if (n <= 0) return;
    const int team = blockIdx.y;
    const int per = a.M / teams, rem = a.M % teams;
    const int row0 = team * per + min(team, rem);
    const int row1 = row0 + per + (team < rem ? 1 : 0);
    float dw[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int row = row0; row < row1; ++row) {
        const Chunk<T> ch = load_chunk(static_cast<const T*>(a.h) + row * a.ldh + 8 * (int64_t)c, n);
        const Chunk<T> cy = load_chunk(static_cast<const T*>(a.dy) + row * a.lddy + 8 * (int64_t)c, n);
        const float r = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = fmaf(widen(cy.e[e]), widen(ch.e[e]) * r, dw[e]);
    }
    store_chunk(reinterpret_cast<Fp32*>(a.part) + (int64_t)team * a.K + 8 * (int64_t)c, narrow8<Fp32>(dw), n);
}

// dw[k] = T(sum of the teams' partials, lanes of a column striding the teams, then a tree over the lanes); no
// teams: +0. 32 columns (a 128-byte line of a partial) x 32 lanes per column, the launch's from k_base on.
template <class T>
__global__ void __launch_bounds__(1024)
norm_grad_dw_kernel(const float* __restrict__ part, void* dw, int K, int teams, int k_base)
{
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, ln = threadIdx.x >> 5;
    const int k = k_base + blockIdx.x * 32 + col;
    float s = 0.0f;
    if (k < K) {
        // 8 loads in flight, those past the last team of the last team's value, which is not added
        for (int t = ln; t < teams; t += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)min(t + 32 * i, teams - 1) * K + k];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += t + 32 * i < teams ? v[i] : 0.0f;
        }
    }
    red[ln][col] = s;
    __syncthreads();
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1) {
        if (ln < step) red[ln][col] += red[ln + step][col];
        __syncthreads();
    }
    if (ln == 0 && k < K) static_cast<T*>(dw)[k] = narrow<T>(red[0][col]);
}

// ---- host ----------------------------------------------------------------------

namespace {

constexpr int kNormRows = 1 << 21;  // rows per launch: a grid holds fewer than 2^32 threads
constexpr int kGradColumns = 1 << 26;  // columns per launch of the join of dw, 32 threads each: likewise
constexpr int kNormMaxK = 64 * kNormMaxWaves * kNormMaxChunks * 8;  // a row in one workgroup's registers

// Waves per row and chunks per lane.  One chunk while the rows are too few to fill the card (a row then takes
// the fewest serial steps) and for 4-byte types; else two, which leaves fewer waves per barrier.  8192 x 5120
// bf16 with residual to e4m3: 59.4 us (4.96 TB/s; a copy reaches 5.2) with two, 65.7 with one, 69.3 with four;
// 8192 x 8192 fp32: 203 us with one, 219 with two.
struct RowShape {
    int wpr, chunks;
};
RowShape norm_shape(int M, int K, int size)
{
    const int need = (K + 511) / 512;  // waves at one chunk per lane
    int c = M >= 1024 && need > 1 && size == 2 ? 2 : 1;
    while ((need + c - 1) / c > kNormMaxWaves) c *= 2;
    return {(need + c - 1) / c, c};
}

// The backward holds three rows and their successors beside w and dw: one chunk per lane up to 8192 columns (at
// 4096, 118.5 us for 16384 rows against 137 with two, and 106 since its reads go past the caches), two above, where
// registers allow: 16-bit types only.
constexpr int kGradMaxK = 64 * kNormMaxWaves * 8;
int64_t grad_max_k(int dtype) { return dtype == GLU_DTYPE_FP32 ? kGradMaxK : 2 * kGradMaxK; }
// A few rows go to the teams of one workgroup and need no second launch: up to 2 a team, each some 1.8 us (3 x 780
// 3.9 us against 5.2, and 3 us less on the host).  Single waves, which share no barrier, are 16 to a workgroup and
// leave one partial sum for all: 3090 x 192 6.8 us against 12.0, 8192 x 512 12.5 against 21.7.  So do longer rows' teams
// where each has one row or two, pairs of waves up to four, though they wait for each other: 4096 x 1024 13.2 against
// 18.5, 1500 x 600 fp32 7.9 against 12.0, 6000 x 800 14.3 against 17.4; with more rows each that costs (1612 x 3392
// 24.0 against 18.1, 5000 x 1500 29.5 against 22.7), and with up to 256 teams, whose sums are quickly joined (203 x
// 2560: 7.7 against 6.7).  Else 16 waves per CU, all resident at once: at 16384
// x 4096 118.5 us (reads through the caches), against 132 at half and 119 at twice as many.
struct GradShape {
    int wpr, chunks, teams, grid;  // waves per row, chunks per lane, teams per workgroup
};
constexpr int kGradRows = 2;
GradShape grad_shape(int M, int K)
{
    const int need = (K + 511) / 512;
    if (need > kNormMaxWaves) {
        const int wpr = (need + 1) / 2, most = 4096 / wpr;
        return {wpr, 2, 1, M < most ? M : most};
    }
    const int fit = kNormMaxWaves / need;
    if (M <= kGradRows * fit) return {need, 1, M < fit ? M : fit, 1};
    const int most = 4096 / need;
    const int teams = M <= most ? M : M <= 2 * most ? (M + 1) / 2 : most;
    const int share = need == 1 || (teams > 256 && M <= (need == 2 ? 4 : 2) * teams) ? fit : 1;
    return {need, 1, share, (teams + share - 1) / share};
}

// partial sums of dw that a second kernel joins; 0: none
int grad_parts(int dtype, int M, int K)
{
    if (M < 1) return 0;
    if (K > grad_max_k(dtype)) return M < 64 ? M : 64;
    const GradShape p = grad_shape(M, K);
    return p.grid > 1 ? p.grid : 0;
}

// What the backward reads is dropped from the caches where they could not hold it for the next reader anyway: 16384
// x 4096 bf16 (403 MB) 113.9 -> 106.3 us; where they hold it that costs: 2048 x 4096 19.7 -> 22.3.
constexpr int64_t kLastLevelCache = 256 << 20;
using GradFn = void (*)(NormGradArgs, int, int);
template <class T, int C, int WAVES>
GradFn grad_kernel(bool once)
{
    if constexpr (sizeof(T) == 2) {
        if (once) return norm_grad_kernel<T, C, WAVES, true>;
    }
    return norm_grad_kernel<T, C, WAVES, false>;
}

template <class T, bool E4M3>
hipError_t norm_launch_t(const NormArgs& a, hipStream_t s)
{
    if (a.K > kNormMaxK) {
        hipLaunchKernelGGL((norm_long_kernel<T, E4M3>), dim3(a.M), dim3(64 * kNormMaxWaves), 0, s, a);
        return hipGetLastError();
    }
    const RowShape p = norm_shape(a.M, a.K, sizeof(T));
    const int rpw = p.wpr == 1 ? 4 : 1;
    const dim3 grid((unsigned)((a.M + rpw - 1) / rpw)), block(64 * p.wpr * rpw);
    switch (p.chunks) {
    case 1: hipLaunchKernelGGL((norm_kernel<T, E4M3, 1>), grid, block, 0, s, a, p.wpr, rpw); break;
    case 2: hipLaunchKernelGGL((norm_kernel<T, E4M3, 2>), grid, block, 0, s, a, p.wpr, rpw); break;
    default: hipLaunchKernelGGL((norm_kernel<T, E4M3, 4>), grid, block, 0, s, a, p.wpr, rpw); break;
    }
    return hipGetLastError();
}

template <class T>
hipError_t norm_grad_launch_t(int dtype, const NormGradArgs& a, hipStream_t s)
{
    const int parts = grad_parts(dtype, a.M, a.K);
    if (a.M > 0) {
        if (a.K > grad_max_k(dtype)) {
            for (int64_t row = 0; row < a.M; row += kNormRows) {
                const int rows = (int)(a.M - row < kNormRows ? a.M - row : kNormRows);
                hipLaunchKernelGGL((norm_grad_long_kernel<T>), dim3(rows), dim3(64 * kNormMaxWaves), 0, s, a,
                                   (int)row);
            }
            const int chunks = (a.K + 7) / 8;
            hipLaunchKernelGGL((norm_grad_long_dw_kernel<T>), dim3((chunks + 255) / 256, parts), dim3(256), 0, s, a,
                               parts);
        } else {
            const GradShape p = grad_shape(a.M, a.K);
            const int waves = p.wpr * p.teams;
            const bool once = sizeof(T) == 2 && (int64_t)a.M * a.K * 2 * (a.dres ? 3 : 2) > kLastLevelCache;
            const auto run = [&](auto kernel) {
                const size_t lds = p.teams > 1 ? (size_t)p.teams * a.K * 4 : 0;
                hipLaunchKernelGGL(kernel, dim3(p.grid), dim3(64 * waves), lds, s, a, p.wpr, p.teams);
            };
            if (p.chunks == 2) {
                if constexpr (sizeof(T) == 2) run(grad_kernel<T, 2, 16>(once));
            } else if (waves > 8) {
                run(grad_kernel<T, 1, 16>(once));
            } else {
                run(grad_kernel<T, 1, 8>(once));
            }
            if (parts == 0) return hipGetLastError();
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    for (int64_t k = 0; k < a.K; k += kGradColumns) {
        const int columns = (int)(a.K - k < kGradColumns ? a.K - k : kGradColumns);
        hipLaunchKernelGGL((norm_grad_dw_kernel<T>), dim3((columns + 31) / 32), dim3(1024), 0, s, a.part, a.dw, a.K,
                           parts, (int)k);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t norm_launch(int dtype, bool e4m3, const NormArgs& all, hipStream_t s)
{
    const int esize = dtype == GLU_DTYPE_FP32 ? 4 : 2;
    for (int64_t row = 0; row < all.M; row += kNormRows) {
        NormArgs a = all;
        a.M = (int)(all.M - row < kNormRows ? all.M - row : kNormRows);
        a.x = static_cast<const char*>(all.x) + row * all.ldx * esize;
        if (all.res) {
            a.res = static_cast<const char*>(all.res) + row * all.ldr * esize;
            a.sum = static_cast<char*>(all.sum) + row * all.ldsum * esize;
        }
        a.out = static_cast<char*>(all.out) + row * all.ldo * (e4m3 ? 1 : esize);
        if (e4m3) a.scale = all.scale + row;
        if (all.rstd) a.rstd = all.rstd + row;
        hipError_t e;
        switch (dtype) {
        case GLU_DTYPE_BF16: e = e4m3 ? norm_launch_t<Bf16, true>(a, s) : norm_launch_t<Bf16, false>(a, s); break;
        case GLU_DTYPE_FP16: e = e4m3 ? norm_launch_t<Fp16, true>(a, s) : norm_launch_t<Fp16, false>(a, s); break;
        default: e = e4m3 ? norm_launch_t<Fp32, true>(a, s) : norm_launch_t<Fp32, false>(a, s); break;
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t norm_grad_part_floats(int dtype, int M, int K)
{
    return (int64_t)grad_parts(dtype, M, K) * K;
}

hipError_t norm_grad_launch(int dtype, const NormGradArgs& a, hipStream_t s)
{
    switch (dtype) {
    case GLU_DTYPE_BF16: return norm_grad_launch_t<Bf16>(dtype, a, s);
    case GLU_DTYPE_FP16: return norm_grad_launch_t<Fp16>(dtype, a, s);
    default: return norm_grad_launch_t<Fp32>(dtype, a, s);
    }
}

}  // namespace glu
