// Block-scaled e4m3 products for few rows of x: weights go from memory
// straight into matrix instructions, each read once.
//
// Bound by the weights' bytes.  A workgroup owns R weight rows (of each matrix) and its waves take K-blocks in
// turn, so that together they read R rows of consecutive 128-byte blocks.  With R = 16 the 16 rows of the matrix
// instruction's A operand are 16 weight rows; with R = 4 they are the same 4 rows at 4 neighbouring K-blocks,
// the B operand holds x at those K-blocks in the same order, and of the 16 x 16 results the blocks on the
// diagonal are the products wanted.  That gives 4 times the workgroups, each reading 4 times as far along a row,
// for x of up to 4 rows: at one row 8.1 us against 8.9 (K = 9216 N = 2560), dual 35.0 against 37.4 (K = 5120 N
// = 17408, 178 MB); at 8 rows, which 8 weight rows would serve, 16 is the faster (12.8 against 14.7 us at K =
// 12288 N = 4096).  The pair of matrices, read past the caches' keeping, takes whole 128-byte lines per load for
// it: dual K = 5120 N = 17408 32.3 -> 29.2 us, K = 2560 N = 9216 11.6 -> 11.0 (weights from memory; 11.0 either way
// where they stay in the last-level cache).  One matrix keeps half lines, cached: K = 17408 N = 5120 18.6 us
// against 18.0, but 16.8 against 17.6 from the last-level cache.  Longer-lived workgroups that keep x in registers and
// load one run of rows ahead were slower (one row, K = 9216 N = 2560: 9.6 us).  The waves' sums meet in LDS in
// wave order.  The products run on the bf16 unit, whose sums are
// fp32 (glu_fp8_mfma.h).
#include "glu_fp8_mfma.h"

namespace glu {

namespace {

constexpr int kStreamMaxWaves = 8;

// Layout of the rows: whole K-blocks in whole instructions; chunks of 16 bytes; or any bytes
enum { kWhole, kChunks, kBytes };

template <bool ONCE>
__device__ __forceinline__ raw4_t read16(const uint8_t* p)
{
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const raw4_t*>(p));
    else return *reinterpret_cast<const raw4_t*>(p);
}

// ONCE: data that nothing reads again
template <int MODE, bool ONCE>
__device__ __forceinline__ raw4_t chunk16(const uint8_t* row, int64_t off, int K)
{
    if constexpr (MODE == kWhole) {
        return read16<ONCE>(row + off);
    } else if constexpr (MODE == kChunks) {
        // K is a multiple of 16: the chunk is inside or outside as a whole; outside it is read at 0 and dropped
        const bool in = off < K;
        const raw4_t v = read16<ONCE>(row + (in ? off : 0));
        return in ? v : raw4_t{0u, 0u, 0u, 0u};
    } else {
        if (off + 16 <= K) return *reinterpret_cast<const u32x4_any*>(row + off);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (off + i < K) w[i >> 2] |= (uint32_t)row[off + i] << (8 * (i & 3));
        }
        return raw4_t{w[0], w[1], w[2], w[3]};
    }
}

}  // namespace

template <int NM, int R, int MODE>
__global__ void __launch_bounds__(64 * kStreamMaxWaves)
fp8_stream_kernel(Fp8Args a, int waves, int splits, int nbn, int m_base)
{
    constexpr int S = 16 / R;               // K-blocks per instruction
    constexpr int U = MODE == kBytes ? 1 : NM == 2 ? 2 : 4;  // steps whose loads are in flight
    extern __shared__ float red[];          // [waves][NM][4][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    // LINES: the two 16-byte chunks of a lane are of K-blocks sel / 2 and sel / 2 + 2, at half sel % 2, so that 8
    // neighbouring lanes load a whole 128-byte line; each chunk has its own product and scale then
    constexpr bool LINES = NM == 2 && R == 4;
    constexpr int SC = LINES ? 2 : 1;  // scales per step and operand
    const int sel = i16 / R;  // this lane's place on the diagonal (both operands): a K-block, or half of two
    const int mb = blockIdx.x / nbn;
    const int n0 = (blockIdx.x - mb * nbn) * R;
    const int m0 = m_base + mb * 16;
    const int split = blockIdx.y;
    const int KB = (a.K + kGroup - 1) / kGroup;
    const int steps = (KB + S - 1) / S;

    const uint8_t* wr[NM];
    const float* ws[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        wr[m] = a.w[m] + (int64_t)min(n0 + i16 % R, a.N - 1) * a.ldw[m];
        ws[m] = a.sw[m] + (int64_t)(n0 / kGroup) * a.ldsw[m];
    }
    const int xrow = min(m0 + i16 % R, a.M - 1);
    const uint8_t* xr = a.x + (int64_t)xrow * a.ldx;
    const float* xs = a.sx + (int64_t)xrow * a.sxm;

    f32x4 acc[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    raw4_t wv[U][NM][2], xv[U][2];
    float sc[U][NM + 1][SC];
    auto load = [&](int u, int s) __attribute__((always_inline)) {
        const int kb = S * s + (LINES ? sel >> 1 : sel);
        const int64_t off = (int64_t)kb * kGroup + 16 * q + (LINES ? 64 * (sel & 1) : 0);
        constexpr int APART = LINES ? 2 * kGroup : 64;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            wv[u][m][0] = chunk16<MODE, LINES>(wr[m], off, a.K);
            wv[u][m][1] = chunk16<MODE, LINES>(wr[m], off + APART, a.K);
        }
        xv[u][0] = chunk16<MODE, false>(xr, off, a.K);
        xv[u][1] = chunk16<MODE, false>(xr, off + APART, a.K);
#pragma unroll
        for (int c = 0; c < SC; ++c) {
            const int kbs = min(kb + 2 * c, KB - 1);
#pragma unroll
            for (int m = 0; m < NM; ++m) sc[u][m][c] = ws[m][kbs];
            sc[u][NM][c] = xs[kbs * a.sxg];
        }
    };
    auto use = [&](int u, int s) __attribute__((always_inline)) {
        // past the last K-block the operands are zeros, and so is the scale: the last block's, which was read, may be
        // infinite (chosen here and not where it is read: a branch there waits for the loads, K = 2704 N = 9216 one
        // row 6.6 -> 8.1 us)
        const int kb = S * s + (LINES ? sel >> 1 : sel);
        auto scale_at = [&](int m, int c) __attribute__((always_inline)) {
            const float scale = sc[u][m][c] * sc[u][NM][c];
            return MODE == kWhole || S == 1 || kb + 2 * c < KB ? scale : 0.0f;
        };
        const Wide x = widen32(xv[u][0], xv[u][1]);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const Wide w = widen32(wv[u][m][0], wv[u][m][1]);
            if constexpr (LINES) {
                f32x4 p[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // the two products' instructions in turn
                    const int c = i & 1, v = 2 * c + (i >> 1);
                    p[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[v], x.v[v], p[c], 0, 0, 0);
                }
#pragma unroll
                for (int c = 0; c < SC; ++c) {
                    const float scale = scale_at(m, c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][e] = fmaf(p[c][e], scale, acc[m][e]);
                }
            } else {
                const f32x4 p = mfma_wide(w, x);
                const float scale = scale_at(m, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][e] = fmaf(p[e], scale, acc[m][e]);
            }
        }
    };
    // a ring of U steps: one is refilled as soon as it is used, so that U - 1 remain in flight
    const int stride = waves * splits;
    int s = split * waves + wave;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (s + u * stride < steps) load(u, s + u * stride);
    }
    for (; s + (2 * U - 1) * stride < steps; s += U * stride) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            use(u, s + u * stride);
            load(u, s + (u + U) * stride);
        }
    }
    for (; s < steps; s += U * stride) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u * stride < steps) use(u, s + u * stride);
            if (s + (u + U) * stride < steps) load(u, s + (u + U) * stride);
        }
    }

#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave * NM + m) * 4 + e) * 64 + lane] = acc[m][e];
    }
    __syncthreads();
    // weight row r and row j of x, for matrix m: D[sel R + r][sel R + j] of every wave
    auto sum = [&](int m, int r, int j) __attribute__((always_inline)) {
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) {
#pragma unroll
            for (int b = 0; b < S; ++b) {
                const int i = b * R + r;
                v += red[((w * NM + m) * 4 + (i & 3)) * 64 + (i >> 2) * 16 + b * R + j];
            }
        }
        return v;
    };
    for (int idx = threadIdx.x; idx < R * R; idx += 64 * waves) {  // one output a thread
        const int r = idx % R, j = idx / R;
        const int n = n0 + r, row = m0 + j;
        if (n >= a.N || row >= a.M) continue;
        float v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) v[m] = sum(m, r, j);
        if (a.out_dtype == kPartial) {
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                a.part[((int64_t)(split * NM + m) * a.M + row) * a.N + n] = v[m];
            }
        } else {
            store_value(a.out, a.out_dtype, row * a.ldo + n, NM == 2 ? silu_mul(v[0], v[NM - 1]) : v[0]);
        }
    }
}

namespace {

using StreamFn = void (*)(Fp8Args, int, int, int, int);

template <int NM>
StreamFn pick_stream(const StreamConfig& c, int K)
{
    if (c.any) return c.rows == 16 ? fp8_stream_kernel<NM, 16, kBytes> : nullptr;
    const bool whole = c.rows > 0 && K % (kGroup * 16 / c.rows) == 0;
    if (c.rows == 4) return whole ? fp8_stream_kernel<NM, 4, kWhole> : fp8_stream_kernel<NM, 4, kChunks>;
    if (c.rows == 16) return whole ? fp8_stream_kernel<NM, 16, kWhole> : fp8_stream_kernel<NM, 16, kChunks>;
    return nullptr;
}

size_t stream_lds(int mats, const StreamConfig& c) { return (size_t)c.waves * mats * 1024; }

}  // namespace

bool fp8_stream_supported(const StreamConfig& c, int M)
{
    if (c.waves < 1 || c.waves > kStreamMaxWaves || c.splits < 1) return false;
    if (c.rows != 16 && (c.any || c.rows != 4)) return false;
    return c.rows == 16 || M <= c.rows;
}

hipError_t fp8_stream_launch(int mats, const StreamConfig& c, const Fp8Args& a, hipStream_t stream)
{
    const StreamFn f = mats == 1 ? pick_stream<1>(c, a.K) : pick_stream<2>(c, a.K);
    const int rows_x = c.rows;  // rows of x per workgroup
    const int nbn = (int)(((int64_t)a.N + c.rows - 1) / c.rows);
    // slices of x's rows that keep a grid below 2^32 threads (one launch for anything but vast outputs)
    const int64_t tiles = ((int64_t)a.M + rows_x - 1) / rows_x;
    const int64_t fit = 0xffffffffLL / (64 * c.waves) / nbn / c.splits;
    for (int64_t t = 0; t < tiles; t += fit) {
        const int64_t n = tiles - t < fit ? tiles - t : fit;
        hipLaunchKernelGGL(f, dim3((unsigned)(nbn * n), (unsigned)c.splits), dim3(64 * c.waves), stream_lds(mats, c),
                           stream, a, c.waves, c.splits, nbn, (int)(t * rows_x));
    }
    return hipGetLastError();
}

}  // namespace glu
