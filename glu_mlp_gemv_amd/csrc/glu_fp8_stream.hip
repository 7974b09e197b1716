// Block-scaled e4m3 products for few rows of x: weights go from memory
// straight into matrix instructions, each read once.
//
// Bound by the weights' bytes.  A workgroup owns R weight rows (of each matrix) and its waves take
// K-blocks in turn, so that together they read R rows of consecutive 128-byte blocks.  With R = 16 the 16 rows of the
// matrix instruction's A operand are 16 weight rows; with R = 8 or 4 they are the same rows at 2 or 4 neighbouring
// K-blocks, the B operand holds x at those K-blocks in the same order, and of the 16 x 16 results the
// blocks on the diagonal are the products wanted.  That gives narrow matrices 2 and 4 times the workgroups, for x of
// up to R rows.  The waves' sums meet in LDS in wave order.  The products run on the bf16 unit, whose sums are fp32
// (glu_fp8_mfma.h).
#include "glu_fp8_mfma.h"

namespace glu {

namespace {

constexpr int kStreamMaxWaves = 16;

template <bool ANY>
__device__ __forceinline__ raw4_t chunk16(const uint8_t* row, int64_t off, int K)
{
    raw4_t z = {0u, 0u, 0u, 0u};
    if constexpr (ANY) {
        if (off + 16 <= K) return *reinterpret_cast<const u32x4_any*>(row + off);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (off + i < K) w[i >> 2] |= (uint32_t)row[off + i] << (8 * (i & 3));
        }
        return raw4_t{w[0], w[1], w[2], w[3]};
    } else {
        // K is a multiple of 16: the chunk is inside or outside as a whole; outside it is read at 0 and dropped
        const bool in = off < K;
        const raw4_t v = *reinterpret_cast<const raw4_t*>(row + (in ? off : 0));
        return in ? v : z;
    }
}

}  // namespace

template <int NM, int R, bool ANY>
__global__ void __launch_bounds__(64 * kStreamMaxWaves)
fp8_stream_kernel(Fp8Args a, int waves, int splits, int nbn, int m_base)
{
    constexpr int S = 16 / R;          // K-blocks per instruction
    constexpr int U = NM == 2 ? 2 : 4;  // steps whose loads are issued together
    extern __shared__ float red[];     // [waves][NM][4][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    const int sel = i16 / R;  // this lane's K-block within the instruction (both operands)
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
    const int stride = waves * splits;
    for (int s0 = split * waves + wave; s0 < steps; s0 += U * stride) {
        raw4_t wv[U][NM][2], xv[U][2];
        float sc[U][NM];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * stride;
            if (s >= steps) break;
            const int kb = S * s + sel;
            const int64_t off = (int64_t)kb * kGroup + 16 * q;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                wv[u][m][0] = chunk16<ANY>(wr[m], off, a.K);
                wv[u][m][1] = chunk16<ANY>(wr[m], off + 64, a.K);
            }
            const int kbs = min(kb, KB - 1);
            xv[u][0] = chunk16<ANY>(xr, off, a.K);
            xv[u][1] = chunk16<ANY>(xr, off + 64, a.K);
            const float sx = xs[kbs * a.sxg];
#pragma unroll
            for (int m = 0; m < NM; ++m) sc[u][m] = sx * ws[m][kbs];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * stride >= steps) break;
            const Wide x = widen32(xv[u][0], xv[u][1]);
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const f32x4 p = mfma_wide(widen32(wv[u][m][0], wv[u][m][1]), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][e] = fmaf(p[e], sc[u][m], acc[m][e]);
            }
        }
    }

#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave * NM + m) * 4 + e) * 64 + lane] = acc[m][e];
    }
    __syncthreads();
    // one output a thread: weight row r, row j of x; its sums are D[sel R + r][sel R + j] of every wave
    for (int idx = threadIdx.x; idx < R * R; idx += 64 * waves) {
        const int r = idx % R, j = idx / R;
        const int n = n0 + r, row = m0 + j;
        if (n >= a.N || row >= a.M) continue;
        float v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            v[m] = 0.0f;
            for (int w = 0; w < waves; ++w) {
#pragma unroll
                for (int b = 0; b < S; ++b) {
                    const int i = b * R + r;
                    v[m] += red[((w * NM + m) * 4 + (i & 3)) * 64 + (i >> 2) * 16 + b * R + j];
                }
            }
        }
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
StreamFn pick_stream(const StreamConfig& c)
{
    if (c.any) return c.rows == 16 ? fp8_stream_kernel<NM, 16, true> : nullptr;
    if (c.rows == 4) return fp8_stream_kernel<NM, 4, false>;
    if (c.rows == 8) return fp8_stream_kernel<NM, 8, false>;
    return c.rows == 16 ? fp8_stream_kernel<NM, 16, false> : nullptr;
}

size_t stream_lds(int mats, const StreamConfig& c) { return (size_t)c.waves * mats * 1024; }

}  // namespace

bool fp8_stream_supported(int mats, const StreamConfig& c, int M)
{
    if (c.waves < 1 || c.waves > kStreamMaxWaves || c.splits < 1) return false;
    if ((mats == 1 ? pick_stream<1>(c) : pick_stream<2>(c)) == nullptr) return false;
    return c.rows == 16 || M <= c.rows;
}

hipError_t fp8_stream_launch(int mats, const StreamConfig& c, const Fp8Args& a, hipStream_t stream)
{
    const StreamFn f = mats == 1 ? pick_stream<1>(c) : pick_stream<2>(c);
    const int rows_x = c.rows;
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
