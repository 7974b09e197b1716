// Conversions to e4m3 with scales: activations with one scale per row and 128
// columns, weights with one per block of 128 x 128; and the end of the products
// whose partial sums are joined outside their kernel.
//
//   s = max(amax |v| / 448, 2^-126)      q = e4m3(v / s)
//
// One pass, bound by memory: a lane holds chunks of 8 values, 16 lanes one group of
// 128 columns, whose maximum is a DPP reduction.  Measured: a weight of 17408 x 5120 bf16 in 52 us, 5.1 TB/s (a
// copy of 1 GiB reaches 5.2); 77 rows of 4096 in 2.8 us, which is a launch.
#include "../../include/glu_fp8.h"
#include "glu_fp8_device.h"
#include "glu_quantize.h"

namespace glu {

namespace {

constexpr int kRowsPerWave = 4;  // rows a wave takes through its 512 columns, all loaded before the first is used

// sources of 8 values at (row, chunk c), the first n of them present
template <class T>
struct RowSource {
    const T* x;
    int64_t ld;
    __device__ __forceinline__ void load(int row, int c, int n, float (&v)[8]) const
    {
        const Chunk<T> ch = load_chunk(x + row * ld + 8 * (int64_t)c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = widen(ch.e[e]);
    }
};

struct PartSource {
    const float* part;
    int64_t plane;  // M * N
    int N, splits, mats;
    __device__ __forceinline__ void sum(const float* p, int64_t step, int n, float (&v)[8]) const
    {
        if (splits == 0) {  // an empty contraction
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            return;
        }
        const Chunk<Fp32> first = load_chunk(reinterpret_cast<const Fp32*>(p), n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = first.e[e].v;
        for (int s = 1; s < splits; ++s) {
            const Chunk<Fp32> ch = load_chunk(reinterpret_cast<const Fp32*>(p + s * step), n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += ch.e[e].v;
        }
    }
    __device__ __forceinline__ void load(int row, int c, int n, float (&v)[8]) const
    {
        const float* p = part + (int64_t)row * N + 8 * (int64_t)c;
        if (mats == 2) {
            float u[8];
            sum(p, 2 * plane, n, v);
            sum(p + plane, 2 * plane, n, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = silu_mul(v[e], u[e]);
        } else {
            sum(p, plane, n, v);
        }
    }
};

// 4 waves; a wave takes 512 columns (4 groups) of `R` rows, the launch's first of which is row_base
template <class Src, class Out, int R>
__global__ void __launch_bounds__(256)
convert_rows_kernel(Src src, void* out, int64_t ldo, float* scale, int64_t lds, int M, int K, int col_blocks,
                    int row_base)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rb = blockIdx.x / col_blocks, cb = blockIdx.x - rb * col_blocks;
    const int c = cb * 64 + lane;
    const int n = K - 8 * c;
    const int row0 = row_base + (rb * 4 + wave) * R;
    float v[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (n > 0 && row0 + i < M) {
            src.load(row0 + i, c, n, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = row0 + i;
        const bool live = n > 0 && row < M;
        if constexpr (sizeof(Out) == 1) {
            const Scale s = scale_of(max16(abs_max8(v[i])));
            if (live) {
                store_e4m3x8(static_cast<uint8_t*>(out) + row * ldo + 8 * (int64_t)c, e4m3x8(v[i], s), n);
                if ((lane & 15) == 0) scale[(c >> 4) * lds + row] = s.s;
            }
        } else {
            if (live) store_chunk(static_cast<Out*>(out) + row * ldo + 8 * (int64_t)c, narrow8<Out>(v[i]), n);
        }
    }
}

// A workgroup of 256 holds one 128 x 128 block in registers: 16 lanes a row, 16 rows a step, 8 steps.
template <class T>
__global__ void __launch_bounds__(256)
quantize_blocks_kernel(const T* __restrict__ w, int64_t ldw, uint8_t* __restrict__ q, int64_t ldq,
                       float* __restrict__ scale, int64_t lds, int N, int K, int col_blocks)
{
    __shared__ uint32_t red[4];
    const int rb = blockIdx.x / col_blocks, cb = blockIdx.x - rb * col_blocks;
    const int c = cb * 16 + (threadIdx.x & 15);
    const int n = K - 8 * c;
    const int row0 = rb * kGroup + (threadIdx.x >> 4);
    Chunk<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + 16 * i;
        if (n > 0 && row < N) v[i] = load_chunk(w + row * ldw + 8 * (int64_t)c, n);
        else v[i] = Chunk<T>{};
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, abs_bits(widen(v[i].e[e])));
    }
    m = max16(m);
    m = max(m, (uint32_t)__builtin_amdgcn_ds_swizzle((int)m, 0x401F));  // lane ^ 16
    auto pr = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max((uint32_t)pr[0], (uint32_t)pr[1]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    const Scale s = scale_of(max(max(red[0], red[1]), max(red[2], red[3])));
    if (threadIdx.x == 0) scale[rb * lds + cb] = s.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + 16 * i;
        if (n > 0 && row < N) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = widen(v[i].e[e]);
            store_e4m3x8(q + row * ldq + 8 * (int64_t)c, e4m3x8(f, s), n);
        }
    }
}

// A lane copies 16 bytes of each of 4 rows, all loaded before the first is stored.
__global__ void __launch_bounds__(256)
copy_rows_kernel(const uint8_t* __restrict__ x, int64_t ldx, uint8_t* __restrict__ out, int kp, int rows, int K,
                 int col_blocks, int row_base)
{
    const int rb = blockIdx.x / col_blocks, cb = blockIdx.x - rb * col_blocks;
    const int off = 16 * (cb * 64 + (threadIdx.x & 63));
    const int row0 = row_base + (rb * 4 + (threadIdx.x >> 6)) * kRowsPerWave;
    if (off >= kp) return;
    raw4_t v[kRowsPerWave];
#pragma unroll
    for (int i = 0; i < kRowsPerWave; ++i) {
        const uint8_t* p = x + min(row0 + i, rows - 1) * ldx + off;
        if (off + 16 <= K) {
            v[i] = *reinterpret_cast<const u32x4_any*>(p);
        } else {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int b = 0; b < 16; ++b) {
                if (off + b < K) w[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
            }
            v[i] = raw4_t{w[0], w[1], w[2], w[3]};
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsPerWave; ++i) {
        if (row0 + i < rows) *reinterpret_cast<raw4_t*>(out + (row0 + i) * (int64_t)kp + off) = v[i];
    }
}

// Launches over `rows` rows, `per_block` a workgroup of 256 threads and col_blocks workgroups wide, with the workgroups and
// the first row of each: a grid holds fewer than 2^32 threads, which takes more than one launch from 2^28 rows on.
template <class F>
void by_rows(int rows, int per_block, int col_blocks, const F& launch)
{
    const int64_t blocks = ((int64_t)rows + per_block - 1) / per_block, fit = 0xffffffffLL / 256 / col_blocks;
    for (int64_t b = 0; b < blocks; b += fit) {
        launch(dim3((unsigned)((blocks - b < fit ? blocks - b : fit) * col_blocks)), (int)(b * per_block));
    }
}

// rows per wave: one while the rows would not fill the card otherwise
template <class Out, class Src>
hipError_t convert_rows(const Src& src, void* out, int64_t ldo, float* scale, int64_t lds, int M, int K,
                        hipStream_t stream)
{
    const int col_blocks = (K + 511) / 512;
    if (((int64_t)M + 4 * kRowsPerWave - 1) / (4 * kRowsPerWave) * col_blocks >= 1024) {
        by_rows(M, 4 * kRowsPerWave, col_blocks, [&](dim3 grid, int row) {
            hipLaunchKernelGGL((convert_rows_kernel<Src, Out, kRowsPerWave>), grid, dim3(256), 0, stream, src, out, ldo,
                               scale, lds, M, K, col_blocks, row);
        });
    } else {
        by_rows(M, 4, col_blocks, [&](dim3 grid, int row) {
            hipLaunchKernelGGL((convert_rows_kernel<Src, Out, 1>), grid, dim3(256), 0, stream, src, out, ldo, scale,
                               lds, M, K, col_blocks, row);
        });
    }
    return hipGetLastError();
}

template <class T>
hipError_t blocks_t(const void* w, int64_t ldw, uint8_t* q, int64_t ldq, float* scale, int64_t lds, int N, int K,
                    hipStream_t stream)
{
    const int col_blocks = (K + kGroup - 1) / kGroup, row_blocks = (N + kGroup - 1) / kGroup;
    hipLaunchKernelGGL((quantize_blocks_kernel<T>), dim3((unsigned)(col_blocks * row_blocks)), dim3(256), 0, stream,
                       static_cast<const T*>(w), ldw, q, ldq, scale, lds, N, K, col_blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t quantize_rows_launch(int dtype, const void* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale,
                                int64_t lds, int M, int K, hipStream_t stream)
{
    const auto run = [&](auto src) { return convert_rows<uint8_t>(src, q, ldq, scale, lds, M, K, stream); };
    switch (dtype) {
    case GLU_DTYPE_BF16: return run(RowSource<Bf16>{static_cast<const Bf16*>(x), ldx});
    case GLU_DTYPE_FP16: return run(RowSource<Fp16>{static_cast<const Fp16*>(x), ldx});
    default: return run(RowSource<Fp32>{static_cast<const Fp32*>(x), ldx});
    }
}

hipError_t quantize_blocks_launch(int dtype, const void* w, int64_t ldw, uint8_t* q, int64_t ldq, float* scale,
                                  int64_t lds, int N, int K, hipStream_t stream)
{
    switch (dtype) {
    case GLU_DTYPE_BF16: return blocks_t<Bf16>(w, ldw, q, ldq, scale, lds, N, K, stream);
    case GLU_DTYPE_FP16: return blocks_t<Fp16>(w, ldw, q, ldq, scale, lds, N, K, stream);
    default: return blocks_t<Fp32>(w, ldw, q, ldq, scale, lds, N, K, stream);
    }
}

hipError_t copy_rows_launch(const uint8_t* x, int64_t ldx, uint8_t* out, int kp, int rows, int K, hipStream_t stream)
{
    const int col_blocks = (kp + 1023) / 1024;
    by_rows(rows, 4 * kRowsPerWave, col_blocks, [&](dim3 grid, int row) {
        hipLaunchKernelGGL(copy_rows_kernel, grid, dim3(256), 0, stream, x, ldx, out, kp, rows, K, col_blocks, row);
    });
    return hipGetLastError();
}

hipError_t finish_launch(int out_dtype, const FinishArgs& a, hipStream_t stream)
{
    const PartSource src{a.part, (int64_t)a.M * a.N, a.N, a.splits, a.mats};
    switch (out_dtype) {
    case GLU_DTYPE_BF16: return convert_rows<Bf16>(src, a.out, a.ldo, a.scale, a.lds, a.M, a.N, stream);
    case GLU_DTYPE_FP16: return convert_rows<Fp16>(src, a.out, a.ldo, a.scale, a.lds, a.M, a.N, stream);
    case GLU_DTYPE_FP32: return convert_rows<Fp32>(src, a.out, a.ldo, a.scale, a.lds, a.M, a.N, stream);
    default: return convert_rows<uint8_t>(src, a.out, a.ldo, a.scale, a.lds, a.M, a.N, stream);
    }
}

}  // namespace glu
