// Dropout with a residual: out = residual + (draw >= drop ? x c : 0), the draws 16-bit pieces of Philox4x32-10.
//
// Bound by memory, if the generator is cheap enough: ten rounds of two 32 x 32 -> 64 bit products give eight draws, so
// a chunk of 8 numbers costs 20 wide multiplications, at a quarter of the vector rate, and some 60 other instructions.
// Twice that, with a draw of 32 bits per number, would take longer than memory.  16384 x 4096 bf16: 47 us, 5.7 TB/s.
#include "../../include/glu_fp8.h"
#include "glu_dropout.h"
#include "glu_fp8_device.h"

namespace glu {

namespace {

constexpr int kThreads = 256;

struct Draws { uint32_t w[4]; };  // draw i: half i % 2 of word i / 2

__device__ __forceinline__ Draws philox(uint32_t c0, uint32_t c1, uint64_t offset, uint64_t seed)
{
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)q;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Draws{{c0, c1, c2, c3}};
}

template <class T>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutArgs a, int chunks, int64_t total)
{
    const uint64_t seed = a.seed_at ? *a.seed_at : a.seed;
    for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int m = (int)(id / chunks), c = (int)(id - (int64_t)m * chunks);
        const int n = min(8, a.K - 8 * c);
        const Chunk<T> x = load_chunk(static_cast<const T*>(a.x) + m * a.ldx + 8 * (int64_t)c, n);
        Chunk<T> r{};
        if (a.res) r = load_chunk(static_cast<const T*>(a.res) + m * a.ldr + 8 * (int64_t)c, n);
        const Draws d = philox((uint32_t)c, (uint32_t)m, a.offset, seed);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t draw = e & 1 ? d.w[e >> 1] >> 16 : d.w[e >> 1] & 0xffffu;
            const float kept = draw >= a.drop ? widen(x.e[e]) * a.scale : 0.0f;
            v[e] = a.res ? widen(r.e[e]) + kept : kept;
        }
        store_chunk(static_cast<T*>(a.out) + m * a.ldo + 8 * (int64_t)c, narrow8<T>(v), n);
    }
}

}  // namespace

hipError_t dropout_launch(int dtype, const DropoutArgs& a, hipStream_t stream)
{
    const int chunks = (a.K + 7) / 8;
    const int64_t total = (int64_t)a.M * chunks, blocks = (total + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
    if (dtype == GLU_DTYPE_BF16) hipLaunchKernelGGL(dropout_kernel<Bf16>, grid, dim3(kThreads), 0, stream, a, chunks, total);
    else if (dtype == GLU_DTYPE_FP16) hipLaunchKernelGGL(dropout_kernel<Fp16>, grid, dim3(kThreads), 0, stream, a, chunks, total);
    else hipLaunchKernelGGL(dropout_kernel<Fp32>, grid, dim3(kThreads), 0, stream, a, chunks, total);
    return hipGetLastError();
}

}  // namespace glu
