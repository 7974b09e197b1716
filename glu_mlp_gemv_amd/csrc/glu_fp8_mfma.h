// Pieces shared by the block-scaled e4m3 products.
#pragma once

#include "../../include/glu_fp8.h"
#include "glu_fp8.h"
#include "glu_fp8_device.h"

namespace glu {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// One 16 x 16 x 128 product of e4m3 operands, which is exactly one K-block: lane l supplies 32 bytes of
// row l % 16 of either operand and receives D[4 (l / 16) + e][l % 16].  Which 32 of the block's 128
// bytes a lane supplies is free as long as both operands agree: it takes 16-byte chunks l / 16 and l / 16 + 4.
//
// mfma_e4m3 is the matrix unit's 8-bit rate.  Its sums are not quite fp32: within 8 neighbouring products the
// unit aligns to the largest and drops what lies 13 to 14 bits below it, before adding the eighths in fp32
// (seen on exact inputs; the K = 32 form does the same).  On normally distributed operands that is 2^-19 of the
// sum of magnitudes, without bias, some 2^-16 of a result: nothing beside the rounding to 16 or 8 bits that
// follows, but too coarse for fp32 results and for the fp32 scales of an e4m3 result, which take mfma_wide.  The
// unit-scale form: the hardware's own scales are powers of two per 32 values and cannot hold these.
__device__ __forceinline__ f32x4 mfma_e4m3(raw4_t a0, raw4_t a1, raw4_t b0, raw4_t b1)
{
    i32x8_t a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = (int)a0[i];
        a[4 + i] = (int)a1[i];
        b[i] = (int)b0[i];
        b[4 + i] = (int)b1[i];
    }
    const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The same product with sums good to fp32: every e4m3 value is a bf16 value, and the bf16 unit's products and
// sums keep 24 bits.  A quarter of the rate and 2 conversions per 4 bytes, which a kernel bound by its weights'
// bytes has to spare: at one row of x the matrix and vector units are below a fifth busy.
struct Wide { bf16x8 v[4]; };
__device__ __forceinline__ Wide widen32(raw4_t c0, raw4_t c1)
{
    Wide w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t d = i < 4 ? c0[i] : c1[i - 4];
        const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false);
        const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true);
        w.v[i >> 1][4 * (i & 1) + 0] = lo[0];
        w.v[i >> 1][4 * (i & 1) + 1] = lo[1];
        w.v[i >> 1][4 * (i & 1) + 2] = hi[0];
        w.v[i >> 1][4 * (i & 1) + 3] = hi[1];
    }
    return w;
}
__device__ __forceinline__ f32x4 mfma_wide(const Wide& a, const Wide& b)
{
    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
    return d;
}

// weight scales are uniform over a wave: scalar loads
__device__ __forceinline__ float scalar_load(const float* p)
{
    return *(const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

__device__ __forceinline__ void store_value(void* out, int dtype, int64_t at, float v)
{
    if (dtype == GLU_DTYPE_BF16) static_cast<Bf16*>(out)[at] = narrow<Bf16>(v);
    else if (dtype == GLU_DTYPE_FP16) static_cast<Fp16*>(out)[at] = narrow<Fp16>(v);
    else static_cast<float*>(out)[at] = v;
}

// 4 consecutive values of a row, the first n of them
__device__ __forceinline__ void store_values4(void* out, int dtype, int64_t at, f32x4 v, int n)
{
    if (n >= 4) {
        if (dtype == GLU_DTYPE_FP32) {
            raw4_t w;
            __builtin_memcpy(&w, &v, 16);
            *reinterpret_cast<u32x4_any*>(static_cast<float*>(out) + at) = w;
        } else {
            raw2_t w;
            if (dtype == GLU_DTYPE_BF16) {
                const Bf16 t[4] = {narrow<Bf16>(v[0]), narrow<Bf16>(v[1]), narrow<Bf16>(v[2]), narrow<Bf16>(v[3])};
                __builtin_memcpy(&w, t, 8);
            } else {
                const Fp16 t[4] = {narrow<Fp16>(v[0]), narrow<Fp16>(v[1]), narrow<Fp16>(v[2]), narrow<Fp16>(v[3])};
                __builtin_memcpy(&w, t, 8);
            }
            *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(out) + at) = w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e < n) store_value(out, dtype, at + e, v[e]);
        }
    }
}

}  // namespace glu
