// Matrix-unit operands of 16-bit types, shared by the adapter and expert kernels.
//
// v_mfma_f32_16x16x32: lane l supplies 8 numbers of row l % 16 of either operand, those at places 8 (l / 16) .. + 7
// of the contraction, and receives D[4 (l / 16) + e][l % 16].
#pragma once

#include "glu_fp8_device.h"

namespace glu {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ f32x4 mfma16(raw4_t a, raw4_t b, f32x4 c)
{
    if constexpr (sizeof(T) == 2 && __is_same(T, Bf16)) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    }
}

template <class T> __device__ __forceinline__ uint16_t bits16(float f)
{
    return __builtin_bit_cast(uint16_t, narrow<T>(f));
}

// 8 numbers at p, of which the first n exist (n may be negative); the others read as +0
template <class T>
__device__ __forceinline__ raw4_t load8(const T* p, int n)
{
    if (n >= 8) return *reinterpret_cast<const u32x4_any*>(p);
    const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
    raw4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < n) v[i >> 1] |= (uint32_t)u[i] << (16 * (i & 1));
    }
    return v;
}

// the largest of the wave's numbers, in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = max16(x);
    x = max(x, (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 0x401F));  // lane ^ 16
    auto pr = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return max(pr[0], pr[1]);
}

// A number of 32 bits as two of 16: its rounding and the rounding of what that left (nothing where it is not finite,
// which would be inf - inf).
template <class T>
__device__ __forceinline__ void split16(float f, uint16_t& hi, uint16_t& lo)
{
    const T h = narrow<T>(f);
    const float w = widen(h);
    hi = __builtin_bit_cast(uint16_t, h);
    lo = abs_bits(w) < 0x7f800000u ? bits16<T>(f - w) : (uint16_t)0;
}

// The bits of |f|, or 0 where f is not finite: what the largest of numbers is taken from that share a power of two.
__device__ __forceinline__ uint32_t finite_bits(float f)
{
    const uint32_t b = abs_bits(f);
    return b < 0x7f800000u ? b : 0u;
}

// fp16 has too small a range for any fp32 number: numbers whose largest finite magnitude has these bits are multiplied by a
// power of two that brings it to 2^14 .. 2^15, which leaves infinities what they are, and the sums by its reciprocal.  Both are
// normal numbers; 1 where the largest is zero, and for bf16, which has fp32's range.
struct Pow2 { float up, down; };
template <class T>
__device__ __forceinline__ Pow2 pow2_for(uint32_t amax)
{
    if (__is_same(T, Bf16) || amax == 0) return Pow2{1.0f, 1.0f};
    const int e = min(268 - (int)(amax >> 23), 253);
    return Pow2{__uint_as_float((uint32_t)e << 23), __uint_as_float((uint32_t)(254 - e) << 23)};
}

// W (1, 2 or 4) neighbouring columns of 8 rows as W operands of 8 numbers each, one column's 8 rows.  row(i): the
// address of the first of the columns in row i; n: how many of the columns exist (the others read as +0).
template <class T, int W, class Row>
__device__ __forceinline__ void load_columns(Row row, int n, raw4_t (&f)[W])
{
    if constexpr (W == 1) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t a = n > 0 ? *reinterpret_cast<const uint16_t*>(row(2 * h)) : 0u;
            const uint32_t b = n > 0 ? *reinterpret_cast<const uint16_t*>(row(2 * h + 1)) : 0u;
            f[0][h] = a | b << 16;
        }
    } else {
        typedef uint32_t __attribute__((aligned(1))) u32_any;
        uint32_t v[8][W / 2];
        if (n >= W) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (W == 2) {
                    v[i][0] = *reinterpret_cast<const u32_any*>(row(i));
                } else {
                    const raw2_t d = *reinterpret_cast<const u32x2_any*>(row(i));
                    v[i][0] = d[0];
                    v[i][1] = d[1];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(row(i));
#pragma unroll
                for (int d = 0; d < W / 2; ++d) {
                    v[i][d] = (2 * d < n ? (uint32_t)p[2 * d] : 0u) | (2 * d + 1 < n ? (uint32_t)p[2 * d + 1] << 16 : 0u);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int d = 0; d < W / 2; ++d) {
                f[2 * d][h] = __builtin_amdgcn_perm(v[2 * h + 1][d], v[2 * h][d], 0x05040100u);
                f[2 * d + 1][h] = __builtin_amdgcn_perm(v[2 * h + 1][d], v[2 * h][d], 0x07060302u);
            }
        }
    }
}

// which of dword h of such an operand belong to its first `rows` rows
__device__ __forceinline__ uint32_t first_rows_mask(int h, int rows)
{
    return (2 * h < rows ? 0xffffu : 0u) | (2 * h + 1 < rows ? 0xffff0000u : 0u);
}

}  // namespace glu
