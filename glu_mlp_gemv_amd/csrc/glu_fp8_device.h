// Device helpers of the norm and e4m3 kernels: element types, chunk loads of 8
// at any element alignment, group maxima and the conversion to scaled e4m3.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "glu_device.h"

namespace glu {

constexpr int kGroup = 128;             // columns (and weight rows) that share a scale
constexpr float kE4m3Max = 448.0f;      // largest finite e4m3
constexpr float kScaleMin = 0x1p-126f;  // smallest scale: an all-zero group keeps finite quotients

struct Bf16 { uint16_t bits; };
struct Fp16 { _Float16 v; };
struct Fp32 { float v; };

// 16- and 8-byte vectors at the alignment of one element: global memory takes them as one access
// at any address, so a row of odd length needs no other code than its last chunk
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t raw4_t __attribute__((ext_vector_type(4)));
typedef uint32_t raw2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float widen(Bf16 e) { return bf16_to_f32(e.bits); }
__device__ __forceinline__ float widen(Fp16 e) { return (float)e.v; }
__device__ __forceinline__ float widen(Fp32 e) { return e.v; }

// fp32 to the element type, to nearest even (NaN stays NaN, overflow goes to infinity)
template <class T> __device__ __forceinline__ T narrow(float f);
template <> __device__ __forceinline__ Bf16 narrow<Bf16>(float f)
{
    return Bf16{__builtin_bit_cast(uint16_t, (__bf16)f)};
}
template <> __device__ __forceinline__ Fp16 narrow<Fp16>(float f) { return Fp16{(_Float16)f}; }
template <> __device__ __forceinline__ Fp32 narrow<Fp32>(float f) { return Fp32{f}; }

// A chunk: 8 consecutive elements of a row, as stored.
template <class T> struct Chunk { T e[8]; };

// The chunk at p, of which the first n (>= 1) elements exist; the others read as +0.  ONCE: whole chunks of 2-byte
// types are not kept in the caches (a 4-byte type's two halves would each fetch the line).
template <bool ONCE = false, class T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p, int n)
{
    Chunk<T> c;
    if (n >= 8) {
        if constexpr (sizeof(T) == 2) {
            const u32x4_any* p4 = reinterpret_cast<const u32x4_any*>(p);
            const raw4_t v = ONCE ? (raw4_t)__builtin_nontemporal_load(p4) : (raw4_t)*p4;
            __builtin_memcpy(&c, &v, 16);
        } else {
            const raw4_t a = reinterpret_cast<const u32x4_any*>(p)[0];
            const raw4_t b = reinterpret_cast<const u32x4_any*>(p)[1];
            __builtin_memcpy(&c, &a, 16);
            __builtin_memcpy(reinterpret_cast<char*>(&c) + 16, &b, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c.e[i] = i < n ? p[i] : T{};
    }
    return c;
}

template <class T>
__device__ __forceinline__ void store_chunk(T* p, const Chunk<T>& c, int n)
{
    if (n >= 8) {
        if constexpr (sizeof(T) == 2) {
            raw4_t v;
            __builtin_memcpy(&v, &c, 16);
            *reinterpret_cast<u32x4_any*>(p) = v;
        } else {
            raw4_t a, b;
            __builtin_memcpy(&a, &c, 16);
            __builtin_memcpy(&b, reinterpret_cast<const char*>(&c) + 16, 16);
            reinterpret_cast<u32x4_any*>(p)[0] = a;
            reinterpret_cast<u32x4_any*>(p)[1] = b;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) p[i] = c.e[i];
        }
    }
}

template <class T>
__device__ __forceinline__ Chunk<T> narrow8(const float (&v)[8])
{
    Chunk<T> c;
#pragma unroll
    for (int i = 0; i < 8; ++i) c.e[i] = narrow<T>(v[i]);
    return c;
}

// |v| maxima are taken on the bit patterns: they order as the magnitudes do, and a NaN, which is
// above infinity there, is kept instead of being dropped as the float maximum drops it.
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t abs_max8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false));
}

// maximum over the lane's aligned group of 16, in every lane of it (16 chunks of 8 = one group of 128)
__device__ __forceinline__ uint32_t max16(uint32_t x)
{
    x = dpp_max<0xB1>(x);   // lane ^ 1
    x = dpp_max<0x4E>(x);   // lane ^ 2
    x = dpp_max<0x141>(x);  // the other quad of 8
    return dpp_max<0x140>(x);  // the other half of 16
}

// The scale of a group whose largest magnitude has these bits, and its reciprocal: both IEEE
// divisions.  An infinite group maximum gives an infinite scale, a NaN a NaN.
struct Scale {
    float s;    // as stored
    float div;  // the divisor of the remainder step: 1 where s is infinite, so that no 0 * inf arises
    float r;    // 1 / s
};
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits)
{
    Scale c;
    const float s = __uint_as_float(amax_bits) / kE4m3Max;
    c.s = s < kScaleMin ? kScaleMin : s;  // NaN compares false and stays
    c.r = 1.0f / c.s;
    c.div = c.s == __builtin_inff() ? 1.0f : c.s;
    return c;
}

// v / s: the product with the reciprocal and one remainder step, which gives the correctly rounded
// quotient in three operations instead of the division's ten or so.  The step matters: where v / s lies on a
// border between two e4m3 values a last-bit difference would change the stored value.
__device__ __forceinline__ float quotient(float v, const Scale& c)
{
    const float q = v * c.r;
    return fmaf(-fmaf(q, c.div, -v), c.r, q);  // in these signs a zero keeps its own
}

// 8 quotients as e4m3 (nearest even; |v / s| <= 448 (1 + 2^-23), which rounds to at most 448)
__device__ __forceinline__ raw2_t e4m3x8(const float (&v)[8], const Scale& c)
{
    raw2_t w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int d = 0;
        d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * h], c), quotient(v[4 * h + 1], c), d, false);
        d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * h + 2], c), quotient(v[4 * h + 3], c), d, true);
        w[h] = (uint32_t)d;
    }
    return w;
}

__device__ __forceinline__ void store_e4m3x8(uint8_t* p, raw2_t w, int n)
{
    if (n >= 8) {
        *reinterpret_cast<u32x2_any*>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        }
    }
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32.  exp(-g) = 2^t with t = -g log2(e), and the rounding
// error of t, up to 2^-18 of the result at |g| = 80, is put back to first order; the hardware's
// 2^t and reciprocal are each good to one unit in the last place.  Against the library's exp and the IEEE
// division this takes a third of the instructions, which counts in an epilogue of tens of millions of values.
// Where 2^t or g is infinite the correction would be NaN and is left out: g = +inf gives +inf * u, -inf
// gives NaN (as -inf / inf does), and g < -88 gives -0 * u (the definition: below 2^-119 |u|).
__device__ __forceinline__ float silu_mul(float g, float u)
{
    constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.69314718055994530942f;
    const float t = -g * kLog2e;
    const float err = fminf(fmaxf(fmaf(-g, kLog2e, -t) - g * kLog2eLow, -1.0f), 1.0f);
    const float p = __builtin_amdgcn_exp2f(t);
    const float e = p == __builtin_inff() ? p : fmaf(p, err * kLn2, p);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// block -> work item so that each XCD, which gets every eighth workgroup, has one run of consecutive items
__device__ __forceinline__ int xcd_run(int bid, int n)
{
    const int per = n >> 3, rem = n & 7, xcd = bid & 7, slot = bid >> 3;
    return (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + slot;
}

}  // namespace glu
