// A mixture-of-experts GLU layer for a few tokens.
//
//   out[m] = sum over the experts e of row m of p_e down_e (silu(gate_e x[m]) * (up_e x[m]))
//
// Bound by the bytes of the experts that some row chose: each of their matrices is read once.  Three launches.  The
// first ranks the logits, one wave per row, and lists the active experts with their rows: a row's bit in a 64-bit
// mask per expert, so that the lists come out in order whatever order the waves ran in.  The second gives each active
// expert's gate and up, 16 rows of weights at a time, to a workgroup whose waves share the contraction.  The third gives 16
// rows of every active expert's down to a workgroup whose waves take experts in turn, and each wave adds what its experts
// give to rows of its own in LDS, which are summed in wave order at the end.
// The weights go from memory straight into matrix instructions as their 16 rows; the columns are rows of x, of
// which an expert of a small batch has one or two: the matrix unit has more than ten times the rate needed.
#include "../../include/glu_fp8.h"
#include "glu_mat16.h"
#include "glu_moe.h"

namespace glu {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kPerLane = kMaxExperts / 64;
constexpr int kUpThreads = 256;
constexpr int kUpWaves = kUpThreads / 64;
constexpr int kDownThreads = 512;
constexpr int kDownWaves = kDownThreads / 64;

// ---- routing -----------------------------------------------------------------------

// Order of logits as unsigned numbers: -inf (masked) is 0x007fffff, NaN is above all, and -0 equals +0.
__device__ __forceinline__ uint32_t order_of(float f)
{
    const uint32_t b = __float_as_uint(f + 0.0f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t kMasked = 0x007fffffu;

__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
}

template <class L>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(MoeArgs a)
{
    __shared__ uint32_t mask[kMaxExperts][2];  // rows of an expert
    __shared__ int first[kMaxExperts];
    __shared__ int sums[kRouteWaves][2];
    extern __shared__ int chosen[];            // [M][top] expert, or -1; then [M][top] its weight
    float* p = reinterpret_cast<float*>(chosen + a.M * a.top);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) mask[e][0] = mask[e][1] = 0u;
    __syncthreads();
    for (int m = wave; m < a.M; m += kRouteWaves) {
        const L* row = static_cast<const L*>(a.logits) + m * a.ldl;
        float f[kPerLane];
        uint32_t left = 0;  // which of this lane's logits are not taken yet
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = lane + 64 * i;
            f[i] = e < a.E ? widen(row[e]) : 0.0f;
            if (e < a.E && order_of(f[i]) != kMasked) left |= 1u << i;
        }
        float most = 0.0f, sum = 0.0f;
        for (int j = 0; j < a.top; ++j) {
            uint64_t best = 0;  // order, then the lowest expert
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                const uint64_t key = (uint64_t)order_of(f[i]) << 32 | (uint32_t)(kMaxExperts - lane - 64 * i);
                if ((left >> i & 1) && key > best) best = key;
            }
            best = wave_max(best);
            if (best == 0) {
                if (lane == 0) chosen[m * a.top + j] = -1;
                continue;
            }
            const int e = kMaxExperts - (int)(uint32_t)best;
            float l = 0.0f;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (lane + 64 * i == e) {
                    left &= ~(1u << i);
                    l = f[i];
                }
            }
            l = __shfl(l, e & 63);
            if (j == 0) most = l;
            const float w = expf(l - most);
            sum += w;
            if (lane == 0) {
                chosen[m * a.top + j] = e;
                p[m * a.top + j] = w;
                atomicOr(&mask[e][m >> 5], 1u << (m & 31));
            }
        }
        if (!a.normalize) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (lane + 64 * i < a.E) s += expf(f[i] - most);
            }
            sum = wave_sum(s);
        }
        for (int j = lane; j < a.top; j += 64) p[m * a.top + j] /= sum;
    }
    __syncthreads();
    // slots and the list of active experts, ascending
    const int e = threadIdx.x;
    const int count = e < a.E ? __popc(mask[e][0]) + __popc(mask[e][1]) : 0;
    int slots = count, actives = count > 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int s = __shfl_up(slots, d), n = __shfl_up(actives, d);
        if (lane >= d) {
            slots += s;
            actives += n;
        }
    }
    if (lane == 63) {
        sums[wave][0] = slots;
        sums[wave][1] = actives;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        slots += sums[w][0];
        actives += sums[w][1];
    }
    if (e < a.E) {
        first[e] = slots - count;
        if (count > 0) a.active[actives - 1] = Active{e, slots - count, count};
    }
    if (e == kRouteThreads - 1) *a.actives = actives;
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * a.top; i += kRouteThreads) {
        const int x = chosen[i], m = i / a.top;
        if (x < 0) continue;
        const uint32_t low = m < 32 ? (1u << m) - 1u : 0xffffffffu, high = m < 32 ? 0u : (1u << (m - 32)) - 1u;
        const int slot = first[x] + __popc(mask[x][0] & low) + __popc(mask[x][1] & high);
        a.row[slot] = m;
        a.weight[slot] = p[i];
    }
}

// ---- products ----------------------------------------------------------------------

struct Whole { static constexpr bool value = true; };
struct Part { static constexpr bool value = false; };

// 16 e4m3 numbers as two operands of T; every one of them is a number of T
template <class T>
__device__ __forceinline__ void widen16(raw4_t c, raw4_t (&v)[2])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (__is_same(T, Bf16)) {
            v[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false));
            v[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true));
        } else {
            v[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, false));
            v[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, true));
        }
    }
}

__device__ __forceinline__ raw4_t bytes16(const uint8_t* p, int n)
{
    if (n >= 16) return *reinterpret_cast<const u32x4_any*>(p);
    raw4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i < n) v[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
    return v;
}

// contraction per stage: a whole 128-byte line of each weight row
template <bool E8> constexpr int kStageCols = E8 ? 128 : 64;

// Stages s0, s0 + step, .. below s1 of NM products of 16 weight rows (this lane's at w[i]) with 16 TT rows of v (this lane's
// at v[t]), C columns.  sc[i]: the scales of the weight rows' block, one per 128 columns.
template <class T, bool E8, int NM, int TT>
__device__ __forceinline__ void products(const uint8_t* const (&w)[NM], const float* const (&sc)[NM], const T* const (&v)[TT],
                                         int C, int s0, int s1, int step, int q, f32x4 (&acc)[NM][TT])
{
    constexpr int SC = kStageCols<E8>;
    auto stage = [&](int s, auto tag) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(tag)::value;
        if constexpr (E8) {
            const int c = s * SC + 16 * q;
            raw4_t wv[NM][2], xv[TT][4];
#pragma unroll
            for (int i = 0; i < NM; ++i) {
#pragma unroll
                for (int h = 0; h < 2; ++h) wv[i][h] = WHOLE ? *reinterpret_cast<const u32x4_any*>(w[i] + c + 64 * h) : bytes16(w[i] + c + 64 * h, C - c - 64 * h);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int k = c + 64 * (h >> 1) + 8 * (h & 1);
                    xv[t][h] = WHOLE ? *reinterpret_cast<const u32x4_any*>(v[t] + k) : load8(v[t] + k, C - k);
                }
            }
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                raw4_t lo[2], hi[2];
                widen16<T>(wv[i][0], lo);
                widen16<T>(wv[i][1], hi);
                const float scale = sc[i][s];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
                    p = mfma16<T>(lo[0], xv[t][0], p);
                    p = mfma16<T>(lo[1], xv[t][1], p);
                    p = mfma16<T>(hi[0], xv[t][2], p);
                    p = mfma16<T>(hi[1], xv[t][3], p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][t][e] = fmaf(p[e], scale, acc[i][t][e]);
                }
            }
        } else {
            const int c = s * SC + 8 * q;
            raw4_t wv[NM][2], xv[TT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = c + 32 * h;
#pragma unroll
                for (int i = 0; i < NM; ++i) {
                    const T* p = reinterpret_cast<const T*>(w[i]) + k;
                    wv[i][h] = WHOLE ? *reinterpret_cast<const u32x4_any*>(p) : load8(p, C - k);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) xv[t][h] = WHOLE ? *reinterpret_cast<const u32x4_any*>(v[t] + k) : load8(v[t] + k, C - k);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < NM; ++i) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) acc[i][t] = mfma16<T>(wv[i][h], xv[t][h], acc[i][t]);
                }
            }
        }
    };
    const int whole = min(s1, C / SC);
    int s = s0;
#pragma unroll 4
    for (; s < whole; s += step) stage(s, Whole{});
    if (s < s1) stage(s, Part{});
}

// act[slot][n] = T(silu(gate x) * (up x)) of one active expert, 16 columns n
template <class T, bool E8, int TT>
__device__ __forceinline__ void gate_up(const MoeArgs& a, const Active& x, int n0, int t0, float (*red)[2][TT][256])
{
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int ES = E8 ? 1 : 2;
    const uint8_t* w[2];
    const float* sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = a.w[i].data + (x.expert * a.w[i].stack + min(n0 + i16, a.N - 1) * a.w[i].ld) * ES;
        sc[i] = E8 ? a.w[i].scale + x.expert * a.w[i].scale_stack + (n0 / kGroup) * a.w[i].scale_ld : nullptr;
    }
    const T* v[TT];
    f32x4 acc[2][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        v[t] = static_cast<const T*>(a.x) + a.row[x.first + min(t0 + 16 * t + i16, x.count - 1)] * a.ldx;
        acc[0][t] = acc[1][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int stages = (a.K + kStageCols<E8> - 1) / kStageCols<E8>;
    products<T, E8, 2, TT>(w, sc, v, a.K, wave, stages, kUpWaves, q, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int t = 0; t < TT; ++t) *reinterpret_cast<f32x4*>(&red[wave][i][t][4 * lane]) = acc[i][t];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < TT * 256; j += kUpThreads) {
        const int i = j & 15, c = j >> 4 & 15, t = j >> 8, s = t0 + 16 * t + c, n = n0 + i;
        if (s >= x.count || n >= a.N) continue;
        const int at = 4 * ((i >> 2) * 16 + c) + (i & 3);
        float g = red[0][0][t][at], u = red[0][1][t][at];
#pragma unroll
        for (int k = 1; k < kUpWaves; ++k) {
            g += red[k][0][t][at];
            u += red[k][1][t][at];
        }
        a.act[(x.first + s) * a.ld_act + n] = bits16<T>(silu_mul(g, u));
    }
    __syncthreads();
}

template <class T, bool E8>
__global__ void __launch_bounds__(kUpThreads) moe_up_kernel(MoeArgs a, int blocks)
{
    __shared__ float red[kUpWaves][2][4][256];
    const int j = blockIdx.x / blocks, n0 = (blockIdx.x - j * blocks) * 16;
    if (j >= *a.actives) return;
    const Active x = a.active[j];
    if (x.count <= 16) gate_up<T, E8, 1>(a, x, n0, 0, reinterpret_cast<float(*)[2][1][256]>(&red[0][0][0][0]));
    else gate_up<T, E8, 4>(a, x, n0, 0, red);
}

// out[m][c], 16 columns c, of the active experts that are this split's
template <class T, bool E8>
__global__ void __launch_bounds__(kDownThreads) moe_down_kernel(MoeArgs a, MoePlan p)
{
    extern __shared__ float sums[];  // [wave][M][16]
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = blockIdx.x * 16, split = blockIdx.y;
    float* mine = sums + wave * a.M * 16;
    for (int i = lane; i < a.M * 16; i += 64) mine[i] = 0.0f;
    __builtin_amdgcn_wave_barrier();  // a row's sums pass between the wave's lanes, in LDS order
    const int actives = *a.actives;
    const int stages = (a.N + kStageCols<E8> - 1) / kStageCols<E8>;
    const int per = (stages + p.parts - 1) / p.parts;
    constexpr int ES = E8 ? 1 : 2;
    for (int u = wave; ; u += kDownWaves) {
        const int j = u / p.parts * p.splits + split, part = u % p.parts;
        if (j >= actives) break;
        const Active x = a.active[j];
        const uint8_t* const w[1] = {a.w[2].data + (x.expert * a.w[2].stack + min(c0 + i16, a.K - 1) * a.w[2].ld) * ES};
        const float* const sc[1] = {E8 ? a.w[2].scale + x.expert * a.w[2].scale_stack + (c0 / kGroup) * a.w[2].scale_ld : nullptr};
        for (int t = 0; t < x.count; t += 16) {
            const int s = x.first + min(t + i16, x.count - 1);
            const T* const v[1] = {reinterpret_cast<const T*>(a.act) + s * a.ld_act};
            f32x4 acc[1][1] = {{{0.0f, 0.0f, 0.0f, 0.0f}}};
            products<T, E8, 1, 1>(w, sc, v, a.N, part * per, min(stages, (part + 1) * per), 1, q, acc);
            if (t + i16 < x.count) {
                float* to = mine + a.row[s] * 16 + 4 * q;
                const float weight = a.weight[s];
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e] = fmaf(weight, acc[0][0][e], to[e]);
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * 16; i += kDownThreads) {
        const int m = i >> 4, c = c0 + (i & 15);
        if (c >= a.K) continue;
        float v = sums[i];
#pragma unroll
        for (int k = 1; k < kDownWaves; ++k) v += sums[k * a.M * 16 + i];
        if (p.splits == 1) static_cast<T*>(a.out)[m * a.ldo + c] = narrow<T>(v);
        else a.part[((int64_t)split * a.M + m) * a.K + c] = v;
    }
}

template <class T>
__global__ void __launch_bounds__(256) moe_join_kernel(MoeArgs a, int splits)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)a.M * a.K;
    if (i >= n) return;
    float v = a.part[i];
    for (int s = 1; s < splits; ++s) v += a.part[s * n + i];
    static_cast<T*>(a.out)[i / a.K * a.ldo + i % a.K] = narrow<T>(v);
}

template <class T, bool E8>
hipError_t launch(int logits_dtype, const MoeArgs& a, const MoePlan& p, hipStream_t stream)
{
    const size_t lds = (size_t)a.M * a.top * 8;
    if (logits_dtype == GLU_DTYPE_FP32) {
        hipLaunchKernelGGL(moe_route_kernel<Fp32>, dim3(1), dim3(kRouteThreads), lds, stream, a);
    } else {
        hipLaunchKernelGGL(moe_route_kernel<T>, dim3(1), dim3(kRouteThreads), lds, stream, a);
    }
    const int most = a.M * a.top < a.E ? a.M * a.top : a.E;
    if (a.N > 0) {
        const int blocks = (a.N + 15) / 16;
        hipLaunchKernelGGL((moe_up_kernel<T, E8>), dim3((unsigned)(most * blocks)), dim3(kUpThreads), 0, stream, a, blocks);
    }
    hipLaunchKernelGGL((moe_down_kernel<T, E8>), dim3((a.K + 15) / 16, p.splits), dim3(kDownThreads),
                       (size_t)kDownWaves * a.M * 64, stream, a, p);
    if (p.splits > 1) {
        const int64_t n = (int64_t)a.M * a.K;
        hipLaunchKernelGGL(moe_join_kernel<T>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, a, p.splits);
    }
    return hipGetLastError();
}

}  // namespace

MoePlan moe_plan(int M, int K, int N, int E, int top, bool e4m3)
{
    const int most = M * top < E ? M * top : E, stages = (N + (e4m3 ? 127 : 63)) / (e4m3 ? 128 : 64);
    MoePlan p{1, 1};
    // every wave of a workgroup has something to do
    while (most * p.parts < kDownWaves && p.parts < stages) p.parts *= 2;
    // and workgroups fill the CUs twice
    const int blocks = (K + 15) / 16;
    while (blocks * p.splits < 512 && most * p.parts >= 2 * kDownWaves * p.splits && p.splits < 8) p.splits *= 2;
    return p;
}

hipError_t moe_launch(int dtype, int logits_dtype, bool e4m3, const MoeArgs& a, const MoePlan& p, hipStream_t stream)
{
    if (dtype == GLU_DTYPE_BF16) return e4m3 ? launch<Bf16, true>(logits_dtype, a, p, stream) : launch<Bf16, false>(logits_dtype, a, p, stream);
    return e4m3 ? launch<Fp16, true>(logits_dtype, a, p, stream) : launch<Fp16, false>(logits_dtype, a, p, stream);
}

}  // namespace glu
