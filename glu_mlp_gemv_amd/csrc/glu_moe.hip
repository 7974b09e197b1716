// A mixture-of-experts GLU layer for a few tokens.
//
//   out[m] = sum over the experts e of row m of p_e down_e (silu(gate_e x[m]) * (up_e x[m]))
//
// Bound by the bytes of the experts that some row chose: each of their matrices is read once, down of more than 8 rows of an
// expert again from the caches.  Three launches, or two for up to 4 rows, and a join where the third is cut.  The first ranks
// the logits, one wave per row, and lists the active experts with their rows: a row's bit in a 64-bit mask per expert, so
// that the lists come out in order whatever order the waves ran in.  The second gives each active
// expert's gate and up, 16 rows of weights at a time, to a workgroup whose waves share the contraction.  The third gives 16
// rows of every active expert's down to a workgroup whose waves take experts in turn, and each wave adds what its experts
// give to rows of its own in LDS, which are summed in wave order at the end.
// The weights go from memory straight into matrix instructions as their 16 rows; the columns are rows of x, of
// which an expert of a small batch has one or two: the matrix unit has more than ten times the rate needed.  37 rows, K =
// 4096 N = 768, 8 of 128 experts, bf16: 9 + 249 + 143 us, 5.9 and 5.1 TB/s; 6 rows, N = 1536, e4m3: 6 + 103 + 61 us, 5.0 and
// 4.3 TB/s; one row, K = 2560 N = 1024, 8 of 64: 19 + 12 us, 4.4 and 3.4 TB/s with a launch's ramp.
#include "../../include/glu_fp8.h"
#include "glu_mat16.h"
#include "glu_moe.h"

namespace glu {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;
constexpr int kRoutedRows = 4;
constexpr int kUpThreads = 256;
constexpr int kUpWaves = kUpThreads / 64;

// ---- routing -----------------------------------------------------------------------

// Order of logits as unsigned numbers, above 0: NaN is above all, -0 equals +0, and -inf, which masks an expert, is 0.
__device__ __forceinline__ uint32_t order_of(float f)
{
    const uint32_t b = __float_as_uint(f + 0.0f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return b == 0xff800000u ? 0u : b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t order)
{
    return __uint_as_float(order ^ (order >> 31 ? 0x80000000u : 0xffffffffu));
}

// What a workgroup of THREADS knows of the rows' experts, in LDS
template <int THREADS>
struct Routing {
    uint32_t mask[kMaxExperts][2];  // rows of an expert
    int first[kMaxExperts];         // its first slot
    int sums[THREADS / 64][2];
};

// Ranks the logits, a wave per row, and lists the active experts with their rows.  chosen [M][top] and p [M][top]: LDS;
// active, row and weight may be in LDS too.  PER: logits per lane.  Returns how many experts are active.
template <int THREADS, int PER, class L>
__device__ __forceinline__ int route(const MoeArgs& a, Routing<THREADS>& r, int* chosen, float* p, Active* active, int* row,
                                     float* weight)
{
    constexpr int WAVES = THREADS / 64, EACH = kMaxExperts / THREADS;  // experts per thread
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int e = threadIdx.x; e < a.E; e += THREADS) r.mask[e][0] = r.mask[e][1] = 0u;
    __syncthreads();
    L next[PER];  // the logits of the wave's next row
    auto load = [&](int m) __attribute__((always_inline)) {
        const L* logits = static_cast<const L*>(a.logits) + m * a.ldl;
#pragma unroll
        for (int i = 0; i < PER; ++i) next[i] = logits[min(lane + 64 * i, a.E - 1)];
    };
    if (wave < a.M) load(wave);
    for (int m = wave; m < a.M; m += WAVES) {
        uint32_t key[PER], all[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = all[i] = lane + 64 * i < a.E ? order_of(widen(next[i])) : 0u;
        if (m + WAVES < a.M) load(m + WAVES);
        uint32_t best = 0;  // lane j: the j-th of the row
        int expert = -1;
        for (int j = 0; j < a.top; ++j) {
            uint32_t most = key[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) most = max(most, key[i]);
            most = wave_max(most);
            if (most == 0) break;
            int e = -1;  // of equal ones the lowest
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint64_t b = __ballot(key[i] == most);
                if (e < 0 && b) e = 64 * i + __builtin_ctzll(b);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) key[i] = e == lane + 64 * i ? 0u : key[i];
            if (lane == j) {
                best = most;
                expert = e;
            }
        }
        const float top = logit_of(__builtin_amdgcn_readfirstlane(best));
        float w = expert >= 0 ? expf(logit_of(best) - top) : 0.0f, sum = w;
        if (!a.normalize) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += all[i] ? expf(logit_of(all[i]) - top) : 0.0f;
        }
        sum = wave_sum(sum);
        if (lane < a.top) {
            chosen[m * a.top + lane] = expert;
            p[m * a.top + lane] = w / sum;
            if (expert >= 0) atomicOr(&r.mask[expert][m >> 5], 1u << (m & 31));
        }
    }
    __syncthreads();
    // slots and the list of active experts, ascending
    const int e0 = threadIdx.x * EACH;
    int count[EACH], slots = 0, actives = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        count[i] = e0 + i < a.E ? __popc(r.mask[e0 + i][0]) + __popc(r.mask[e0 + i][1]) : 0;
        slots += count[i];
        actives += count[i] > 0;
    }
    const int my_slots = slots, my_actives = actives;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int s = __shfl_up(slots, d), n = __shfl_up(actives, d);
        if (lane >= d) {
            slots += s;
            actives += n;
        }
    }
    if (lane == 63) {
        r.sums[wave][0] = slots;
        r.sums[wave][1] = actives;
    }
    __syncthreads();
    slots -= my_slots;
    actives -= my_actives;
    int total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (w < wave) {
            slots += r.sums[w][0];
            actives += r.sums[w][1];
        }
        total += r.sums[w][1];
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (e0 + i < a.E) r.first[e0 + i] = slots;
        if (count[i] > 0) active[actives++] = Active{e0 + i, slots, count[i]};
        slots += count[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * a.top; i += THREADS) {
        const int x = chosen[i], m = i / a.top;
        if (x < 0) continue;
        const uint32_t low = m < 32 ? (1u << m) - 1u : 0xffffffffu, high = m < 32 ? 0u : (1u << (m - 32)) - 1u;
        const int slot = r.first[x] + __popc(r.mask[x][0] & low) + __popc(r.mask[x][1] & high);
        row[slot] = m;
        weight[slot] = p[i];
    }
    return total;
}

template <class L, int PER>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(MoeArgs a)
{
    __shared__ Routing<kRouteThreads> r;
    extern __shared__ int chosen[];  // [M][top] experts, then weights
    const int n = route<kRouteThreads, PER, L>(a, r, chosen, reinterpret_cast<float*>(chosen + a.M * a.top), a.active, a.row,
                                               a.weight);
    if (threadIdx.x == 0) *a.actives = n;
}

// ---- products ----------------------------------------------------------------------

struct Whole { static constexpr bool value = true; };
struct Part { static constexpr bool value = false; };

// The type of an activation's two numbers.  fp16's range is too small for any fp32 number: behind e4m3 weights, which
// are numbers of bf16 too, they are bf16; behind fp16 weights they are fp16 times a power of two (kScaled) of 16 columns,
// whose products are summed apart and multiplied by its reciprocal.
template <class T, bool E8> struct Act { using type = T; };
template <> struct Act<Fp16, true> { using type = Bf16; };
template <class T, bool E8> constexpr bool kScaled = __is_same(T, Fp16) && !E8;

// Those 16 columns are an instruction of 16 places of lanes that read 8 neighbours each: number i of group g (n0 = 16 g)
__device__ __forceinline__ int scaled_column(int n0, int i) { return (n0 & ~31) + 8 * (i >> 2) + (n0 >> 2 & 4) + (i & 3); }
// Whether a workgroup has anything to do (a group's factor is written even if its columns are all past N)
template <class T, bool E8>
__device__ __forceinline__ bool has_columns(int n0, int N) { return (kScaled<T, E8> ? n0 & ~31 : n0) < N; }

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

// numbers 4 h .. + 3 of eight
template <int H>
__device__ __forceinline__ f16x4_t four_of(raw4_t v)
{
    return __builtin_bit_cast(f16x4_t, raw2_t{v[2 * H], v[2 * H + 1]});
}

// Stages s0, s0 + step, .. below s1 of NM products of 16 weight rows (this lane's at w[i]) with 16 TT rows of v (this lane's
// at v[t]), C columns.  sc[i]: the scales of the weight rows' block, one per 128 columns.  With S places along the columns
// a stage is S times as long, and this lane's rows are at `place` of it.  SCALED: f[t] are the factors of v[t]'s groups of 16
// columns, four per stage.  U > 1: so many stages are read ahead.
template <class T, bool E8, int NM, int TT, int S, int U = 1, bool SCALED = false>
__device__ __forceinline__ void products(const uint8_t* const (&w)[NM], const float* const (&sc)[NM], const T* const (&v)[TT],
                                         int C, int s0, int s1, int step, int q, int place, f32x4 (&acc)[NM][TT],
                                         const float* const (&f)[TT])
{
    constexpr int SC = kStageCols<E8>, XH = E8 ? 4 : 2;
    raw4_t wv[U][NM][2], xv[U][TT][XH];
    f32x4 by[U][TT];
    auto load = [&](int u, int s, auto tag) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(tag)::value;
        const int c = (s * S + place) * SC + (E8 ? 16 : 8) * q;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = c + (E8 ? 64 : 32) * h;
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                const uint8_t* p = w[i] + (E8 ? k : 2 * k);
                if constexpr (WHOLE) wv[u][i][h] = *reinterpret_cast<const u32x4_any*>(p);
                else if constexpr (E8) wv[u][i][h] = bytes16(p, C - k);
                else wv[u][i][h] = load8(reinterpret_cast<const T*>(p), C - k);
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
#pragma unroll
            for (int h = 0; h < XH; ++h) {
                const int k = c + (E8 ? 64 * (h >> 1) + 8 * (h & 1) : 32 * h);
                xv[u][t][h] = WHOLE ? *reinterpret_cast<const u32x4_any*>(v[t] + k) : load8(v[t] + k, C - k);
            }
            if constexpr (SCALED) {
                by[u][t] = *reinterpret_cast<const f32x4*>(f[t] + 4 * (WHOLE ? s * S + place : min(s * S + place, (C - 1) / SC)));
                if constexpr (!WHOLE) {  // past the last group operands are zeros and factors are whatever memory holds
                    const int left = C - (s * S + place) * SC;
                    const f32x4 b = by[u][t];
                    by[u][t] = f32x4{left > 0 ? b[0] : 0.0f, left > 0 ? b[1] : 0.0f, left > 32 ? b[2] : 0.0f, left > 32 ? b[3] : 0.0f};
                }
            }
        }
    };
    auto use = [&](int u, int s, auto tag) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(tag)::value;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            if constexpr (E8) {
                raw4_t lo[2], hi[2];
                widen16<T>(wv[u][i][0], lo);
                widen16<T>(wv[u][i][1], hi);
                float scale = sc[i][S == 1 || WHOLE ? s * S + place : min(s * S + place, (C - 1) / kGroup)];
                // places past the last block hold zeros, and so does the scale: the last one, which was read, may be infinite
                if (S > 1 && !WHOLE && (s * S + place) * SC >= C) scale = 0.0f;
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
                    p = mfma16<T>(lo[0], xv[u][t][0], p);
                    p = mfma16<T>(lo[1], xv[u][t][1], p);
                    p = mfma16<T>(hi[0], xv[u][t][2], p);
                    p = mfma16<T>(hi[1], xv[u][t][3], p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][t][e] = fmaf(p[e], scale, acc[i][t][e]);
                }
            } else if constexpr (SCALED) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                    f32x4 p[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        p[2 * h] = __builtin_amdgcn_mfma_f32_16x16x16f16(four_of<0>(wv[u][i][h]), four_of<0>(xv[u][t][h]), zero, 0, 0, 0);
                        p[2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x16f16(four_of<1>(wv[u][i][h]), four_of<1>(xv[u][t][h]), zero, 0, 0, 0);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) acc[i][t][e] = fmaf(p[g][e], by[u][t][g], acc[i][t][e]);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) acc[i][t] = mfma16<T>(wv[u][i][h], xv[u][t][h], acc[i][t]);
                }
            }
        }
    };
    const int whole = min(s1, C / (SC * S));
    int s = s0;
    if constexpr (U == 1) {
#pragma unroll 4
        for (; s < whole; s += step) {
            load(0, s, Whole{});
            use(0, s, Whole{});
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u * step < whole) load(u, s + u * step, Whole{});
        }
        while (s < whole) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s >= whole) break;
                use(u, s, Whole{});
                if (s + U * step < whole) load(u, s + U * step, Whole{});
                s += step;
            }
        }
    }
    if (s < s1) {
        load(0, s, Part{});
        use(0, s, Part{});
    }
}

// act[slot][..][n] = silu(gate x) * (up x) of one active expert, 16 columns n, as two 16-bit numbers: rounded once to T a
// result would be 1.4 times as far off as by its own rounding alone.
template <class T, bool E8, int TT>
__device__ __forceinline__ void gate_up(const MoeArgs& a, const int* row, const Active& x, int n0, int t0,
                                        float (*red)[2][TT][256])
{
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int ES = E8 ? 1 : 2;
    const uint8_t* w[2];
    const float* sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = kScaled<T, E8> ? scaled_column(n0, i16) : n0 + i16;
        w[i] = a.w[i].data + (x.expert * a.w[i].stack + min(n, a.N - 1) * a.w[i].ld) * ES;
        sc[i] = E8 ? a.w[i].scale + x.expert * a.w[i].scale_stack + (n0 / kGroup) * a.w[i].scale_ld : nullptr;
    }
    const T* v[TT];
    f32x4 acc[2][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        v[t] = static_cast<const T*>(a.x) + row[x.first + min(t0 + 16 * t + i16, x.count - 1)] * a.ldx;
        acc[0][t] = acc[1][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int stages = (a.K + kStageCols<E8> - 1) / kStageCols<E8>;
    const float* const none[TT] = {};
    products<T, E8, 2, TT, 1>(w, sc, v, a.K, wave, stages, kUpWaves, q, 0, acc, none);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int t = 0; t < TT; ++t) *reinterpret_cast<f32x4*>(&red[wave][i][t][4 * lane]) = acc[i][t];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < TT * 256; j += kUpThreads) {
        const int i = j & 15, c = j >> 4 & 15, t = j >> 8, s = t0 + 16 * t + c;
        const int n = kScaled<T, E8> ? scaled_column(n0, i) : n0 + i;
        const int at = 4 * ((i >> 2) * 16 + c) + (i & 3);
        float g = red[0][0][t][at], u = red[0][1][t][at];
#pragma unroll
        for (int k = 1; k < kUpWaves; ++k) {
            g += red[k][0][t][at];
            u += red[k][1][t][at];
        }
        float act = silu_mul(g, u);
        if constexpr (kScaled<T, E8>) {
            const Pow2 f = pow2_for<T>(max16(n < a.N ? finite_bits(act) : 0u));
            act *= f.up;
            if (i == 0 && s < x.count) a.factor[(x.first + s) * a.ld_factor + (n0 >> 4)] = f.down;
        }
        if (s >= x.count || n >= a.N) continue;
        uint16_t hi, lo, *to = a.act + (x.first + s) * 2 * a.ld_act + n;
        split16<typename Act<T, E8>::type>(act, hi, lo);
        to[0] = hi;
        to[a.ld_act] = lo;
    }
    __syncthreads();
}

template <class T, bool E8>
__global__ void __launch_bounds__(kUpThreads) moe_up_kernel(MoeArgs a, int blocks)
{
    __shared__ float red[kUpWaves][2][4][256];
    const int j = blockIdx.x / blocks, n0 = (blockIdx.x - j * blocks) * 16;
    if (j >= *a.actives || !has_columns<T, E8>(n0, a.N)) return;
    const Active x = a.active[j];
    if (x.count <= 16) gate_up<T, E8, 1>(a, a.row, x, n0, 0, reinterpret_cast<float(*)[2][1][256]>(&red[0][0][0][0]));
    else gate_up<T, E8, 4>(a, a.row, x, n0, 0, red);
}

// The same for up to kRoutedRows rows, a wave for each: every workgroup ranks the logits itself, which takes less time
// than a launch before it, and the first one leaves the lists for the next launch.
template <class T, bool E8, class L, int PER>
__global__ void __launch_bounds__(kUpThreads) moe_routed_up_kernel(MoeArgs a, int blocks)
{
    __shared__ union {
        Routing<kUpThreads> r;
        float red[kUpWaves][2][1][256];
    } u;
    __shared__ int chosen[kRoutedRows * kMaxTop], row[kRoutedRows * kMaxTop];
    __shared__ float p[kRoutedRows * kMaxTop], weight[kRoutedRows * kMaxTop];
    __shared__ Active active[kRoutedRows * kMaxTop];
    const int j = blockIdx.x / blocks, n0 = (blockIdx.x - j * blocks) * 16;
    const int n = route<kUpThreads, PER, L>(a, u.r, chosen, p, active, row, weight);
    __syncthreads();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *a.actives = n;
        for (int i = threadIdx.x; i < a.M * a.top; i += kUpThreads) {
            if (i < n) a.active[i] = active[i];
            a.row[i] = row[i];  // slots past the last hold nothing that is read
            a.weight[i] = weight[i];
        }
    }
    if (has_columns<T, E8>(n0, a.N) && j < n) gate_up<T, E8, 1>(a, row, active[j], n0, 0, u.red);
}

// Adds one active expert's part of the results' ROWS columns from c0 on to the wave's sums, for TT tiles of its slots from t0
// on.  The two numbers of an activation are two columns of the matrix instruction, whose sums are added: a tile is ROWS / 2
// slots, which is as many as an expert of a small batch has, and the second numbers cost no instruction and no load.
// ROWS = 4: see the kernel.
template <class T, bool E8, int ROWS, int TT>
__device__ __forceinline__ void down(const MoeArgs& a, const Active& x, int c0, int t0, int s0, int s1, float* mine)
{
    using A = typename Act<T, E8>::type;
    constexpr int S = 16 / ROWS, EACH = ROWS / 2, ES = E8 ? 1 : 2;
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int place = i16 / ROWS, at = i16 % EACH, second = i16 / EACH % 2;
    const uint8_t* const w[1] = {a.w[2].data + (x.expert * a.w[2].stack + min(c0 + i16 % ROWS, a.K - 1) * a.w[2].ld) * ES};
    const float* const sc[1] = {E8 ? a.w[2].scale + x.expert * a.w[2].scale_stack + (c0 / kGroup) * a.w[2].scale_ld : nullptr};
    const A* v[TT];
    const float* f[TT];
    f32x4 acc[1][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int s = x.first + min(t0 + EACH * t + at, x.count - 1);
        v[t] = reinterpret_cast<const A*>(a.act) + (s * 2 + second) * a.ld_act;
        f[t] = a.factor + s * a.ld_factor;
        acc[0][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // stages read ahead where a workgroup has its CU to itself and registers to spare (37 rows, K = 4096 N = 768, 128 experts,
    // the layer: fp16 408 us with three, 429 with one; bf16 395 and 403)
    constexpr int U = ROWS == 16 && !E8 && TT == 1 ? 3 : 1;
    products<A, E8, 1, TT, S, U, kScaled<T, E8>>(w, sc, v, a.N, s0, s1, 1, q, place, acc, f);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // lane ^ EACH: a turn of 16 lanes by 8, or of 4 lanes by 2
            const float sum = acc[0][t][e];
            const int other = __builtin_amdgcn_update_dpp(0, __float_as_int(sum), EACH == 8 ? 0x128 : 0x4E, 0xF, 0xF, false);
            // an infinite sum of the first numbers is the result's: a weight's infinity meets second numbers of either sign, or 0
            if (abs_bits(sum) != 0x7f800000u) acc[0][t][e] = sum + __int_as_float(other);
        }
        const int slot = t0 + EACH * t + at;
        // rows 4 q .. + 3 of the instruction: with 4 places, place q
        if (slot < x.count && !second && (S == 1 || place == q)) {
            const int m = a.row[x.first + slot];
            float* to = mine + (S == 1 ? m * 16 + 4 * q : (place * a.M + m) * 4);
            const float weight = a.weight[x.first + slot];
#pragma unroll
            for (int e = 0; e < 4; ++e) to[e] = fmaf(weight, acc[0][t][e], to[e]);
        }
    }
    __builtin_amdgcn_wave_barrier();  // a row's sums pass between the wave's lanes, in LDS order
}

// out[m][c], ROWS columns c, of the active experts that are this split's.  ROWS = 4, for up to 4 rows of x, takes the same 4
// weight rows at 4 places along their columns as the 16 rows of an instruction, and x's rows likewise: of the results
// the blocks on the diagonal are wanted, and there are 4 times the workgroups.
template <class T, bool E8, int ROWS, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) moe_down_kernel(MoeArgs a, MoePlan p)
{
    constexpr int S = 16 / ROWS;     // places
    constexpr int EACH = ROWS / 2;   // slots per tile
    extern __shared__ float sums[];  // [wave][place][M][ROWS]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = blockIdx.x * ROWS, split = blockIdx.y;
    float* mine = sums + wave * a.M * 16;
    for (int i = lane; i < a.M * 16; i += 64) mine[i] = 0.0f;
    __builtin_amdgcn_wave_barrier();
    const int actives = *a.actives;
    const int stages = (a.N + kStageCols<E8> * S - 1) / (kStageCols<E8> * S);
    const int per = (stages + p.parts - 1) / p.parts;
    for (int u = wave; ; u += WAVES) {
        const int j = u / p.parts * p.splits + split, part = u % p.parts;
        if (j >= actives) break;
        const Active x = a.active[j];
        const int s0 = part * per, s1 = min(stages, (part + 1) * per);
        // the registers of two tiles cost a workgroup per CU with 4 places (one row, K = 2560 N = 1024 of e4m3: 23.8 us, 21.0
        // with one), and those of four are too many with e4m3 or factors
        constexpr int MOST = ROWS == 4 ? 1 : E8 || kScaled<T, E8> ? 2 : 4;
        for (int t = 0; t < x.count;) {
            const int left = x.count - t;
            if (MOST == 1 || left <= EACH) {
                down<T, E8, ROWS, 1>(a, x, c0, t, s0, s1, mine);
                t += EACH;
            } else if (MOST == 2 || left <= 2 * EACH) {
                if constexpr (MOST >= 2) down<T, E8, ROWS, 2>(a, x, c0, t, s0, s1, mine);
                t += 2 * EACH;
            } else {
                if constexpr (MOST == 4) down<T, E8, ROWS, 4>(a, x, c0, t, s0, s1, mine);
                t += 4 * EACH;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * ROWS; i += 64 * WAVES) {
        const int m = i / ROWS, c = c0 + i % ROWS;
        if (c >= a.K) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WAVES * S; ++k) v += sums[k * a.M * ROWS + i];
        if (p.splits == 1) static_cast<T*>(a.out)[m * a.ldo + c] = narrow<T>(v);
        else a.part[((int64_t)split * a.M + m) * a.K + c] = v;
    }
}

// The splits' sums of one row, in order
template <class T>
__global__ void __launch_bounds__(256) moe_join_kernel(MoeArgs a, int splits)
{
    const int c = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (c >= a.K) return;
    const float* p = a.part + (int64_t)m * a.K + c;
    float v = 0.0f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += p[(int64_t)s * a.M * a.K];
    static_cast<T*>(a.out)[m * a.ldo + c] = narrow<T>(v);
}

// logits[m][e] = x[m] router[e] in fp32: 16 experts and 16 TT rows, whose columns the waves share.  Bound by the chain of
// its loads: with the launch, one row, K = 2560, 64 experts 4.4 us; 37 rows, K = 4096, 128 experts 15; 1024 rows 20.
template <class T, int TT, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) moe_logits_kernel(LogitsArgs a, int blocks, int tile0)
{
    __shared__ float red[WAVES][TT][256];
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = (int)(blockIdx.x % blocks) * 16, m0 = (tile0 + (int)(blockIdx.x / blocks)) * 16 * TT;
    const uint8_t* const w[1] = {static_cast<const uint8_t*>(a.router) + min(e0 + i16, a.E - 1) * a.ldr * 2};
    const float* const none[TT] = {}, *const no_scale[1] = {};
    const T* v[TT];
    f32x4 acc[1][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        v[t] = static_cast<const T*>(a.x) + min(m0 + 16 * t + i16, a.M - 1) * a.ldx;
        acc[0][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int stages = (a.K + kStageCols<false> - 1) / kStageCols<false>;
    products<T, false, 1, TT, 1>(w, no_scale, v, a.K, wave, stages, WAVES, q, 0, acc, none);
#pragma unroll
    for (int t = 0; t < TT; ++t) *reinterpret_cast<f32x4*>(&red[wave][t][4 * lane]) = acc[0][t];
    __syncthreads();
    for (int j = threadIdx.x; j < TT * 256; j += 64 * WAVES) {
        const int i = j & 15, c = j >> 4 & 15, t = j >> 8, m = m0 + 16 * t + c, e = e0 + i;
        if (m >= a.M || e >= a.E) continue;
        const int at = 4 * ((i >> 2) * 16 + c) + (i & 3);
        float sum = red[0][t][at];
#pragma unroll
        for (int k = 1; k < WAVES; ++k) sum += red[k][t][at];
        a.logits[(int64_t)m * a.E + e] = sum;
    }
}

template <class T, int TT, int WAVES>
void logits_launches(const LogitsArgs& a, hipStream_t stream)
{
    const int blocks = (a.E + 15) / 16, tiles = (int)(((int64_t)a.M + 16 * TT - 1) / (16 * TT)), fit = (1 << 20) / blocks;
    for (int t = 0; t < tiles; t += fit) {
        const dim3 grid((unsigned)((tiles - t < fit ? tiles - t : fit) * blocks));
        hipLaunchKernelGGL((moe_logits_kernel<T, TT, WAVES>), grid, dim3(64 * WAVES), 0, stream, a, blocks, t);
    }
}

template <class T>
hipError_t logits(const LogitsArgs& a, hipStream_t stream)
{
    if (a.M <= 16) logits_launches<T, 1, 16>(a, stream);
    else logits_launches<T, 4, 8>(a, stream);
    return hipGetLastError();
}

template <class T, bool E8, class L, int PER>
void first_launches(const MoeArgs& a, hipStream_t stream)
{
    // whole pairs of 16 columns, which share an activation's lines
    const int most = a.M * a.top < a.E ? a.M * a.top : a.E, blocks = a.N > 0 ? (a.N + 31) / 32 * 2 : 1;
    const dim3 grid((unsigned)(most * blocks));
    if (a.M <= kRoutedRows) {
        hipLaunchKernelGGL((moe_routed_up_kernel<T, E8, L, PER>), grid, dim3(kUpThreads), 0, stream, a, blocks);
        return;
    }
    hipLaunchKernelGGL((moe_route_kernel<L, PER>), dim3(1), dim3(kRouteThreads), (size_t)a.M * a.top * 8, stream, a);
    if (a.N > 0) hipLaunchKernelGGL((moe_up_kernel<T, E8>), grid, dim3(kUpThreads), 0, stream, a, blocks);
}

template <class T, bool E8, class L>
void first_launches(const MoeArgs& a, hipStream_t stream)
{
    if (a.E <= 128) first_launches<T, E8, L, 2>(a, stream);
    else if (a.E <= 256) first_launches<T, E8, L, 4>(a, stream);
    else first_launches<T, E8, L, 16>(a, stream);
}

template <class T, bool E8>
hipError_t launch(int logits_dtype, const MoeArgs& a, const MoePlan& p, hipStream_t stream)
{
    if (logits_dtype == GLU_DTYPE_FP32) first_launches<T, E8, Fp32>(a, stream);
    else first_launches<T, E8, T>(a, stream);
    const dim3 grid((a.K + p.rows - 1) / p.rows, p.splits);
    const size_t lds = (size_t)a.M * 64;  // per wave
    if (p.rows == 4) hipLaunchKernelGGL((moe_down_kernel<T, E8, 4, 8>), grid, dim3(512), 8 * lds, stream, a, p);
    else hipLaunchKernelGGL((moe_down_kernel<T, E8, 16, 16>), grid, dim3(1024), 16 * lds, stream, a, p);
    if (p.splits > 1) {
        hipLaunchKernelGGL(moe_join_kernel<T>, dim3((a.K + 255) / 256, a.M), dim3(256), 0, stream, a, p.splits);
    }
    return hipGetLastError();
}

}  // namespace

// The second product's cut.  16 rows per workgroup of 16 waves, which share experts in halves or smaller parts so that no
// wave has much more to do than another (6 rows of e4m3, K = 4096 N = 1536, 128 experts: 64 us with whole experts, 62 with
// halves; 37 rows of bf16, N = 768: 143 either way).  Workgroups for half of the CUs at least: their sums' join costs 5 us.
MoePlan moe_plan(int M, int K, int N, int E, int top, bool e4m3)
{
    const int most = M * top < E ? M * top : E;
    MoePlan p{1, 1, M <= 4 ? 4 : 16};
    const int waves = p.rows == 4 ? 8 : 16, cols = (e4m3 ? 128 : 64) * 16 / p.rows, stages = (N + cols - 1) / cols;
    if (p.rows == 16 && stages >= 2) p.parts = 2;
    while (most * p.parts < waves && 2 * p.parts <= stages) p.parts *= 2;
    const int blocks = (K + p.rows - 1) / p.rows;
    while (p.rows == 16 && blocks * p.splits < 128 && most * p.parts >= 2 * waves * p.splits && p.splits < 8) p.splits *= 2;
    return p;
}

hipError_t moe_launch(int dtype, int logits_dtype, bool e4m3, const MoeArgs& a, const MoePlan& p, hipStream_t stream)
{
    if (dtype == GLU_DTYPE_BF16) return e4m3 ? launch<Bf16, true>(logits_dtype, a, p, stream) : launch<Bf16, false>(logits_dtype, a, p, stream);
    return e4m3 ? launch<Fp16, true>(logits_dtype, a, p, stream) : launch<Fp16, false>(logits_dtype, a, p, stream);
}

hipError_t moe_logits_launch(int dtype, const LogitsArgs& a, hipStream_t stream)
{
    return dtype == GLU_DTYPE_BF16 ? logits<Bf16>(a, stream) : logits<Fp16>(a, stream);
}

}  // namespace glu
