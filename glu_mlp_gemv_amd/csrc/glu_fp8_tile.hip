// Block-scaled e4m3 products tiled through LDS, for more rows of x than the
// streaming kernels take.
//
// A workgroup of WM x WN waves owns BM = 16 TM WM rows of x and BR = 16 TN WN weight rows (with two matrices
// half of each, so that gate and up of one output meet in one lane).  K is walked one block of 128 at a time: a
// stage is BM + BR rows of 128 bytes and the scales of x, brought straight from memory into one of STAGES
// buffers of LDS.  The matrix instruction sums exactly one K-block, so its result is multiplied by the two
// scales and added to the accumulator on the vector unit, 4 fused multiply-adds per lane against 32 cycles
// (8-bit) or 64 (bf16) of the matrix unit.
//
// What bounds it, at M = 4096 K = 17408 N = 4096 (256 tiles of 256 x 256, one round): 234 us, 2.50 PFLOP/s on
// the 8-bit unit, where the library's unscaled product at 8192^3 runs at 3.29 in short runs and 2.86 once the
// card has warmed to its power limit (its clock falls from 1.9 to 1.6 GHz).  The matrix unit is busy 68 % of the
// cycles; without the loads of the main loop the kernel takes 191 us, without the scaling 217.  On the bf16 unit
// (dual, K = 17408 N = 2048) 421 us, 1.39 PFLOP/s against the library's 1.65 and 1.5: there conversions,
// scaling and products together fill 95 % of the issue slots that the products' time has.  Steps that led there,
// at the first size: operands fetched across the stage's end and one barrier in its middle 262 -> 250, tiles in
// blocks of 8 x 4 per XCD (a third fewer L2 misses) no change in time, loads spread over the steps 250 -> 243,
// weights fetched two rows of tiles ahead 243 -> 234.  Half as much again in flight (three buffers of weights,
// those of x refilled in mid-stage) gave nothing: 244.
//
// In LDS, 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7): every group of 16 lanes that a ds_read_b128
// serves together then touches 16 different slots of the 256-byte bank line (no conflict counted).  A wave's
// direct load writes 64 consecutive slots (8 rows), so the exchange is made in the source addresses.
#include <type_traits>

#include "glu_fp8_mfma.h"

namespace glu {

const TileShape kTileShapes[kTileShapeCount] = {
    {256, 256, 512, 2},
    {128, 256, 512, 3},
    {64, 256, 256, 3},
    {64, 128, 256, 4},
    {32, 128, 256, 4},
};

namespace {

// 16 bytes per lane from base + off into LDS at lds_base + 16 lane; ONCE: not kept in the caches
template <bool ONCE>
__device__ __forceinline__ void lds_load16(const uint8_t* base, uint32_t off, uint8_t* lds)
{
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void*)(base + off),
        (__attribute__((address_space(3))) void*)lds, 16, 0, ONCE ? 2 : 0);
}

struct Narrow { raw4_t c0, c1; };
template <bool WIDE> struct Form { using type = Narrow; };
template <> struct Form<true> { using type = Wide; };

template <bool WIDE>
__device__ __forceinline__ typename Form<WIDE>::type operand(raw4_t c0, raw4_t c1)
{
    if constexpr (WIDE) return widen32(c0, c1);
    else return Narrow{c0, c1};
}

// a K-block's product
__device__ __forceinline__ f32x4 multiply(const Narrow& a, const Narrow& b)
{
    return mfma_e4m3(a.c0, a.c1, b.c0, b.c1);
}
__device__ __forceinline__ f32x4 multiply(const Wide& a, const Wide& b) { return mfma_wide(a, b); }

template <int N>
__device__ __forceinline__ void wait_vm()
{
    // vmcnt in bits 3:0 and 15:14, everything else not waited for
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

}  // namespace

// WIDE: products on the bf16 unit, for outputs that show more than the 8-bit unit's sums hold: e4m3, whose fp32
// scales are the largest sums themselves, and fp32.  E4M3: the kernel converts by itself (a workgroup holds
// whole groups).  ONCE: the weights are not kept in the caches.
template <int NM, int TM, int TN, int WM, int WN, int STAGES, bool WIDE, bool E4M3, bool ONCE>
__global__ void __launch_bounds__(64 * WM * WN)
fp8_tile_kernel(Fp8Args a, int nbm, int nbn, int splits)
{
    constexpr int WAVES = WM * WN;
    constexpr int BM = 16 * TM * WM, BR = 16 * TN * WN, BN = BR / NM;
    constexpr int TNM = TN / NM;                      // 16-row tiles of each matrix per wave
    constexpr int LPW = (BM + BR) / 8 / WAVES;        // direct loads (8 rows each) per wave and stage
    constexpr int XPW = BM / 8 / WAVES;               // ... of which rows of x
    constexpr int SXW = (BM + 63) / 64;               // waves that load scales of x
    constexpr int STAGE = (BM + BR) * kGroup + 4 * SXW * 64;
    static_assert(BM % (8 * WAVES) == 0 && BR % (8 * NM * WAVES) == 0 && TN % 2 == 0 && TN % NM == 0,
                  "whole loads per wave");
    static_assert(WAVES % 2 == 0, "a wave's loads lie a multiple of 16 rows apart");

    extern __shared__ __attribute__((aligned(256))) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int i16 = lane & 15, q = lane >> 4;

    // An XCD takes a run of tiles, in blocks 8 tiles of x high: the 32 that it works on at a time then read 8
    // row blocks of x and 4 of the weights between them, the least that its L2 has to fetch.
    constexpr int HIGH = 8;
    const int t = xcd_run(blockIdx.x, nbm * nbn);
    const int band = t / (HIGH * nbn);
    const int high = min(HIGH, nbm - band * HIGH);
    const int r = t - band * HIGH * nbn;
    const int nb = r / high, mb = band * HIGH + r - nb * high;
    const int m0 = mb * BM, n0 = nb * BN;
    const int KB = (a.K + kGroup - 1) / kGroup;
    const int split = blockIdx.y;
    const int kb0 = (int)((int64_t)KB * split / splits), kb1 = (int)((int64_t)KB * (split + 1) / splits);
    const int stages = kb1 - kb0;

    // sources of this wave's direct loads: lane l fills slot l % 8 of row l / 8, with chunk (l % 8) ^ swizzle
    const int lr = lane >> 3, lc = lane & 7;
    const uint8_t* base[1 + NM];
    base[0] = a.x + (int64_t)m0 * a.ldx;
#pragma unroll
    for (int m = 0; m < NM; ++m) base[1 + m] = a.w[m] + (int64_t)n0 * a.ldw[m];
    // the same chunk in every load: rows of two loads differ by a multiple of 16
    const int chunk = lc ^ ((wave * 4 + (lr >> 1)) & 7);
    uint32_t off[LPW];
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
        // rows of the stage in LDS: x, then each matrix
        const int r = i < XPW ? (i * WAVES + wave) * 8 + lr : BM + ((i - XPW) * WAVES + wave) * 8 + lr;
        if (i < XPW) {
            off[i] = (uint32_t)min(r, a.M - 1 - m0) * (uint32_t)a.ldx;
        } else {
            const int m = (i - XPW) / ((LPW - XPW) / NM);
            off[i] = (uint32_t)min(r - BM - m * BN, a.N - 1 - n0) * (uint32_t)a.ldw[m];
        }
        off[i] += 16 * chunk;
    }
    const int sxrow = min(m0 + (wave % SXW) * 64 + lane, a.M - 1);
    const float* sxp = a.sx + (int64_t)sxrow * a.sxm;

    // Loads the stage of K-block kb into a buffer; past the last stage the last one again, so that every stage
    // issues, and waits for, the same number of loads.  Past the row's end its own first chunk is read instead.
    const uint32_t past_end = (KB - 1) * kGroup + 16 * chunk >= a.K ? 16 * chunk : 0;
    auto issue = [&](int kb, int buf, int first, int count) __attribute__((always_inline)) {
        kb = min(kb, kb1 - 1);
        uint8_t* st = smem + buf * STAGE;
        const uint32_t back = kb == KB - 1 ? past_end : 0;
#pragma unroll
        for (int i = first; i < first + count; ++i) {
            if (i < LPW) {
                const int b = i < XPW ? 0 : 1 + (i - XPW) / ((LPW - XPW) / NM);
                const int r8 = i < XPW ? i * WAVES + wave : BM / 8 + (i - XPW) * WAVES + wave;
                const uint8_t* from = base[b] + (int64_t)kb * kGroup;
                if (i < XPW) lds_load16<false>(from, off[i] - back, st + r8 * 1024);
                else lds_load16<ONCE>(from, off[i] - back, st + r8 * 1024);
            } else if (i == LPW) {
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(sxp + kb * a.sxg),
                                                 (__attribute__((address_space(3))) void*)(st + (BM + BR) * kGroup +
                                                                                           (wave % SXW) * 256),
                                                 4, 0, 0);
            }
        }
    };
    // A stage's loads are issued a few per step (below): all at once they would fill the address units' queue
    // and hold up the waves' products behind them.
    constexpr int PER_STEP = (LPW + 1 + TM * TN - 1) / (TM * TN);
    // those in the last row of the stage before
    constexpr int EARLY = TM * PER_STEP < LPW + 1 ? TM * PER_STEP : LPW + 1;

    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // this wave's weight rows within a matrix, and the scale row they share (a wave's rows lie in one block of
    // 128)
    const int wr0 = wn * (TNM * 16);
    const float* swp[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) swp[m] = a.sw[m] + (int64_t)min((n0 + wr0) / kGroup, (a.N - 1) / kGroup) * a.ldsw[m];

    // slots of the operand reads: rows 16 t + l % 16 share the swizzle of l % 16
    const int swz = (i16 >> 1) & 7;
    const int rd0 = i16 * kGroup + ((q ^ swz) << 4), rd1 = i16 * kGroup + (((q + 4) ^ swz) << 4);

    using Operand = typename Form<WIDE>::type;
    const int xrd = wm * (TM * 16) * kGroup;
    auto read_x = [&](int buf, int j, raw4_t (&b)[2]) __attribute__((always_inline)) {
        const uint8_t* xs = smem + buf * STAGE + xrd + j * 16 * kGroup;
        b[0] = *reinterpret_cast<const raw4_t*>(xs + rd0);
        b[1] = *reinterpret_cast<const raw4_t*>(xs + rd1);
    };
    auto read_w = [&](int buf, int i, raw4_t (&w)[2]) __attribute__((always_inline)) {
        const int m = i / TNM;
        const uint8_t* ws = smem + buf * STAGE + (BM + m * BN + wr0 + (i - m * TNM) * 16) * kGroup;
        w[0] = *reinterpret_cast<const raw4_t*>(ws + rd0);
        w[1] = *reinterpret_cast<const raw4_t*>(ws + rd1);
    };
    auto meet = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's reads are in registers
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int s = 0; s < STAGES; ++s) issue(kb0 + s, s, 0, s < STAGES - 1 ? LPW + 1 : EARLY);
    wait_vm<(STAGES - 2) * (LPW + 1) + EARLY>();  // all but stage 0's
    meet();
    constexpr int AHEAD = !WIDE && TN >= 4 ? 2 : 1, SLOTS = 2 * AHEAD;
    raw4_t b[TM][2], w[SLOTS][2];
    float sx[TM];
    auto read_first = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) read_w(buf, i, w[i]);
        const float* src = reinterpret_cast<const float*>(smem + buf * STAGE + (BM + BR) * kGroup) + wm * (TM * 16);
#pragma unroll
        for (int j = 0; j < TM; ++j) sx[j] = src[16 * j + i16];
    };
    // past K in the last K-block: zeros for x, so that what was read there instead, of the same rows, adds
    // nothing
    auto clear = [&](int s, raw4_t (&b)[2]) __attribute__((always_inline)) {
        const bool in0 = (kb0 + s) * kGroup + 16 * q < a.K, in1 = (kb0 + s) * kGroup + 64 + 16 * q < a.K;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            b[0][e] = in0 ? b[0][e] : 0u;
            b[1][e] = in1 ? b[1][e] : 0u;
        }
    };
    if constexpr (!WIDE) {
#pragma unroll
        for (int j = 0; j < TM; ++j) read_x(0, j, b[j]);
        read_first(0);
    }

    // One stage.  Its first operands are in registers already, but for the wide form, which has none left for
    // that and reads them here.  No branch in it: the compiler would carry the sums past one, in ever more
    // registers.
    auto stage = [&](int s, int buf, auto last) __attribute__((always_inline)) {
        constexpr bool LAST = decltype(last)::value;
        const int next = buf + 1 == STAGES ? 0 : buf + 1, before = buf == 0 ? STAGES - 1 : buf - 1;
        if constexpr (WIDE) {
            read_x(buf, 0, b[0]);
            read_first(buf);
        }
        float sc[NM][TM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const float sw = scalar_load(swp[m] + kb0 + s);
#pragma unroll
            for (int j = 0; j < TM; ++j) sc[m][j] = sx[j] * sw;
        }
        // One step is one 16 x 16 product, in a fixed order: the sums of the product LAG steps before it, which
        // is done by now, free the registers that this one takes, and the operands of a step to come are
        // fetched behind it.
        constexpr int LAG = WIDE ? 1 : TM;
        Operand aw, bw[TM];
        f32x4 p[LAG + (WIDE ? 1 : 0)];
        constexpr int P = sizeof(p) / sizeof(p[0]);
        auto add = [&](int step) __attribute__((always_inline)) {
            const int i = step / TM, j = step % TM;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[step % P][e], sc[i / TNM][j], acc[i][j][e]);
        };
#pragma unroll
        for (int i = 0; i < TN; ++i) {
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int step = i * TM + j;
                if (!WIDE && step >= LAG) add(step - LAG);
                if (i == 0) {
                    if (WIDE && j + 1 < TM) read_x(buf, j + 1, b[j + 1]);
                    if (LAST) clear(s, b[j]);
                    bw[j] = operand<WIDE>(b[j][0], b[j][1]);
                }
                if (j == 0) aw = operand<WIDE>(w[i % SLOTS][0], w[i % SLOTS][1]);
                p[step % P] = multiply(aw, bw[j]);
                if (WIDE && step >= LAG) add(step - LAG);
                if (j == 0 && i + AHEAD < TN) read_w(buf, i + AHEAD, w[(i + AHEAD) % SLOTS]);
                if (!LAST && i == TN - 2 && j == TM - 1) {
                    // The stage's last operands are in registers, the next stage is in LDS: with a row of
                    // products in hand the waves meet, begin to refill this buffer and fetch the next stage's
                    // first operands.
                    wait_vm<(STAGES - 2) * (LPW + 1)>();  // all but those after stage s + 1
                    meet();
                }
                if (!LAST && i == TN - 1) issue(kb0 + s + STAGES, buf, j * PER_STEP, PER_STEP);
                if (!LAST && EARLY + step * PER_STEP < LPW + 1) {
                    issue(kb0 + s + STAGES - 1, before, EARLY + step * PER_STEP, PER_STEP);
                }
                if (!WIDE && !LAST && i == TN - 1) {
                    read_x(next, j, b[j]);
                    if (j == 0) read_first(next);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int step = TN * TM - LAG; step < TN * TM; ++step) add(step);
    };
    int buf = 0;
    for (int s = 0; s + 1 < stages; ++s) {
        stage(s, buf, std::false_type{});
        buf = buf + 1 == STAGES ? 0 : buf + 1;
    }
    stage(stages - 1, buf, std::true_type{});
    wait_vm<0>();  // the repeated loads have landed before LDS is given up or used again

    // lane l holds weight rows 4 (l / 16) + e of each tile, for row l % 16 of x
    const int mrow = m0 + wm * (TM * 16) + i16;
    const int ncol = n0 + wr0 + 4 * q;
    if (!E4M3 && a.out_dtype == kPartial) {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int m = i / TNM, n = ncol + (i - m * TNM) * 16;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int row = mrow + 16 * j;
                if (row < a.M && n < a.N) {
                    const int64_t at = ((int64_t)(split * NM + m) * a.M + row) * a.N + n;
                    store_values4(a.part, GLU_DTYPE_FP32, at, acc[i][j], a.N - n);
                }
            }
        }
        return;
    }
    if constexpr (NM == 2) {
#pragma unroll
        for (int i = 0; i < TNM; ++i) {
#pragma unroll
            for (int j = 0; j < TM; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = silu_mul(acc[i][j][e], acc[TNM + i][j][e]);
            }
        }
    }
    if constexpr (E4M3) {
        // rows past N hold copies of row N - 1 and may not count towards the maximum
        constexpr int GW = TNM * 16 >= kGroup ? 1 : kGroup / (TNM * 16);  // waves that share a group
        uint32_t* gmax = reinterpret_cast<uint32_t*>(smem);               // [WN][BM]
        __syncthreads();
        uint32_t am[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < TNM; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (ncol + 16 * i + e < a.N) m = max(m, abs_bits(acc[i][j][e]));
                }
            }
            m = max(m, (uint32_t)__builtin_amdgcn_ds_swizzle((int)m, 0x401F));  // lane ^ 16
            auto pr = __builtin_amdgcn_permlane32_swap(m, m, false, false);
            am[j] = max((uint32_t)pr[0], (uint32_t)pr[1]);
        }
        if constexpr (GW > 1) {
            if (lane < 16) {
#pragma unroll
                for (int j = 0; j < TM; ++j) gmax[wn * BM + wm * (TM * 16) + 16 * j + i16] = am[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int g0 = wn / GW * GW;
#pragma unroll
                for (int w = 0; w < GW; ++w) am[j] = max(am[j], gmax[(g0 + w) * BM + wm * (TM * 16) + 16 * j + i16]);
            }
        }
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int row = mrow + 16 * j;
            const Scale s = scale_of(am[j]);
            if (row >= a.M) continue;
#pragma unroll
            for (int i = 0; i < TNM; ++i) {
                const int n = ncol + 16 * i;
                if (n >= a.N) continue;
                int d = 0;
                d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(acc[i][j][0], s), quotient(acc[i][j][1], s), d, false);
                d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(acc[i][j][2], s), quotient(acc[i][j][3], s), d, true);
                uint8_t* o = static_cast<uint8_t*>(a.out) + row * a.ldo + n;
                if (n + 3 < a.N) {
                    __builtin_memcpy(o, &d, 4);
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        if (n + e < a.N) o[e] = (uint8_t)(d >> (8 * e));
                    }
                }
            }
            if (q == 0 && wn % GW == 0 && n0 + wr0 < a.N) a.scale[(int64_t)((n0 + wr0) / kGroup) * a.lds + row] = s.s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < TNM; ++i) {
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int row = mrow + 16 * j, n = ncol + 16 * i;
                if (row < a.M && n < a.N) store_values4(a.out, a.out_dtype, row * a.ldo + n, acc[i][j], a.N - n);
            }
        }
    }
}

namespace {

using TileFn = void (*)(Fp8Args, int, int, int);

template <int NM, bool WIDE, bool E4M3, bool ONCE>
TileFn pick_small(int shape)
{
    // a pair's 128 weight rows are 64 columns: no whole group
    constexpr bool HALF = E4M3 && NM == 2;
    switch (shape) {
    case 2: return fp8_tile_kernel<NM, 4, 4, 1, 4, 3, WIDE, E4M3, ONCE>;
    case 3: return HALF ? nullptr : fp8_tile_kernel<NM, 4, 2, 1, 4, 4, WIDE, E4M3 && !HALF, ONCE>;
    case 4: return HALF ? nullptr : fp8_tile_kernel<NM, 2, 2, 1, 4, 4, WIDE, E4M3 && !HALF, ONCE>;
    }
    return nullptr;
}

template <int NM, bool WIDE, bool E4M3>
TileFn pick_tile(int shape, bool once)
{
    if (shape == 0) return fp8_tile_kernel<NM, 4, 8, 4, 2, 2, WIDE, E4M3, false>;
    if (shape == 1) return fp8_tile_kernel<NM, 4, 4, 2, 4, 3, WIDE, E4M3, false>;
    return once ? pick_small<NM, WIDE, E4M3, true>(shape) : pick_small<NM, WIDE, E4M3, false>(shape);
}

template <int NM>
TileFn pick_tile(int shape, bool wide, bool e4m3, bool once)
{
    if (e4m3) return pick_tile<NM, true, true>(shape, once);
    return wide ? pick_tile<NM, true, false>(shape, once) : pick_tile<NM, false, false>(shape, once);
}

// Weights that one row of tiles reads once, and that are too many for the last-level cache (256 MB, which
// everything between two calls passes through) to hold until the next call, are not kept in the caches: dual M = 37
// K = 4096 N = 12288 24.0 -> 22.3 us, M = 48 K = 5120 N = 17408 47.2 -> 44.8.  Where they would have stayed it costs:
// dual M = 64 K = 2560 N = 9216 to e4m3 22.9 -> 25.4.
constexpr int64_t kOnceBytes = 64 << 20;

size_t tile_lds(int shape)
{
    const TileShape& t = kTileShapes[shape];
    return (size_t)t.stages * ((t.bm + t.br) * kGroup + 4 * ((t.bm + 63) / 64) * 64);
}

}  // namespace

bool fp8_tile_owns_groups(int mats, int shape) { return kTileShapes[shape].br / mats % kGroup == 0; }

hipError_t fp8_tile_launch(int mats, const TileConfig& c, const Fp8Args& a, hipStream_t stream)
{
    const TileShape& t = kTileShapes[c.shape];
    const bool e4m3 = a.out_dtype == GLU_DTYPE_E4M3;
    const bool once = a.M <= t.bm && (int64_t)mats * a.N * a.K > kOnceBytes;
    const TileFn f = mats == 1 ? pick_tile<1>(c.shape, c.wide, e4m3, once) : pick_tile<2>(c.shape, c.wide, e4m3, once);
    if (!f) return hipErrorInvalidValue;
    const size_t lds = tile_lds(c.shape);
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)lds);
    if (e != hipSuccess) return e;
    const int bn = t.br / mats;
    const int nbm = (int)(((int64_t)a.M + t.bm - 1) / t.bm), nbn = (int)(((int64_t)a.N + bn - 1) / bn);
    hipLaunchKernelGGL(f, dim3((unsigned)(nbm * nbn), (unsigned)c.splits), dim3(t.threads), lds, stream, a, nbm, nbn,
                       c.splits);
    return hipGetLastError();
}

}  // namespace glu
