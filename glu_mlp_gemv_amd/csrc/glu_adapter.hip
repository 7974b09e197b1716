// Low-rank adapters beside a shared projection: the two products of
//
//   t[m] = x[m] a[i]^T,   out[m] = y[m] + scale[i] t[m] b[i]^T,   i = index[m]
//
// and the same two products of the backward, d = dout b and dx = scale d a, whose weights lie the other way round.
//
// Bound by memory: x, y and out are touched once and the products are 2 R operations per number of them.  Rows of
// one adapter need not lie together: a tile of 16 or 64 neighbouring rows finds the distinct adapters among its
// own rows and goes through them one after another (a prefill: one or two), or, where a batch mixes requests, in
// workgroups of their own.  So no call sorts anything, and an adapter's weights are read once per tile that has it.
// In every product the rows of w are the matrix instruction's rows and the batch's rows its columns: a lane then
// holds neighbouring numbers of one row of the result, and a row's own adapter is a lane's own condition.  Rows
// of other adapters are left out of the loads and stores, not multiplied by zero.
#include "../../include/glu_fp8.h"
#include "glu_adapter.h"
#include "glu_mat16.h"

namespace glu {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kStage = 64;  // contraction per wave and stage: one 128-byte line per row

struct Whole { static constexpr bool value = true; };
struct Part { static constexpr bool value = false; };

// adapter of a row; -1: none
__device__ __forceinline__ int adapter_of(const int32_t* index, int m, int M, int L)
{
    if (m >= M) return -1;
    const int i = index[m];
    return (unsigned)i < (unsigned)L ? i : -1;
}

// the first adapter left in a tile (the same in every lane); -1: none
template <int TM>
__device__ __forceinline__ int next_adapter(const int (&left)[TM])
{
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const uint64_t b = __ballot(left[t] >= 0);
        if (b) return __builtin_amdgcn_readlane(left[t], __builtin_ctzll(b));
    }
    return -1;
}

template <int TM>
__device__ __forceinline__ void take_out(int (&left)[TM], int cur)
{
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        if (left[t] == cur) left[t] = -1;
    }
}

// First product.  Tile: 16 TM rows of v, 16 RT rows of w; the 4 waves take stages of 64 columns in turn and join in LDS.
// COLUMNS: w is [C][R], and operand j of a lane is column RT (l % 16) + j.
template <class T, int TM, int RT, bool COLUMNS>
__global__ void __launch_bounds__(kThreads) adapter_low_kernel(LowArgs a, int slots, int rgroups, int tile0)
{
    __shared__ float red[kWaves][TM * RT][256];
    __shared__ int rows_of[16 * TM];
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (tile0 + blockIdx.x) * 16 * TM;
    const int split = blockIdx.y % a.splits, rg = blockIdx.y / a.splits % rgroups, mat = blockIdx.y / a.splits / rgroups;
    const int slot = blockIdx.z;
    const int r0 = rg * 16 * RT;
    const int stages = (a.C + kStage - 1) / kStage;
    const int per = (stages + a.splits - 1) / a.splits;
    const int s_end = min(stages, (split + 1) * per);
    float* part = a.part + (int64_t)(split * a.mats + mat) * a.M * a.R;

    int idx[TM], left[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        idx[t] = left[t] = adapter_of(a.index, m0 + 16 * t + i16, a.M, a.L);
        if (wave == 0 && q == 0) rows_of[16 * t + i16] = idx[t];
    }
    __syncthreads();
    if (slot == 0) {
        for (int j = threadIdx.x; j < 16 * TM * 16 * RT; j += kThreads) {
            const int m = m0 + j / (16 * RT), r = r0 + j % (16 * RT);
            if (m < a.M && r < a.R && rows_of[j / (16 * RT)] < 0) part[(int64_t)m * a.R + r] = 0.0f;
        }
    }
    int seen = 0;
    for (;;) {
        const int cur = next_adapter<TM>(left);
        if (cur < 0) break;
        take_out<TM>(left, cur);
        if (seen++ % slots != slot) continue;

        // rows of v: lanes whose row has another adapter read the first of this one's along
        const T* v[TM];
        {
            int first = 0;
#pragma unroll
            for (int t = TM - 1; t >= 0; --t) {
                const uint64_t b = __ballot(idx[t] == cur);
                if (b) first = m0 + 16 * t + __builtin_ctzll(b);
            }
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                const int m = idx[t] == cur ? m0 + 16 * t + i16 : first;
                v[t] = static_cast<const T*>(a.v) + m * a.ldv;
            }
        }
        const T* w = static_cast<const T*>(a.w[mat].w) + cur * a.w[mat].stack;
        const int64_t wrow = a.w[mat].row;
        f32x4 acc[TM][RT];
#pragma unroll
        for (int t = 0; t < TM; ++t) {
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const int rl = r0 + RT * i16;  // COLUMNS: this lane's first column of w
        auto stage = [&](int s, auto whole_tag) __attribute__((always_inline)) {
            constexpr bool WHOLE = decltype(whole_tag)::value;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = s * kStage + 32 * h + 8 * q;
                raw4_t vf[TM], wf[RT];
#pragma unroll
                for (int t = 0; t < TM; ++t) vf[t] = WHOLE ? *reinterpret_cast<const u32x4_any*>(v[t] + c) : load8(v[t] + c, a.C - c);
                if constexpr (COLUMNS) {
                    load_columns<T, RT>([&](int i) { return w + min(c + i, a.C - 1) * wrow + rl; }, a.R - rl, wf);
                    if constexpr (!WHOLE) {
#pragma unroll
                        for (int j = 0; j < RT; ++j) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) wf[j][e] &= first_rows_mask(e, a.C - c);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < RT; ++j) {
                        const T* p = w + min(r0 + 16 * j + i16, a.R - 1) * wrow + c;
                        wf[j] = WHOLE ? *reinterpret_cast<const u32x4_any*>(p) : load8(p, a.C - c);
                    }
                }
#pragma unroll
                for (int t = 0; t < TM; ++t) {
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[t][j] = mfma16<T>(wf[j], vf[t], acc[t][j]);
                }
            }
        };
        const int whole_end = min(s_end, a.C / kStage);
        int s = split * per + wave;
#pragma unroll 2
        for (; s < whole_end; s += kWaves) stage(s, Whole{});
        if (s < s_end) stage(s, Part{});

#pragma unroll
        for (int t = 0; t < TM; ++t) {
#pragma unroll
            for (int j = 0; j < RT; ++j) *reinterpret_cast<f32x4*>(&red[wave][t * RT + j][4 * lane]) = acc[t][j];
        }
        __syncthreads();
        for (int p = threadIdx.x; p < TM * RT * 64; p += kThreads) {
            const int piece = p >> 6, l = p & 63, t = piece / RT, j = piece % RT;
            const int row = 16 * t + (l & 15);
            if (rows_of[row] != cur) continue;
            f32x4 sum = *reinterpret_cast<const f32x4*>(&red[0][piece][4 * l]);
#pragma unroll
            for (int k = 1; k < kWaves; ++k) sum += *reinterpret_cast<const f32x4*>(&red[k][piece][4 * l]);
            float* to = part + (int64_t)(m0 + row) * a.R;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * (l >> 4) + e;
                const int r = r0 + (COLUMNS ? RT * i + j : 16 * j + i);
                if (r < a.R) to[r] = sum[e];
            }
        }
        __syncthreads();
    }
}

// Second product.  Tile: 16 TM rows of z, which the workgroup first puts into LDS as two numbers of T each, and runs
// of 64 columns for each of its waves.  The contraction is 2 R8 chunks of 8 ranks: those of the first numbers
// and then those of the second, so that ranks up to 16 take one instruction per 16 x 16 results.  The rows of w in an instruction
// are chosen so that a lane's results are 8 neighbouring columns (COLUMNS: 16).
template <class T, int TM, int NM, bool COLUMNS>
__global__ void __launch_bounds__(kThreads) adapter_out_kernel(OutArgs a, int slots, int cblocks, int per, int tile0)
{
    extern __shared__ uint16_t lds[];  // z: [NM][2][16 TM][pitch]; then the rows' powers of two and maxima
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = tile0 + blockIdx.x / cblocks, cb = blockIdx.x % cblocks;
    const int m0 = tile * 16 * TM;
    const int slot = blockIdx.y;
    const int R8 = (a.R + 7) >> 3, pitch = 8 * R8 + 8;
    constexpr int ROWS = 16 * TM;
    float* down = reinterpret_cast<float*>(lds + NM * 2 * ROWS * pitch);  // [NM][ROWS]
    uint32_t* most = reinterpret_cast<uint32_t*>(down + NM * ROWS);

    int idx[TM], left[TM];
    bool bare = false;  // rows without an adapter
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int m = m0 + 16 * t + i16;
        idx[t] = left[t] = adapter_of(a.index, m, a.M, a.L);
        bare |= m < a.M && idx[t] < 0;
    }

    auto z8 = [&](int i, float (&v)[8]) __attribute__((always_inline)) {  // item i: mat, row, chunk
        const int c = i % R8, row = i / R8 % ROWS, mat = i / R8 / ROWS;
        const int n = m0 + row < a.M ? min(8, a.R - 8 * c) : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        for (int s = 0; s < a.splits; ++s) {
            const float* p = a.part + ((int64_t)(s * a.mats + mat) * a.M + m0 + row) * a.R + 8 * c;
            if (n == 8) {
                const Chunk<Fp32> k = load_chunk(reinterpret_cast<const Fp32*>(p), 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += k.e[e].v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e < n) v[e] += p[e];
                }
            }
        }
    };
    const int items = NM * ROWS * R8;
    if constexpr (!__is_same(T, Bf16)) {
        for (int i = threadIdx.x; i < NM * ROWS; i += kThreads) most[i] = 0u;
        __syncthreads();
        for (int i = threadIdx.x; i < items; i += kThreads) {
            float v[8];
            z8(i, v);
            atomicMax(&most[i / R8], abs_max8(v));  // a maximum: any order
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < items; i += kThreads) {
        float v[8];
        z8(i, v);
        const int c = i % R8, at = i / R8, row = at % ROWS, mat = at / ROWS;
        if (a.low && cb == 0 && slot == 0 && m0 + row < a.M) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (8 * c + e < a.R) a.low[(int64_t)(m0 + row) * a.R + 8 * c + e] = v[e];
            }
        }
        Pow2 f{1.0f, 1.0f};
        if constexpr (!__is_same(T, Bf16)) {
            f = pow2_for<T>(most[at]);
            if (c == 0) down[at] = f.down;
        }
        raw4_t hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t h, l;
            split16<T>(v[e] * f.up, h, l);
            hi[e >> 1] |= (uint32_t)h << (16 * (e & 1));
            lo[e >> 1] |= (uint32_t)l << (16 * (e & 1));
        }
        *reinterpret_cast<raw4_t*>(lds + ((mat * 2 + 0) * ROWS + row) * pitch + 8 * c) = hi;
        *reinterpret_cast<raw4_t*>(lds + ((mat * 2 + 1) * ROWS + row) * pitch + 8 * c) = lo;
    }
    __syncthreads();

    const int nblocks = (a.N + 63) >> 6;
    const int nb_first = (cb * per) * kWaves + wave, nb_end = min(nblocks, (cb + 1) * per * kWaves);
    const int steps = (2 * R8 + 3) >> 2;
    // this lane's 16 results of a 64-column block: group g of 8 at columns at[g] .. + 7
    const int at[2] = {COLUMNS ? 16 * q : 8 * q, COLUMNS ? 16 * q + 8 : 32 + 8 * q};

    auto pass = [&](int cur) __attribute__((always_inline)) {  // cur < 0: the rows without an adapter
        const float scale = cur >= 0 && a.scale ? a.scale[cur] : 1.0f;
        for (int nb = nb_first; nb < nb_end; nb += kWaves) {
            const int n0 = 64 * nb;
            f32x4 acc[NM][TM][4];
#pragma unroll
            for (int mat = 0; mat < NM; ++mat) {
#pragma unroll
                for (int t = 0; t < TM; ++t) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[mat][t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
            if (cur >= 0) {
#pragma unroll
                for (int mat = 0; mat < NM; ++mat) {
                    const T* w = static_cast<const T*>(a.w[mat].w) + cur * a.w[mat].stack;
                    const int64_t wrow = a.w[mat].row;
                    for (int s = 0; s < steps; ++s) {
                        const int c = 4 * s + q;
                        const bool there = c < 2 * R8;
                        const int second = c >= R8 ? 1 : 0, cc = there ? c - second * R8 : 0;
                        raw4_t wf[4];
                        if constexpr (COLUMNS) {
                            const int n = n0 + 4 * i16;
                            load_columns<T, 4>([&](int i) { return w + min(8 * cc + i, a.R - 1) * wrow + n; }, a.N - n, wf);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) wf[j][e] &= there ? first_rows_mask(e, a.R - 8 * cc) : 0u;
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int n = n0 + (j >> 1) * 32 + (i16 >> 2) * 8 + (j & 1) * 4 + (i16 & 3);
                                wf[j] = load8(w + min(n, a.N - 1) * wrow + 8 * cc, there ? a.R - 8 * cc : 0);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < TM; ++t) {
                            raw4_t z = *reinterpret_cast<const raw4_t*>(
                                lds + ((mat * 2 + second) * ROWS + 16 * t + i16) * pitch + 8 * cc);
                            if (!there) z = raw4_t{0u, 0u, 0u, 0u};
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[mat][t][j] = mfma16<T>(wf[j], z, acc[mat][t][j]);
                        }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                const int m = m0 + 16 * t + i16;
                if (m >= a.M || idx[t] != cur) continue;
                float f[NM];
#pragma unroll
                for (int mat = 0; mat < NM; ++mat) {
                    f[mat] = cur < 0 ? 0.0f : scale * (__is_same(T, Bf16) ? 1.0f : down[mat * ROWS + 16 * t + i16]);
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int n = n0 + at[g], cnt = a.N - n;
                    if (cnt <= 0) continue;
                    float o[NM][8];
#pragma unroll
                    for (int mat = 0; mat < NM; ++mat) {
                        Chunk<T> y{};
                        if (a.y[mat]) y = load_chunk(static_cast<const T*>(a.y[mat]) + m * a.ldy[mat] + n, cnt);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            // COLUMNS: column 16 q + 4 e' + j is element e' of operand j
                            const float d = COLUMNS ? acc[mat][t][e & 3][2 * g + (e >> 2)] : acc[mat][t][2 * g + (e >> 2)][e & 3];
                            o[mat][e] = fmaf(d, f[mat], widen(y.e[e]));
                        }
                    }
                    if constexpr (NM == 2) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[0][e] = silu_mul(o[0][e], o[1][e]);
                    }
                    store_chunk(static_cast<T*>(a.out) + m * a.ldo + n, narrow8<T>(o[0]), cnt);
                }
            }
        }
    };
    if (slot == 0 && __ballot(bare)) pass(-1);
    int seen = 0;
    for (;;) {
        const int cur = next_adapter<TM>(left);
        if (cur < 0) break;
        take_out<TM>(left, cur);
        if (seen++ % slots == slot) pass(cur);
    }
}

constexpr int64_t kMaxBlocks = 1 << 22;  // workgroups of 256 threads in a launch's first dimension

// Rows per tile: 64 share an adapter's weights where there are enough rows for that to matter, 16 else.  A tile
// of 16 rows has up to 16 adapters, whose workgroups are the launch's `slots`; larger batches are runs of rows.
int tile_m(int M) { return M > 256 ? 4 : 1; }
int slots_of(int M, int L) { return M > 256 ? 1 : (M < 16 ? (L < M ? L : M) : (L < 16 ? L : 16)); }

template <class T, bool COLUMNS>
hipError_t low_launch(const LowArgs& a, hipStream_t stream)
{
    const int tm = tile_m(a.M), slots = slots_of(a.M, a.L);
    const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
    const int rgroups = (a.R + 16 * rt - 1) / (16 * rt);
    const int tiles = (a.M + 16 * tm - 1) / (16 * tm);
    for (int64_t t = 0; t < tiles; t += kMaxBlocks) {
        const dim3 grid((unsigned)(tiles - t < kMaxBlocks ? tiles - t : kMaxBlocks), a.splits * rgroups * a.mats, slots);
#define GLU_LOW(TM, RT) \
    hipLaunchKernelGGL((adapter_low_kernel<T, TM, RT, COLUMNS>), grid, dim3(kThreads), 0, stream, a, slots, rgroups, (int)t)
        if (tm == 1) {
            if (rt == 1) GLU_LOW(1, 1);
            else if (rt == 2) GLU_LOW(1, 2);
            else GLU_LOW(1, 4);
        } else {
            if (rt == 1) GLU_LOW(4, 1);
            else if (rt == 2) GLU_LOW(4, 2);
            else GLU_LOW(4, 4);
        }
#undef GLU_LOW
    }
    return hipGetLastError();
}

template <class T, int NM, bool COLUMNS>
hipError_t out_launch(const OutArgs& a, hipStream_t stream)
{
    // ranks above 64 keep to 16 rows, whose z fits LDS at any rank
    const int tm = a.R <= 64 ? tile_m(a.M) : 1, slots = tm == 1 ? slots_of(a.M, a.L) : 1;
    const int rows = 16 * tm, tiles = (a.M + rows - 1) / rows;
    const int columns = a.N > 0 ? a.N : 1;                              // N == 0: z alone goes to low
    const int groups = (columns + 64 * kWaves - 1) / (64 * kWaves);  // one column block per wave
    // a workgroup keeps its z for several of them where there are workgroups enough
    int per = (int)((int64_t)tiles * groups / 2048);
    per = per < 1 ? 1 : per > 4 ? 4 : per;
    const int cblocks = (groups + per - 1) / per;
    const int R8 = (a.R + 7) / 8;
    const size_t bytes = (size_t)NM * 2 * rows * (8 * R8 + 8) * 2 + (size_t)NM * rows * 8;
    const int64_t fit = kMaxBlocks / cblocks < 1 ? 1 : kMaxBlocks / cblocks;
    for (int64_t t = 0; t < tiles; t += fit) {
        const dim3 grid((unsigned)((tiles - t < fit ? tiles - t : fit) * cblocks), slots);
        if (tm == 1) {
            hipLaunchKernelGGL((adapter_out_kernel<T, 1, NM, COLUMNS>), grid, dim3(kThreads), bytes, stream, a, slots,
                               cblocks, per, (int)t);
        } else {
            hipLaunchKernelGGL((adapter_out_kernel<T, 4, NM, COLUMNS>), grid, dim3(kThreads), bytes, stream, a, slots,
                               cblocks, per, (int)t);
        }
    }
    return hipGetLastError();
}

}  // namespace

// Parts of the contraction: as many as give every CU four waves' workgroups, of at least 4 stages (one per wave).
int adapter_low_splits(int M, int C, int R, int mats)
{
    const int tm = tile_m(M);
    const int64_t groups = ((int64_t)M + 16 * tm - 1) / (16 * tm) * mats * (R <= 64 ? 1 : (R + 63) / 64);
    const int64_t most = ((int64_t)C + kStage * kWaves - 1) / (kStage * kWaves);
    int64_t s = groups ? 512 / groups : 1;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

hipError_t adapter_low_launch(int dtype, bool columns, const LowArgs& a, hipStream_t stream)
{
    if (dtype == GLU_DTYPE_BF16) return columns ? low_launch<Bf16, true>(a, stream) : low_launch<Bf16, false>(a, stream);
    return columns ? low_launch<Fp16, true>(a, stream) : low_launch<Fp16, false>(a, stream);
}

hipError_t adapter_out_launch(int dtype, bool columns, const OutArgs& a, hipStream_t stream)
{
    if (a.mats == 2) {
        return dtype == GLU_DTYPE_BF16 ? out_launch<Bf16, 2, false>(a, stream) : out_launch<Fp16, 2, false>(a, stream);
    }
    if (columns) return dtype == GLU_DTYPE_BF16 ? out_launch<Bf16, 1, true>(a, stream) : out_launch<Fp16, 1, true>(a, stream);
    return dtype == GLU_DTYPE_BF16 ? out_launch<Bf16, 1, false>(a, stream) : out_launch<Fp16, 1, false>(a, stream);
}

}  // namespace glu
