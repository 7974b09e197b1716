// Low-rank adapters beside a shared projection: the two products of
//
//   t[m] = x[m] a[i]^T,   out[m] = y[m] + scale[i] t[m] b[i]^T,   i = index[m]
//
// and the same two products of the backward, d = dout b and dx = scale d a, whose weights lie the other way round.
//
// Bound by memory, and for a few rows by two launches: x, y and out are touched once, and the products are 2 R operations per
// number of them.  Rows of one adapter need not lie together: a tile of neighbouring rows finds the distinct adapters
// among its own rows and goes through them one after another (a prefill: one or two), or, where a batch mixes requests, in
// workgroups of their own.  So no call sorts anything, and an adapter's weights are read once per tile that has it.
// In every product the rows of w are the matrix instruction's rows and the batch's rows its columns, gathered from the
// tile: rows of other adapters are left out, not multiplied by zero.  The first product through LDS alone does not gather: it
// goes through the whole tile once per adapter in it and keeps the columns of that adapter's rows.  Kernel times: one row,
// K = 2560 N = 9216 rank 16, 3.4 + 4.9 us (an empty launch: 2.3); 37 rows of 32 adapters, K = 4096 N = 12288 rank 16, 4.8 +
// 7.6; 8192 rows, K = N = 5120 rank 64, 26 + 49 (84 MB read, 168 MB read and written: 3.3 and 3.4 TB/s); pair, 2050 rows,
// K = 4096 N = 12288 rank 16, 13 + 51.
#include "../../include/glu_fp8.h"
#include "glu_adapter.h"
#include "glu_mat16.h"

namespace glu {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTurnPitch = 68;  // of 64 results: a row's 16-byte pieces are one bank group on from the last row's
constexpr int kStage = 64;  // contraction per wave and stage: one 128-byte line per row

struct Whole { static constexpr bool value = true; };
struct Part { static constexpr bool value = false; };

// adapter of a row; -1: none; -2: no such row
__device__ __forceinline__ int adapter_of(const int32_t* index, int m, int M, int L)
{
    if (m >= M) return -2;
    const int i = index[m];
    return (unsigned)i < (unsigned)L ? i : -1;
}

// the first adapter left in a tile, whose rows' adapters the lanes hold (the same in every lane); -1: none
__device__ __forceinline__ int next_adapter(int left)
{
    const uint64_t b = __ballot(left >= 0);
    return b ? __builtin_amdgcn_readlane(left, __builtin_ctzll(b)) : -1;
}

// Whether this row is the first of 16 that a workgroup takes of the tile's rows with its adapter (or without one); cur: which
// adapter, from: its place among them.  The workgroups of the other rows have nothing to do.
__device__ __forceinline__ bool leads(int idx, int row, int& cur, int& from)
{
    cur = __builtin_amdgcn_readlane(idx, row);
    from = __popcll(__ballot(idx == cur) & ((1ull << row) - 1ull));
    return cur != -2 && from % 16 == 0;
}

// The rows of a tile that have this adapter, in order, to a list of the wave's own in LDS; how many there are
__device__ __forceinline__ int list_rows(int idx, int cur, uint8_t* list)
{
    const int lane = threadIdx.x & 63;
    const uint64_t b = __ballot(idx == cur);
    __builtin_amdgcn_wave_barrier();  // the last list is read; other lanes read this one, in LDS order
    if (idx == cur) list[__popcll(b & ((1ull << lane) - 1ull))] = (uint8_t)lane;
    __builtin_amdgcn_wave_barrier();
    return __popcll(b);
}

// Loads of a tile are a uniform address plus 32 bits per lane: rows of a tile times a row's bytes stay below 2^31
// (kMaxAdapterRow), and a lane keeps one register per row it reads instead of two and additions.
__device__ __forceinline__ raw4_t read16(const char* base, uint32_t lane)
{
    return *reinterpret_cast<const u32x4_any*>(base + lane);
}

// silu(g) u for results of 16 bits: without the correction of silu_mul the rounding of the exponent stays, for g > -87 at most
// 2 |g| units of 2^-24 of the result, of which at most one result in some hundred lands on the number next to it.  Below,
// where silu is less than 2^-119 in magnitude, the result may be -0 u, as with silu_mul (and as exp(-g) overflows in fp32).  A
// prefill's second product (2050 x 12288) takes 51 us instead of 54.
__device__ __forceinline__ float silu_mul16(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896340736f)) * u;
}

// 16 bytes per lane straight to LDS, lane l's at to + 16 l (to: uniform)
__device__ __forceinline__ void direct16(const char* base, uint32_t lane, uint8_t* to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + lane),
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// waits until all but this wave's last N loads are done; vmcnt in bits 3:0 and 15:14, nothing else waited for
template <int N>
__device__ __forceinline__ void wait_direct()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    __builtin_amdgcn_sched_barrier(0);
}

// waits until this wave's LDS reads are in registers
__device__ __forceinline__ void reads_done()
{
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
}

// First product.  Tile: up to 64 rows of v, of which those of one adapter are taken 16 TM at a time, 16 RT rows of w and a
// part of the columns; the 4 waves take stages of 64 columns in turn, keep U of them in flight, and join in LDS.
// COLUMNS: w is [C][R], and operand j of a lane is column RT (l % 16) + j.
template <class T, int TM, int RT, int U, bool COLUMNS>
__global__ void __launch_bounds__(kThreads, 3) adapter_low_kernel(LowArgs a, int tile_rows, bool by_row, int rgroups,
                                                                  int tile0)
{
    constexpr int PIECES = TM * RT;
    __shared__ float red[kWaves][PIECES][256];
    __shared__ uint8_t lists[kWaves][64];
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (tile0 + blockIdx.x) * tile_rows;
    const int split = blockIdx.y % a.splits, rg = blockIdx.y / a.splits % rgroups, mat = blockIdx.y / a.splits / rgroups;
    const int r0 = rg * 16 * RT;
    // this part's stages: first .. first + count - 1 are whole, `tail` is one that ends past the columns, or -1
    const int stages = (a.C + kStage - 1) / kStage, per = (stages + a.splits - 1) / a.splits;
    const int first = min(split * per, a.C / kStage), count = min((split + 1) * per, a.C / kStage) - first;
    const int tail = a.C % kStage && (stages - 1) / per == split ? stages - 1 : -1;
    float* z = a.z + (int64_t)(split * a.mats + mat) * a.M * a.R;

    const int idx = lane < tile_rows ? adapter_of(a.index, m0 + lane, a.M, a.L) : -2;
    int left = idx;
    uint8_t* list = lists[wave];
    int alone, from = 0;  // the workgroup's one adapter, where rows have workgroups of their own
    if (by_row && !leads(idx, blockIdx.z, alone, from)) return;
    const uint64_t bare = __ballot(idx == -1);
    if (bare && (!by_row || (alone == -1 && from == 0))) {
        for (int j = threadIdx.x; j < tile_rows * 16 * RT; j += kThreads) {
            const int row = j / (16 * RT), r = r0 + j % (16 * RT);
            if ((bare >> row & 1) && r < a.R) z[(int64_t)(m0 + row) * a.R + r] = 0.0f;
        }
    }
    const char* vbase = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + m0 * a.ldv);
    for (;;) {
        const int cur = by_row ? alone : next_adapter(left);
        if (cur < 0) break;
        if (left == cur) left = -1;

        int n = list_rows(idx, cur, list);
        if (by_row) n = min(n, from + 16);
        const T* w = static_cast<const T*>(a.w[mat].w) + cur * a.w[mat].stack;
        const int64_t wrow = a.w[mat].row;
        const char* wbase = reinterpret_cast<const char*>(w + (COLUMNS ? r0 : r0 * wrow));
        uint32_t wo[RT];  // COLUMNS: one of this lane's first column
#pragma unroll
        for (int j = 0; j < RT; ++j) wo[j] = ((uint32_t)min(16 * j + i16, a.R - 1 - r0) * (uint32_t)wrow + 8 * q) * 2;
        if constexpr (COLUMNS) wo[0] = ((uint32_t)(8 * q) * (uint32_t)wrow + RT * i16) * 2;
        for (int g = from; g < n; g += 16 * TM) {
            uint32_t vo[TM];  // places past the last row take the last row along
#pragma unroll
            for (int t = 0; t < TM; ++t) vo[t] = ((uint32_t)list[min(g + 16 * t + i16, n - 1)] * (uint32_t)a.ldv + 8 * q) * 2;
            f32x4 acc[TM][RT];
#pragma unroll
            for (int t = 0; t < TM; ++t) {
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            raw4_t vf[U][2][TM], wf[U][2][RT];
            auto load = [&](int u, int s) __attribute__((always_inline)) {
                const int at = (first + s) * kStage;
                const char* vb = vbase + at * 2;
                const char* wb = wbase + (COLUMNS ? at * wrow : (int64_t)at) * 2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int t = 0; t < TM; ++t) vf[u][h][t] = read16(vb + 64 * h, vo[t]);
                    if constexpr (COLUMNS) {
                        load_columns<T, RT>([&](int i) { return wb + (32 * h + i) * wrow * 2 + wo[0]; }, a.R - r0 - RT * i16, wf[u][h]);
                    } else {
#pragma unroll
                        for (int j = 0; j < RT; ++j) wf[u][h][j] = read16(wb + 64 * h, wo[j]);
                    }
                }
            };
            auto load_tail = [&](int u) __attribute__((always_inline)) {
                const int at = tail * kStage;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = at + 32 * h + 8 * q;  // this lane's first column
#pragma unroll
                    for (int t = 0; t < TM; ++t) vf[u][h][t] = load8(reinterpret_cast<const T*>(vbase + vo[t]) + at + 32 * h, a.C - c);
                    if constexpr (COLUMNS) {
                        load_columns<T, RT>([&](int i) { return w + min(c + i, a.C - 1) * wrow + r0 + RT * i16; },
                                            a.R - r0 - RT * i16, wf[u][h]);
#pragma unroll
                        for (int j = 0; j < RT; ++j) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) wf[u][h][j][e] &= first_rows_mask(e, a.C - c);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < RT; ++j) wf[u][h][j] = load8(reinterpret_cast<const T*>(wbase + wo[j]) + at + 32 * h, a.C - c);
                    }
                }
            };
            auto use = [&](int u) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int t = 0; t < TM; ++t) {
#pragma unroll
                        for (int j = 0; j < RT; ++j) acc[t][j] = mfma16<T>(wf[u][h][j], vf[u][h][t], acc[t][j]);
                    }
                }
            };
            // a ring of U stages: one is refilled as soon as it is used
            int s = wave;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s + u * kWaves < count) load(u, s + u * kWaves);
            }
            for (; s + (2 * U - 1) * kWaves < count; s += U * kWaves) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    use(u);
                    load(u, s + (u + U) * kWaves);
                }
            }
            for (; s < count; s += U * kWaves) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (s + u * kWaves < count) use(u);
                    if (s + (u + U) * kWaves < count) load(u, s + (u + U) * kWaves);
                }
            }
            if (tail >= 0 && wave == kWaves - 1) {
                load_tail(0);
                use(0);
            }

#pragma unroll
            for (int p = 0; p < PIECES; ++p) *reinterpret_cast<f32x4*>(&red[wave][p][4 * lane]) = acc[p / RT][p % RT];
            __syncthreads();
            for (int i = threadIdx.x; i < PIECES * 256; i += kThreads) {
                const int l = i >> 2 & 63, piece = i >> 8, t = piece / RT, j = piece % RT;
                const int at = g + 16 * t + (l & 15), k = 4 * (l >> 4) + (i & 3);
                const int r = r0 + (COLUMNS ? RT * k + j : 16 * j + k);
                if (at >= n || r >= a.R) continue;
                float sum = red[0][piece][i & 255];
#pragma unroll
                for (int o = 1; o < kWaves; ++o) sum += red[o][piece][i & 255];
                z[(int64_t)(m0 + list[at]) * a.R + r] = sum;
            }
            __syncthreads();
        }
        if (by_row) break;
    }
}

// The same for larger batches on whole 16-byte chunks.  In the kernel above neighbouring lanes load from different rows;
// here a load takes 8 rows' 128-byte lines, straight to LDS, where a wave has two stages of its own, and the operands are
// read from there; no barrier is needed before the waves join.  With a workgroup per CU (8192 rows of 5120): 16 ranks
// 18.3 us against 21.0, 64 ranks 25.2 against 36.8.  Chunk c of row r is in place c ^ (r / 2) of the row, so that 16 rows'
// chunks lie in different banks.
template <class T, int TM, int RT>
__global__ void __launch_bounds__(kThreads) adapter_low_tile_kernel(LowArgs a, int rgroups, int tile0)
{
    constexpr int PIECES = TM * RT, LOADS = 2 * (TM + RT), STAGE = LOADS * 1024, DEPTH = 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];  // [wave][DEPTH][rows of v, then of w][128 bytes]
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (tile0 + blockIdx.x) * 16 * TM;
    const int split = blockIdx.y % a.splits, rg = blockIdx.y / a.splits % rgroups, mat = blockIdx.y / a.splits / rgroups;
    const int r0 = rg * 16 * RT;
    const int stages = (a.C + kStage - 1) / kStage, per = (stages + a.splits - 1) / a.splits;
    const int first = min(split * per, a.C / kStage), count = min((split + 1) * per, a.C / kStage) - first;
    const int tail = a.C % kStage && (stages - 1) / per == split ? stages - 1 : -1;
    float* z = a.z + (int64_t)(split * a.mats + mat) * a.M * a.R;
    uint8_t* mine = smem + wave * DEPTH * STAGE;

    const int idx = lane < 16 * TM ? adapter_of(a.index, m0 + lane, a.M, a.L) : -2;
    int left = idx;
    const uint64_t bare = __ballot(idx == -1);
    for (int j = threadIdx.x; j < 16 * TM * 16 * RT; j += kThreads) {
        const int row = j / (16 * RT), r = r0 + j % (16 * RT);
        if ((bare >> row & 1) && r < a.R) z[(int64_t)(m0 + row) * a.R + r] = 0.0f;
    }
    const char* vbase = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + m0 * a.ldv);
    // what this lane loads: chunk lane % 8, turned by its row, of row lane / 8 of each 8; rows of two loads differ by 8
    const int lr = lane >> 3, lc = lane & 7;
    uint32_t vo[2 * TM], wo[2 * RT];
#pragma unroll
    for (int i = 0; i < 2 * TM; ++i) {
        const int r = 8 * i + lr;
        vo[i] = (uint32_t)min(r, a.M - 1 - m0) * (uint32_t)a.ldv * 2 + 16 * (lc ^ (r >> 1 & 7));
    }
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) {
        const int r = 8 * i + lr;
        wo[i] = (uint32_t)min(r, a.R - 1 - r0) * (uint32_t)a.w[mat].row * 2 + 16 * (lc ^ (r >> 1 & 7));
    }
    const int rd[2] = {i16 * 128 + ((q ^ (i16 >> 1)) << 4), i16 * 128 + (((q + 4) ^ (i16 >> 1)) << 4)};
    for (;;) {
        const int cur = next_adapter(left);
        if (cur < 0) break;
        if (left == cur) left = -1;
        const uint64_t rows = __ballot(idx == cur);
        const int64_t wrow = a.w[mat].row;
        const char* wbase = reinterpret_cast<const char*>(static_cast<const T*>(a.w[mat].w) + cur * a.w[mat].stack + r0 * wrow);
        f32x4 acc[TM][RT];
#pragma unroll
        for (int t = 0; t < TM; ++t) {
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // past the last stage the last one again, so that every stage waits for the same number of loads
        const int turns = (count - wave + kWaves - 1) / kWaves;  // this wave's stages
        auto load = [&](int k, int buf) __attribute__((always_inline)) {
            const int s = min(k, turns - 1) * kWaves + wave;
            const char* vb = vbase + (first + s) * 128;
            const char* wb = wbase + (first + s) * 128;
            uint8_t* to = mine + buf * STAGE;
#pragma unroll
            for (int i = 0; i < 2 * TM; ++i) direct16(vb, vo[i], to + i * 1024);
#pragma unroll
            for (int i = 0; i < 2 * RT; ++i) direct16(wb, wo[i], to + (2 * TM + i) * 1024);
        };
        auto use = [&](int buf) __attribute__((always_inline)) {
            const uint8_t* from = mine + buf * STAGE;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                raw4_t vf[TM], wf[RT];
#pragma unroll
                for (int t = 0; t < TM; ++t) vf[t] = *reinterpret_cast<const raw4_t*>(from + t * 2048 + rd[h]);
#pragma unroll
                for (int j = 0; j < RT; ++j) wf[j] = *reinterpret_cast<const raw4_t*>(from + (TM + j) * 2048 + rd[h]);
#pragma unroll
                for (int t = 0; t < TM; ++t) {
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[t][j] = mfma16<T>(wf[j], vf[t], acc[t][j]);
                }
            }
        };
        if (turns > 0) {
            load(0, 0);
            load(1, 1);
            for (int k = 0; k < turns; ++k) {
                wait_direct<LOADS>();  // all but the next stage's
                use(k & 1);
                reads_done();
                load(k + 2, k & 1);
            }
            wait_direct<0>();  // the LDS they write is used again
        }
        if (tail >= 0 && wave == kWaves - 1) {
            const int at = tail * kStage;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = at + 32 * h + 8 * q;
                raw4_t vf[TM], wf[RT];
#pragma unroll
                for (int t = 0; t < TM; ++t) {
                    vf[t] = load8(reinterpret_cast<const T*>(vbase + (uint32_t)min(16 * t + i16, a.M - 1 - m0) * (uint32_t)a.ldv * 2) + c, a.C - c);
                }
#pragma unroll
                for (int j = 0; j < RT; ++j) {
                    wf[j] = load8(reinterpret_cast<const T*>(wbase + (uint32_t)min(16 * j + i16, a.R - 1 - r0) * (uint32_t)wrow * 2) + c, a.C - c);
                }
#pragma unroll
                for (int t = 0; t < TM; ++t) {
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[t][j] = mfma16<T>(wf[j], vf[t], acc[t][j]);
                }
            }
        }
        __syncthreads();
        float(*red)[PIECES][256] = reinterpret_cast<float(*)[PIECES][256]>(smem);  // fits: 1 KB a piece, 2 KB a tile of rows
#pragma unroll
        for (int p = 0; p < PIECES; ++p) *reinterpret_cast<f32x4*>(&red[wave][p][4 * lane]) = acc[p / RT][p % RT];
        __syncthreads();
        for (int i = threadIdx.x; i < PIECES * 64; i += kThreads) {
            const int l = i & 63, piece = i >> 6, t = piece / RT, j = piece % RT;
            const int row = 16 * t + (l & 15), r = r0 + 16 * j + 4 * (l >> 4);
            if (!(rows >> row & 1) || r >= a.R) continue;
            f32x4 sum = *reinterpret_cast<const f32x4*>(&red[0][piece][4 * l]);
#pragma unroll
            for (int o = 1; o < kWaves; ++o) sum += *reinterpret_cast<const f32x4*>(&red[o][piece][4 * l]);
            float* to = z + (int64_t)(m0 + row) * a.R + r;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (r + e < a.R) to[e] = sum[e];
            }
        }
        __syncthreads();
    }
}

// Second product.  Tile: up to 64 rows, of which those of one adapter are taken 16 TM at a time: their z, which the
// workgroup puts into LDS as two numbers of T each, and runs of 64 columns for each of its waves, whose y and w are on their
// way meanwhile.  The contraction is RP = ranks rounded up places of the first numbers and then RP of the second, so that up
// to 16 ranks (S = 1) they share one instruction's 32 places; S instructions with H operands of w per 16 columns, or
// (S = 0) as many as there are ranks.  The results, of which a lane holds 4 columns of its own row, go through LDS to lanes
// that hold 8 columns, 8 neighbouring lanes a line: so y is read and out written (8192 x 5120, rank 64: 58 us with each
// lane's own row, 51 so; rank 16 42 and 37).
template <class T, int TM, int NM, int S, bool COLUMNS>
__global__ void __launch_bounds__(kThreads, 2) adapter_out_kernel(OutArgs a, int tile_rows, bool by_row, int cblocks,
                                                                  int per, int tile0)
{
    constexpr int ROWS = 16 * TM, H = S > 1 ? S / 2 : 1;
    // z as T [NM][ROWS][pitch]; the rows' powers of two and maxima [NM][ROWS]
    extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
    __shared__ uint8_t lists[kWaves][64];
    __shared__ __attribute__((aligned(16))) float turned[kWaves][16 * kTurnPitch];
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % cblocks, m0 = (tile0 + blockIdx.x / cblocks) * tile_rows;
    const int nb_first = cb * per * kWaves + wave, nb_end = min((a.N + 63) >> 6, (cb + 1) * per * kWaves);
    const int RP = S ? 16 * (S == 1 ? 1 : S) : (a.R + 31) & ~31, R8 = RP >> 3, pitch = 2 * RP + 8;
    const int steps = S ? S : RP >> 4;
    float* down = reinterpret_cast<float*>(lds + NM * ROWS * pitch);
    uint32_t* most = reinterpret_cast<uint32_t*>(down + NM * ROWS);

    const int idx = lane < tile_rows ? adapter_of(a.index, m0 + lane, a.M, a.L) : -2;
    int left = idx;
    uint8_t* list = lists[wave];
    // what this lane reads and writes: columns 8 (lane % 8) .. + 7 of a 64-column block of each 8th row
    const int lr = lane >> 3, lc = 8 * (lane & 7);
    const char* ybase[NM];
#pragma unroll
    for (int mat = 0; mat < NM; ++mat) {
        ybase[mat] = a.y[mat] ? reinterpret_cast<const char*>(static_cast<const T*>(a.y[mat]) + m0 * a.ldy[mat]) : nullptr;
    }
    char* obase = reinterpret_cast<char*>(static_cast<T*>(a.out) + m0 * a.ldo);
    float* tp = turned[wave];

    // the operands of w for ranks 8 c .. + 7, c = c0 + q, and 64 columns from n0
    auto load_w = [&](int mat, int cur, int n0, int c, raw4_t (&f)[4]) __attribute__((always_inline)) {
        const int64_t wrow = a.w[mat].row;
        const T* w = static_cast<const T*>(a.w[mat].w) + cur * a.w[mat].stack + (COLUMNS ? (int64_t)n0 : n0 * wrow);
        const int r = 8 * c;
        if constexpr (COLUMNS) {
            load_columns<T, 4>(
                [&](int i) { return reinterpret_cast<const char*>(w) + ((uint32_t)min(r + i, a.R - 1) * (uint32_t)wrow + 4 * i16) * 2; },
                r < a.R ? a.N - n0 - 4 * i16 : 0, f);
            if (r + 8 > a.R) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[j][e] &= first_rows_mask(e, a.R - r);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const char* p = reinterpret_cast<const char*>(w) + ((uint32_t)min(16 * j + i16, a.N - 1 - n0) * (uint32_t)wrow + r) * 2;
                f[j] = load8(reinterpret_cast<const T*>(p), a.R - r);
            }
        }
    };

    // rows g .. g + ROWS - 1 of the n that the list holds
    auto pass = [&](int cur, int g, int n, auto with) __attribute__((always_inline)) {
        constexpr bool WITH = decltype(with)::value;  // false: the rows without an adapter
        int own[2 * TM];  // this lane's rows; -1: none
#pragma unroll
        for (int i = 0; i < 2 * TM; ++i) own[i] = g + 8 * i + lr < n ? list[g + 8 * i + lr] : -1;
        // two blocks' y and, where registers hold them, w: the next block's are on their way during this one
        constexpr int WB = H == 1 && NM * TM < 4 ? 2 : 1;
        raw4_t y[2][NM][TM][2], wf[WB][NM][H][4];
        auto load_y = [&](int n0, int buf) __attribute__((always_inline)) {
            const bool whole = n0 + 64 <= a.N;
#pragma unroll
            for (int mat = 0; mat < NM; ++mat) {
                if (!a.y[mat]) continue;
#pragma unroll
                for (int i = 0; i < 2 * TM; ++i) {
                    const char* p = ybase[mat] + 2 * n0 + ((uint32_t)max(own[i], 0) * (uint32_t)a.ldy[mat] + lc) * 2;
                    if (own[i] >= 0) y[buf][mat][i >> 1][i & 1] = load8(reinterpret_cast<const T*>(p), whole ? 8 : a.N - n0 - lc);
                }
            }
        };
        auto load_ws = [&](int n0, int buf) __attribute__((always_inline)) {
            if constexpr (WITH && S > 0) {
#pragma unroll
                for (int mat = 0; mat < NM; ++mat) {
#pragma unroll
                    for (int h = 0; h < H; ++h) load_w(mat, cur, n0, S == 1 ? q & 1 : 4 * h + q, wf[buf % WB][mat][h]);
                }
            }
        };
        if (nb_first < nb_end) {
            load_y(64 * nb_first, 0);
            load_ws(64 * nb_first, 0);
        }

        float scale = 1.0f;
        if constexpr (WITH) {
            if (a.scale) scale = a.scale[cur];
            // z: the parts' sums
            const int items = NM * ROWS * R8;
            auto z8 = [&](int i, float (&v)[8]) __attribute__((always_inline)) {
                const int c = i % R8, at = g + i / R8 % ROWS, mat = i / R8 / ROWS;
                const bool wanted = at < n && 8 * c < a.R;
                const int m = m0 + (wanted ? list[at] : 0);
                const float* p = a.z + ((int64_t)mat * a.M + m) * a.R + 8 * c;
                const int64_t plane = (int64_t)a.mats * a.M * a.R;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.0f;
                if (!wanted) return;
#pragma unroll 4
                for (int s = 0; s < a.splits; ++s) {
                    const Chunk<Fp32> k = load_chunk(reinterpret_cast<const Fp32*>(p + s * plane), a.R - 8 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += k.e[e].v;
                }
            };
            if constexpr (!__is_same(T, Bf16)) {
                for (int i = threadIdx.x; i < NM * ROWS; i += kThreads) most[i] = 0u;
                __syncthreads();
            }
            if constexpr (!__is_same(T, Bf16)) {
                for (int i = threadIdx.x; i < items; i += kThreads) {
                    float v[8];
                    z8(i, v);
                    uint32_t size = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) size = max(size, finite_bits(v[e]));
                    atomicMax(&most[i / R8], size);  // a maximum: any order
                }
                __syncthreads();
            }
            for (int i = threadIdx.x; i < items; i += kThreads) {
                float v[8];
                z8(i, v);
                const int c = i % R8, row_at = i / R8, at = g + row_at % ROWS;
                if (a.low && cb == 0 && at < n && 8 * c < a.R) {
                    store_chunk(reinterpret_cast<Fp32*>(a.low) + (int64_t)(m0 + list[at]) * a.R + 8 * c, narrow8<Fp32>(v), a.R - 8 * c);
                }
                Pow2 f{1.0f, 1.0f};
                if constexpr (!__is_same(T, Bf16)) {
                    f = pow2_for<T>(most[row_at]);
                    if (c == 0) down[row_at] = f.down;
                }
                raw4_t hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint16_t first, second;
                    split16<T>(v[e] * f.up, first, second);
                    hi[e >> 1] |= (uint32_t)first << (16 * (e & 1));
                    lo[e >> 1] |= (uint32_t)second << (16 * (e & 1));
                }
                *reinterpret_cast<raw4_t*>(lds + row_at * pitch + 8 * c) = hi;
                *reinterpret_cast<raw4_t*>(lds + row_at * pitch + RP + 8 * c) = lo;
            }
            __syncthreads();
        } else if (a.low && cb == 0 && wave == 0) {
#pragma unroll
            for (int i = 0; i < 2 * TM; ++i) {
                for (int r = lane & 7; own[i] >= 0 && r < a.R; r += 8) a.low[(int64_t)(m0 + own[i]) * a.R + r] = 0.0f;
            }
        }
        auto block = [&](int nb, int buf) __attribute__((always_inline)) {
            const int n0 = 64 * nb;
            const bool whole = n0 + 64 <= a.N;
            if (nb + kWaves < nb_end) {
                load_y(64 * (nb + kWaves), buf ^ 1);
                if constexpr (WB == 2) load_ws(64 * (nb + kWaves), buf ^ 1);
            }
            f32x4 acc[NM][S ? 1 : TM][4];
            auto z_at = [&](int mat, int t, int s) __attribute__((always_inline)) {
                return *reinterpret_cast<const raw4_t*>(lds + (mat * ROWS + 16 * t + i16) * pitch + 32 * s + 8 * q);
            };
            if constexpr (S == 0) {
#pragma unroll
                for (int mat = 0; mat < NM; ++mat) {
#pragma unroll
                    for (int t = 0; t < TM; ++t) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[mat][t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                    for (int h = 0; WITH && h < steps / 2; ++h) {
                        raw4_t f[4];
                        load_w(mat, cur, n0, 4 * h + q, f);
#pragma unroll
                        for (int t = 0; t < TM; ++t) {
                            const raw4_t first = z_at(mat, t, h), second = z_at(mat, t, steps / 2 + h);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                acc[mat][t][j] = mfma16<T>(f[j], first, acc[mat][t][j]);
                                acc[mat][t][j] = mfma16<T>(f[j], second, acc[mat][t][j]);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                if constexpr (S > 0) {
#pragma unroll
                    for (int mat = 0; mat < NM; ++mat) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[mat][0][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int s = 0; WITH && s < S; ++s) {
                            const raw4_t z = z_at(mat, t, s);
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[mat][0][j] = mfma16<T>(wf[buf % WB][mat][s % H][j], z, acc[mat][0][j]);
                        }
                    }
                }
                float o[2][8];
#pragma unroll
                for (int mat = 0; mat < NM; ++mat) {
                    const f32x4(&d)[4] = acc[mat][S ? 0 : t];
                    if constexpr (WITH) {
                        // COLUMNS: column 4 (4 q + e) + j is element e of operand j, else column 16 j + 4 q + e
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const f32x4 v = COLUMNS ? f32x4{d[0][k], d[1][k], d[2][k], d[3][k]} : d[k];
                            *reinterpret_cast<f32x4*>(tp + i16 * kTurnPitch + (COLUMNS ? 16 * q + 4 * k : 16 * k + 4 * q)) = v;
                        }
                        __builtin_amdgcn_wave_barrier();  // to other lanes of the wave, in LDS order
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Chunk<T> base = __builtin_bit_cast(Chunk<T>, y[buf][mat][t][i]);
                        float v[8];
                        if constexpr (WITH) {
                            const float* from = tp + (8 * i + lr) * kTurnPitch + lc;
                            const f32x4 lo = *reinterpret_cast<const f32x4*>(from), hi = *reinterpret_cast<const f32x4*>(from + 4);
                            const float f = __is_same(T, Bf16) ? scale : scale * down[mat * ROWS + 16 * t + 8 * i + lr];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = fmaf(e < 4 ? lo[e] : hi[e - 4], f, a.y[mat] ? widen(base.e[e]) : 0.0f);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = a.y[mat] ? widen(base.e[e]) : 0.0f;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[i][e] = mat == 0 ? v[e] : silu_mul16(o[i][e], v[e]);
                    }
                    __builtin_amdgcn_wave_barrier();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    char* to = obase + 2 * n0 + ((uint32_t)max(own[2 * t + i], 0) * (uint32_t)a.ldo + lc) * 2;
                    const int cnt = whole ? 8 : a.N - n0 - lc;
                    if (own[2 * t + i] >= 0 && cnt > 0) store_chunk(reinterpret_cast<T*>(to), narrow8<T>(o[i]), cnt);
                }
            }
            if constexpr (WB == 1) {
                if (nb + kWaves < nb_end) load_ws(64 * (nb + kWaves), 0);
            }
        };
        for (int nb = nb_first; nb < nb_end; nb += 2 * kWaves) {
            block(nb, 0);
            if (nb + kWaves < nb_end) block(nb + kWaves, 1);
        }
    };
    bool again = false;
    // rows from .. to - 1 of those with this adapter, or without one
    auto rows_of = [&](int cur, int from, int to) __attribute__((always_inline)) {
        const int n = min(list_rows(idx, cur, list), to);
        for (int g = from; g < n; g += ROWS) {
            if (cur < 0) {
                pass(-1, g, n, Part{});
            } else {
                if (again) __syncthreads();  // z of the rows before is read
                again = true;
                pass(cur, g, n, Whole{});
            }
        }
    };
    if constexpr (TM == 1) {
        if (by_row) {
            int cur, from;
            if (leads(idx, blockIdx.y, cur, from)) rows_of(cur, from, from + 16);
            return;
        }
    }
    rows_of(-1, 0, 64);
    for (;;) {
        const int cur = next_adapter(left);
        if (cur < 0) break;
        if (left == cur) left = -1;
        rows_of(cur, 0, 64);
    }
}

constexpr int kTargetWaves = 2048;
constexpr int64_t kMaxBlocks = 1 << 22;  // workgroups of 256 threads in a launch's first dimension

// How a batch's rows are cut.  A batch of up to kMost rows, fewer than 16 per adapter there is, is taken to mix requests: in
// tiles of 64 rows each row has workgroups of its own (the launch's `slots`), of which every 16th of an adapter's rows takes
// 16 of them, so that its weights are read once for these.  (Going through a tile's adapters to find the workgroup's own took
// 3 us at 32 of them.)  Otherwise the rows are taken to be runs of one adapter, and a tile is what a workgroup takes at a
// time: 16 rows of up to kFew, so that there are workgroups enough, with slots too, so that none has two runs' rows, else 64
// or 32, whose adapters it goes through.  64 rows of 16 adapters (GLU, K = 2560 N = 9216, rank 32): second product 18.2
// us with tiles of 16, 11.9 with 64; 512 rows of 512 adapters, 4096 x 4096: both products 372 us as runs, 42 as a mixture.
constexpr int kFew = 256, kMost = 1024;
struct Cut {
    int rows, slots;       // of a tile
    int64_t tiles, units;  // units: expected adapters of all tiles
};
bool is_mixed(int M, int L) { return M <= kMost && M < 16 * (int64_t)L; }
bool few(int M, int L) { return M <= kFew || is_mixed(M, L); }
Cut cut(int M, int L, int tm)
{
    const bool mixed = is_mixed(M, L);
    Cut c;
    c.rows = tm > 1 ? 16 * tm : mixed ? 64 : 16;
    c.tiles = ((int64_t)M + c.rows - 1) / c.rows;
    c.slots = tm > 1 || !few(M, L) ? 1 : M < c.rows ? M : c.rows;
    c.units = !mixed ? c.tiles : c.tiles * L < M ? c.tiles * L : M;
    return c;
}

// Tiles of the first product: 16 TM rows and 16 RT ranks.  Few rows, or a mixture: one instruction's, so that there are more of
// them; else as many as registers hold with a stage in flight.  64 x 64 (from LDS) and 32 x 64, us: 16384 rows of 4096 34.7
// and 40.2, 8192 of 5120 25.2 and 27.0, 5000 of 4096 23.6 and 23.4, 2050 of 4096 18.0 and 15.3.
struct LowTile { int tm, rt; };
LowTile low_tile(int M, int R, int L, bool columns)
{
    if (few(M, L) || columns) return {1, 1};
    return R <= 16 ? LowTile{4, 1} : R <= 32 ? LowTile{4, 2} : M > 4096 ? LowTile{4, 4} : LowTile{2, 4};
}

template <class T, int TM, int RT, int U, bool COLUMNS>
void low_tiles(const LowArgs& a, hipStream_t stream)
{
    const Cut c = cut(a.M, a.L, TM);
    const int rgroups = (a.R + 16 * RT - 1) / (16 * RT);
    for (int64_t t = 0; t < c.tiles; t += kMaxBlocks) {
        const dim3 grid((unsigned)(c.tiles - t < kMaxBlocks ? c.tiles - t : kMaxBlocks), a.splits * rgroups * a.mats, c.slots);
        hipLaunchKernelGGL((adapter_low_kernel<T, TM, RT, U, COLUMNS>), grid, dim3(kThreads), 0, stream, a, c.rows,
                           c.slots > 1, rgroups, (int)t);
    }
}

// whether rows are whole 16-byte chunks as far as whole stages go
bool aligned(const LowArgs& a)
{
    uintptr_t bits = (uintptr_t)a.v | (uintptr_t)(a.ldv * 2);
    for (int i = 0; i < a.mats; ++i) bits |= (uintptr_t)a.w[i].w | (uintptr_t)(a.w[i].stack * 2) | (uintptr_t)(a.w[i].row * 2);
    return (bits & 15) == 0;
}

template <class T, int TM, int RT>
hipError_t low_direct(const LowArgs& a, hipStream_t stream)
{
    constexpr int bytes = kWaves * 2 * 2 * (TM + RT) * 1024;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(adapter_low_tile_kernel<T, TM, RT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const int rgroups = (a.R + 16 * RT - 1) / (16 * RT);
    const int64_t tiles = ((int64_t)a.M + 16 * TM - 1) / (16 * TM);
    for (int64_t t = 0; t < tiles; t += kMaxBlocks) {
        const dim3 grid((unsigned)(tiles - t < kMaxBlocks ? tiles - t : kMaxBlocks), a.splits * rgroups * a.mats);
        hipLaunchKernelGGL((adapter_low_tile_kernel<T, TM, RT>), grid, dim3(kThreads), bytes, stream, a, rgroups, (int)t);
    }
    return hipGetLastError();
}

template <class T, bool COLUMNS>
hipError_t low_launch(const LowArgs& a, hipStream_t stream)
{
    const LowTile t = low_tile(a.M, a.R, a.L, COLUMNS);
    if (COLUMNS || t.tm == 1) low_tiles<T, 1, 1, COLUMNS ? 1 : 2, COLUMNS>(a, stream);
    else if (aligned(a) && t.rt == 1) return low_direct<T, 4, 1>(a, stream);
    else if (aligned(a) && t.rt == 2) return low_direct<T, 4, 2>(a, stream);
    else if (aligned(a) && t.tm == 4) return low_direct<T, 4, 4>(a, stream);
    else if (aligned(a)) return low_direct<T, 2, 4>(a, stream);
    else if (t.rt == 1) low_tiles<T, 4, 1, 2, false>(a, stream);
    else if (t.rt == 2) low_tiles<T, 4, 2, 2, false>(a, stream);
    else low_tiles<T, 2, 4, 1, false>(a, stream);
    return hipGetLastError();
}

template <class T, int TM, int NM, int S, bool COLUMNS>
void out_tiles(const OutArgs& a, hipStream_t stream)
{
    const Cut c = cut(a.M, a.L, TM);
    const int blocks = a.N > 0 ? (a.N + 63) / 64 : 1;  // N == 0: z alone, to low
    // A wave takes several blocks where there are waves enough: as many, rounded up, as make a round of workgroups, two per
    // CU (8192 x 5120, rank 64: 49 us; 63 with half as many), or three such rounds of the pair, whose workgroups take longer.
    // Rounding up leaves fewer: of the pair, 2050 x 12288, rank 16, 1040 workgroups, 51 us (55 with the 780 of a target of two
    // rounds, 56 with the 455 of one).
    const int64_t target = NM == 2 && TM > 1 ? 3 * kTargetWaves : kTargetWaves;
    int per = (int)((c.units * blocks + target - 1) / target);
    per = per < 1 ? 1 : per > 32 ? 32 : per;
    const int cblocks = (blocks + per * kWaves - 1) / (per * kWaves);
    const int64_t fit = kMaxBlocks / cblocks < 1 ? 1 : kMaxBlocks / cblocks;
    const int RP = S ? 16 * S : (a.R + 31) & ~31, rows = 16 * TM;
    const size_t bytes = (size_t)NM * rows * (2 * RP + 8) * 2 + (size_t)NM * rows * 8;
    for (int64_t t = 0; t < c.tiles; t += fit) {
        const dim3 grid((unsigned)((c.tiles - t < fit ? c.tiles - t : fit) * cblocks), c.slots);
        hipLaunchKernelGGL((adapter_out_kernel<T, TM, NM, S, COLUMNS>), grid, dim3(kThreads), bytes, stream, a, c.rows, c.slots > 1,
                           cblocks, per, (int)t);
    }
}

template <class T, int NM, bool COLUMNS>
hipError_t out_launch(const OutArgs& a, hipStream_t stream)
{
    if (a.R > 64) {
        out_tiles<T, 1, NM, 0, COLUMNS>(a, stream);
    } else if (few(a.M, a.L)) {
        if (a.R <= 16) out_tiles<T, 1, NM, 1, COLUMNS>(a, stream);
        else if (a.R <= 32) out_tiles<T, 1, NM, 2, COLUMNS>(a, stream);
        else out_tiles<T, 1, NM, 4, COLUMNS>(a, stream);
    } else {
        if (a.R <= 16) out_tiles<T, NM == 1 ? 4 : 2, NM, 1, COLUMNS>(a, stream);
        else if (a.R <= 32) out_tiles<T, NM == 1 ? 4 : 2, NM, 2, COLUMNS>(a, stream);
        else out_tiles<T, NM == 1 ? 4 : 2, NM, 4, COLUMNS>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace

// Parts of the columns.  A mixed batch: as many as make some 768 workgroups, of one stage per wave at least, but 4 at
// most, which the second product has to add up (one row of 2560, 9216 columns: both products 10.7 us with 10 parts, 8.8
// with 4, 8.9 with 2; 37 rows of 4096, 12288 columns: 19.6, 17.2 and 17.0).  More rows: as many as make a workgroup per CU,
// whose waves then go through more stages each (8192 rows of 5120, 16 ranks, in 256, 512 and 768 workgroups: 18.3, 21.7
// and 25.4 us; 64 ranks 25.2, 32.6 and 41.4).
int adapter_low_splits(int M, int C, int R, int L, int mats, bool columns)
{
    const LowTile t = low_tile(M, R, L, columns);
    const int64_t groups = cut(M, L, t.tm).units * mats * ((R + 16 * t.rt - 1) / (16 * t.rt));
    const int64_t most = ((int64_t)C + kStage * kWaves - 1) / (kStage * kWaves), cap = t.tm == 1 ? 4 : 16;
    int64_t s = groups ? (t.tm == 1 ? 768 : 256) / groups : 1;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s > cap ? cap : s);
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
