// Gradients of low-rank adapters' weights: for each adapter l
//
//   da[l] = scale[l] sum_{m: index[m] = l} d[m]^T x[m],   db[l] = scale[l] sum_{m: index[m] = l} dout[m]^T t[m]
//
// Bound by memory: x and dout are read once, 4 R operations per number of them.  The contraction runs over rows, so
// the operands lie across it: a lane reads 4 neighbouring columns of 8 rows and turns them into 4 operands by
// byte permutations, without LDS; d or t, which all columns share, goes through LDS, transposed, as two
// numbers of T each.  The rows of an adapter may stand anywhere: a first kernel lists them, in order, and cuts the
// lists into items of `rows` rows, whose fp32 sums a last kernel joins in order.  Up to kDirectRows rows an adapter
// is one item, whose workgroups make the list themselves, and one launch does it all.  16384 rows of 4 adapters, K = N =
// 4096 rank 16: listing and turning 7 us, the sums 68 (268 MB read: 3.9 TB/s, whether a lane reads 8 or 16 bytes, with one to
// eight steps in flight and two to five workgroups a CU), the join 7.5.
#include "../../include/glu_fp8.h"
#include "glu_adapter.h"
#include "glu_mat16.h"

namespace glu {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kDirectRows = 512;
template <int RT> constexpr int kChunkRows = RT == 4 ? 128 : 256;  // rows whose d or t are in LDS at a time
constexpr int kItemStep = 256;        // items are multiples of it
constexpr int kSteps = 2;             // steps of 32 rows in flight
constexpr int kTurn = 256;            // columns that a workgroup turns to rows
constexpr int kOrderThreads = 1024;

int32_t* bounds_of(const GradArgs& a, int64_t items) { return a.items + 4 * items; }  // [L][2]: first, count

// exclusive prefix of v over the workgroup's threads, and the total; scratch: one int per wave
template <int THREADS>
__device__ __forceinline__ int block_prefix(int v, int* scratch, int* total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int p = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(p, d);
        if (lane >= d) p += o;
    }
    __syncthreads();
    if (lane == 63) scratch[wave] = p;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        const int s = scratch[w];
        if (w < wave) before += s;
        all += s;
    }
    *total = all;
    return before + p - v;
}

// An adapter's rows in order, after those of the adapters before it, and its items.  A thread takes 16
// rows at a time, whose numbers it loads together.  Items are numbered first / rows + adapter, which leaves room for all
// of every adapter's whatever the counts.
__device__ __forceinline__ void list_rows(const GradArgs& a, int l, int items, int32_t* bounds, int* scratch)
{
    const int t = threadIdx.x;
    constexpr int EACH = 16;
    auto load = [&](int m0, int (&v)[EACH]) __attribute__((always_inline)) {
        if (m0 + EACH <= a.M) {
            typedef int int4_any __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
            for (int i = 0; i < EACH / 4; ++i) {
                const int4_any d = *reinterpret_cast<const int4_any*>(a.index + m0 + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * i + j] = d[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < EACH; ++i) v[i] = m0 + i < a.M ? a.index[m0 + i] : -1;
        }
    };
    int less = 0, mine = 0, v[EACH];
    for (int m0 = EACH * t; m0 < a.M; m0 += EACH * kOrderThreads) {
        load(m0, v);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            less += v[i] >= 0 && v[i] < l;
            mine += v[i] == l;
        }
    }
    int first, count;
    block_prefix<kOrderThreads>(less, scratch, &first);
    int at = block_prefix<kOrderThreads>(mine, scratch, &count);
    const bool once = a.M <= EACH * kOrderThreads;  // the rows are still at hand, and so is their prefix
    at = once ? first + at : first;
    for (int base = 0; base < a.M; base += EACH * kOrderThreads) {
        const int m0 = base + EACH * t;
        int p = at;
        if (!once) {
            int hits = 0, n;
            if (m0 < a.M) {
                load(m0, v);
#pragma unroll
                for (int i = 0; i < EACH; ++i) hits += v[i] == l;
            }
            p += block_prefix<kOrderThreads>(hits, scratch, &n);
            at += n;
        }
        if (m0 < a.M) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if (v[i] == l) a.order[p++] = m0 + i;
            }
        }
    }
    const int base = first / a.rows + l, end = l == a.L - 1 ? items : (first + count) / a.rows + l + 1;
    for (int k = base + t; k < end; k += kOrderThreads) {
        const int from = min(count, (k - base) * a.rows);
        int32_t* e = a.items + 4 * (int64_t)k;
        e[0] = l;
        e[1] = first + from;
        e[2] = min(a.rows, count - from);
    }
    if (t == 0) {
        bounds[2 * l] = first;
        bounds[2 * l + 1] = count;
    }
}

// Columns c0 .. + 255 of one adapter's w [C][R] as rows: wt[r][c] = w[c][r]
__device__ __forceinline__ void turn(const Turn& w, int R, int l, int c0, uint16_t (*tile)[kTurn + 2])
{
    const uint16_t* from = static_cast<const uint16_t*>(w.from.w) + l * w.from.stack;
    uint16_t* to = w.to + (int64_t)l * R * w.pitch;
    const int bits = R <= 16 ? 4 : 5, ranks = 1 << bits;
    for (int r0 = 0; r0 < R; r0 += ranks) {
        if (r0) __syncthreads();
        for (int i = threadIdx.x; i < kTurn * ranks; i += kOrderThreads) {
            const int c = i >> bits, r = i & (ranks - 1);
            if (c0 + c < w.C && r0 + r < R) tile[r][c] = from[(c0 + c) * w.from.row + r0 + r];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kTurn * ranks; i += kOrderThreads) {
            const int c = i % kTurn, r = i / kTurn;
            if (c0 + c < w.C && r0 + r < R) to[(int64_t)(r0 + r) * w.pitch + c0 + c] = tile[r][c];
        }
    }
}

// What the other kernels need first: the rows by adapter, one workgroup each, and w turned, which the first product
// would otherwise read 2 bytes at a time, once per tile of rows.
__global__ void __launch_bounds__(kOrderThreads)
adapter_prepare_kernel(GradArgs a, int listed, int items, int32_t* bounds, Turn w, int cblocks, int64_t block0)
{
    __shared__ int scratch[kOrderThreads / 64];
    __shared__ uint16_t tile[32][kTurn + 2];
    const int64_t b = block0 + blockIdx.x;
    if (b < listed) list_rows(a, (int)b, items, bounds, scratch);
    else turn(w, a.R, (int)((b - listed) / cblocks), (int)((b - listed) % cblocks) * kTurn, tile);
}

// One item, 64 columns per wave.  DIRECT: the item is the adapter, and its sums are the gradient.
template <class T, int RT, bool DIRECT>
__global__ void __launch_bounds__(kThreads, RT == 4 ? 2 : 3) adapter_grad_kernel(GradArgs a, int cblocks0, int cblocks, int64_t columns,
                                                                   int item0)
{
    constexpr int CHUNK = kChunkRows<RT>, PITCH = CHUNK + 8;
    __shared__ uint16_t zt[2][16 * RT * PITCH];  // [first, second number][rank][row]
    __shared__ int64_t offset[CHUNK];            // of a chunk's rows of v, in bytes
    __shared__ int list[DIRECT ? kDirectRows : 1];
    __shared__ uint32_t most[16 * RT];
    __shared__ int scratch[kWaves];
    const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int item = item0 + blockIdx.x / cblocks, block = blockIdx.x % cblocks;
    const int which = block >= cblocks0 ? 1 : 0;
    const GradSide& s = a.side[which];
    const int c = ((block - (which ? cblocks0 : 0)) * kWaves + wave) * 64 + 4 * i16;  // this lane's 4 columns
    const int r0 = blockIdx.y * 16 * RT, ranks = min(16 * RT, a.R - r0);

    int l, count;
    const int32_t* order = nullptr;
    if constexpr (DIRECT) {
        l = item;
        count = 0;
        for (int m0 = 0; m0 < a.M; m0 += kThreads) {
            const int m = m0 + threadIdx.x;
            const int hit = m < a.M && a.index[m] == l;
            int n;
            const int p = block_prefix<kThreads>(hit, scratch, &n);
            if (hit) list[count + p] = m;
            count += n;
        }
    } else {
        const int32_t* e = a.items + 4 * (int64_t)item;
        l = e[0];
        order = a.order + e[1];
        count = e[2];
        if (count <= 0) return;
    }
    __syncthreads();
    auto row_at = [&](int i) __attribute__((always_inline)) { return DIRECT ? list[i] : order[i]; };
    // EACH ranks of one row of d or t: the sum of its parts
    constexpr int EACH = 16 * RT * CHUNK / kThreads;
    static_assert(EACH % 8 == 0 && 16 * RT % EACH == 0 && CHUNK % 64 == 0, "whole chunks of ranks, the same for a wave");
    auto z_of = [&](int row, int r, float (&z)[EACH]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) z[i] = 0.0f;
        const float* p = s.z + (int64_t)row * a.R + r0 + r;
        for (int k = 0; k < s.splits; ++k, p += (int64_t)a.M * a.R) {
#pragma unroll
            for (int i = 0; i < EACH; i += 8) {
                if (r + i < ranks) {
                    const Chunk<Fp32> d = load_chunk(reinterpret_cast<const Fp32*>(p + i), ranks - r - i);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[i + e] += d.e[e].v;
                }
            }
        }
    };
    const int my_row = threadIdx.x % CHUNK, my_rank = threadIdx.x / CHUNK * EACH;
    if constexpr (!__is_same(T, Bf16)) {  // one power of two per rank for all of the item's rows
        if (threadIdx.x < 16 * RT) most[threadIdx.x] = 0u;
        __syncthreads();
        uint32_t top[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) top[i] = 0u;
        for (int i = my_row; i < count; i += CHUNK) {
            float z[EACH];
            z_of(row_at(i), my_rank, z);
#pragma unroll
            for (int e = 0; e < EACH; ++e) top[e] = max(top[e], finite_bits(z[e]));
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) {  // a wave's lanes have the same ranks
            const uint32_t m = wave_max(top[e]);
            if (lane == e) atomicMax(&most[my_rank + e], m);  // a maximum: any order
        }
        __syncthreads();
    }

    f32x4 acc[RT][4];
#pragma unroll
    for (int k = 0; k < RT; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[k][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const char* v = reinterpret_cast<const char*>(static_cast<const T*>(s.v) + c);
    for (int base = 0; base < count; base += CHUNK) {
        const int n = min(CHUNK, count - base), steps = (n + 31) >> 5;
        if (base) __syncthreads();
        for (int i = threadIdx.x; i < 32 * steps; i += kThreads) offset[i] = row_at(base + min(i, n - 1)) * s.ldv * 2;
        __syncthreads();
        constexpr int U = kSteps;
        uint32_t raw[U][8][2];
        auto load = [&](int u, int k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const char* p = v + offset[32 * k + 8 * q + i];
                if (c + 4 <= s.C) {
                    const raw2_t d = *reinterpret_cast<const u32x2_any*>(p);
                    raw[u][i][0] = d[0];
                    raw[u][i][1] = d[1];
                } else {
                    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        raw[u][i][d] = (c + 2 * d < s.C ? (uint32_t)e[2 * d] : 0u) | (c + 2 * d + 1 < s.C ? (uint32_t)e[2 * d + 1] << 16 : 0u);
                    }
                }
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < steps) load(u, u);
        }
        // the chunk's d or t while its rows are on their way
        if (my_row < 32 * steps) {
            float z[EACH];
            if (my_row < n) {
                z_of(row_at(base + my_row), my_rank, z);
            } else {
#pragma unroll
                for (int e = 0; e < EACH; ++e) z[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                const int r = my_rank + e;
                const float f = __is_same(T, Bf16) ? 1.0f : pow2_for<T>(most[r]).up;
                uint16_t hi, lo;
                split16<T>(z[e] * f, hi, lo);
                zt[0][r * PITCH + my_row] = hi;
                zt[1][r * PITCH + my_row] = lo;
            }
        }
        __syncthreads();
        auto use = [&](int u, int k) __attribute__((always_inline)) {
            raw4_t vf[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    vf[2 * d][h] = __builtin_amdgcn_perm(raw[u][2 * h + 1][d], raw[u][2 * h][d], 0x05040100u);
                    vf[2 * d + 1][h] = __builtin_amdgcn_perm(raw[u][2 * h + 1][d], raw[u][2 * h][d], 0x07060302u);
                }
            }
            const int i0 = 32 * k + 8 * q;
            if (32 * k + 32 > n) {  // rows past the last are a row again: not even a NaN of theirs may count twice
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) vf[j][e] &= first_rows_mask(e, n - i0);
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const raw4_t hi = *reinterpret_cast<const raw4_t*>(&zt[0][(16 * t + i16) * PITCH + i0]);
                const raw4_t lo = *reinterpret_cast<const raw4_t*>(&zt[1][(16 * t + i16) * PITCH + i0]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[t][j] = mfma16<T>(hi, vf[j], acc[t][j]);
                    acc[t][j] = mfma16<T>(lo, vf[j], acc[t][j]);
                }
            }
        };
        for (int k = 0; k < steps; k += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k + u < steps) use(u, k + u);
                if (k + u + U < steps) load(u, k + u + U);
            }
        }
    }

    const float scale = DIRECT && a.scale ? a.scale[l] : 1.0f;
    const int64_t side = which && a.side[0].grad ? a.side[0].C : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = 16 * t + 4 * q;  // this lane's 4 ranks and columns
        float v[4][4];                 // [rank][column]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = __is_same(T, Bf16) ? 1.0f : pow2_for<T>(most[r + e]).down;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[e][j] = acc[t][j][e] * f;
        }
        const bool whole = r + 4 <= ranks && c + 4 <= s.C;
        if constexpr (DIRECT) {
            T* grad = static_cast<T*>(s.grad);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 4 neighbours at a time: columns of a rank, or ranks of a column
                uint16_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = count ? bits16<T>(scale * (s.rank_inner ? v[k][i] : v[i][k])) : (uint16_t)0;
                const int64_t at = s.rank_inner ? ((int64_t)l * s.C + c + i) * a.R + r0 + r
                                                : ((int64_t)l * a.R + r0 + r + i) * s.C + c;
                if (whole) {
                    *reinterpret_cast<u32x2_any*>(grad + at) = raw2_t{o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16};
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool in = s.rank_inner ? r + k < ranks && c + i < s.C : r + i < ranks && c + k < s.C;
                        if (in) reinterpret_cast<uint16_t*>(grad)[at + k] = o[k];
                    }
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float* to = a.part + ((int64_t)item * a.R + r0 + r + e) * columns + side + c;
                if (whole) {
                    raw4_t o;
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = __float_as_uint(v[e][j]);
                    *reinterpret_cast<u32x4_any*>(to) = o;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (r + e < ranks && c + j < s.C) to[j] = v[e][j];
                    }
                }
            }
        }
    }
}

// The items' sums, in order, to the gradient: a thread has 4 columns of a rank (da) or 4 ranks of a column (db), which
// are neighbours where they are stored, and neighbouring threads neighbouring columns, which are where they are read.
// The first `units0` units of workgroups of an adapter are the first side's.
template <class T>
__global__ void __launch_bounds__(kThreads) adapter_join_kernel(GradArgs a, const int32_t* bounds, int64_t columns,
                                                                int units0, int units, int l0)
{
    const int l = l0 + blockIdx.x / units, unit = blockIdx.x % units;
    const int which = unit >= units0 ? 1 : 0;
    const GradSide& s = a.side[which];
    const int inner = s.rank_inner ? s.C : (s.C + 3) >> 2, blocks = (inner + kThreads - 1) / kThreads;
    const int u = unit - (which ? units0 : 0), i = u % blocks * kThreads + threadIdx.x;
    if (i >= inner) return;
    const int r = s.rank_inner ? u / blocks * 4 : u / blocks, c = s.rank_inner ? i : 4 * i;
    const int n_here = s.rank_inner ? min(4, a.R - r) : min(4, s.C - c);
    const int64_t step = s.rank_inner ? columns : 1;
    const int first = bounds[2 * l], count = bounds[2 * l + 1];
    const int n = (count + a.rows - 1) / a.rows;
    const int64_t item = (int64_t)a.R * columns;
    const float* p = a.part + (first / a.rows + l) * item + r * columns + (which && a.side[0].grad ? a.side[0].C : 0) + c;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n_here == 4) {
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += p[k * item + j * step];
        }
    } else {
        for (int k = 0; k < n; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j < n_here) v[j] += p[k * item + j * step];
            }
        }
    }
    const float scale = a.scale ? a.scale[l] : 1.0f;
    T* to = static_cast<T*>(s.grad) + (s.rank_inner ? ((int64_t)l * s.C + c) * a.R + r : ((int64_t)l * a.R + r) * s.C + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j < n_here) to[j] = narrow<T>(n ? scale * v[j] : 0.0f);
    }
}

constexpr int64_t kMaxBlocks = 1 << 22;

template <class T, int RT>
void grad_items(const GradArgs& a, bool direct, int64_t items, int cblocks0, int cblocks, int64_t columns,
                hipStream_t stream)
{
    const int rgroups = (a.R + 16 * RT - 1) / (16 * RT);
    const int64_t fit = kMaxBlocks / cblocks < 1 ? 1 : kMaxBlocks / cblocks;
    for (int64_t i = 0; i < items; i += fit) {
        const dim3 grid((unsigned)((items - i < fit ? items - i : fit) * cblocks), rgroups);
        if (direct) {
            hipLaunchKernelGGL((adapter_grad_kernel<T, RT, true>), grid, dim3(kThreads), 0, stream, a, cblocks0, cblocks,
                               columns, (int)i);
        } else {
            hipLaunchKernelGGL((adapter_grad_kernel<T, RT, false>), grid, dim3(kThreads), 0, stream, a, cblocks0, cblocks,
                               columns, (int)i);
        }
    }
}

template <class T>
hipError_t grad_launch(const GradArgs& a, hipStream_t stream)
{
    const bool direct = adapter_grad_direct(a.M, a.rows);
    const int64_t items = direct ? a.L : adapter_grad_items(a.M, a.L, a.rows);
    const int64_t c0 = a.side[0].grad ? a.side[0].C : 0, c1 = a.side[1].grad ? a.side[1].C : 0, columns = c0 + c1;
    const int cblocks0 = (int)((c0 + 64 * kWaves - 1) / (64 * kWaves)), cblocks1 = (int)((c1 + 64 * kWaves - 1) / (64 * kWaves));
    const int cblocks = cblocks0 + cblocks1;
    if (a.R <= 16) grad_items<T, 1>(a, direct, items, cblocks0, cblocks, columns, stream);
    else if (a.R <= 32) grad_items<T, 2>(a, direct, items, cblocks0, cblocks, columns, stream);
    else grad_items<T, 4>(a, direct, items, cblocks0, cblocks, columns, stream);
    if (!direct) {
        auto units = [&](const GradSide& s) {
            const int inner = s.rank_inner ? s.C : (s.C + 3) / 4;
            return s.grad ? (inner + kThreads - 1) / kThreads * (s.rank_inner ? (a.R + 3) / 4 : a.R) : 0;
        };
        const int units0 = units(a.side[0]), all = units0 + units(a.side[1]);
        const int fit = kMaxBlocks / all < 1 ? 1 : (int)(kMaxBlocks / all);
        for (int l = 0; l < a.L; l += fit) {
            hipLaunchKernelGGL(adapter_join_kernel<T>, dim3((unsigned)((a.L - l < fit ? a.L - l : fit) * all)), dim3(kThreads), 0,
                               stream, a, bounds_of(a, items), columns, units0, all, l);
        }
    }
    return hipGetLastError();
}

}  // namespace

bool adapter_grad_direct(int M, int rows) { return M <= kDirectRows && M <= rows; }

// Items that make some 1024 workgroups with the columns' blocks, each of a few hundred rows at least so that the
// fp32 sums that they leave stay far below the bytes they read.
int adapter_grad_rows(int M, int64_t C)
{
    if (M <= kDirectRows) return kDirectRows;
    const int64_t cblocks = (C + 64 * kWaves - 1) / (64 * kWaves);
    const int64_t rows = ((int64_t)M * cblocks / 1024 + kItemStep - 1) / kItemStep * kItemStep;
    return (int)(rows < kItemStep ? kItemStep : rows > 4096 ? 4096 : rows);
}

int64_t adapter_grad_items(int M, int L, int rows) { return (int64_t)M / rows + L; }

hipError_t adapter_prepare_launch(const GradArgs& a, bool list, const Turn& w, hipStream_t stream)
{
    const int64_t items = adapter_grad_items(a.M, a.L, a.rows);
    const int cblocks = (w.C + kTurn - 1) / kTurn, listed = list ? a.L : 0;
    const int64_t blocks = listed + (int64_t)a.L * cblocks, fit = 1 << 21;
    for (int64_t b = 0; b < blocks; b += fit) {
        hipLaunchKernelGGL(adapter_prepare_kernel, dim3((unsigned)(blocks - b < fit ? blocks - b : fit)), dim3(kOrderThreads), 0,
                           stream, a, listed, (int)items, bounds_of(a, items), w, cblocks, b);
    }
    return hipGetLastError();
}

hipError_t adapter_grad_launch(int dtype, const GradArgs& a, hipStream_t stream)
{
    return dtype == GLU_DTYPE_BF16 ? grad_launch<Bf16>(a, stream) : grad_launch<Fp16>(a, stream);
}

}  // namespace glu
