// Gradients of low-rank adapters' weights: for each adapter l
//
//   da[l] = scale[l] sum_{m: index[m] = l} d[m]^T x[m],   db[l] = scale[l] sum_{m: index[m] = l} dout[m]^T t[m]
//
// Bound by memory: x and dout are read once, 4 R operations per number of them.  The contraction runs over rows, so
// the operands lie across it: a lane reads 4 neighbouring columns of 8 rows and turns them into 4 operands by
// byte permutations, without LDS; d or t, which all columns share, goes through LDS, transposed, as two
// numbers of T each.  The rows of an adapter may stand anywhere: a first kernel lists them, in order, and cuts the
// lists into items of `rows` rows, whose fp32 sums a last kernel joins in order.  Up to kDirectRows rows an adapter
// is one item, whose workgroups make the list themselves, and one launch does it all.
#include "../../include/glu_fp8.h"
#include "glu_adapter.h"
#include "glu_mat16.h"

namespace glu {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kDirectRows = 512;
constexpr int kChunkRows = 128;       // rows whose d or t are in LDS at a time
constexpr int kPitch = kChunkRows + 8;
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

// One workgroup per adapter: its rows in order, after those of the adapters before it, and its items.  Items are
// numbered first / rows + adapter, which leaves room for all of every adapter's whatever the counts.
__global__ void __launch_bounds__(kOrderThreads) adapter_order_kernel(GradArgs a, int items, int32_t* bounds)
{
    __shared__ int scratch[kOrderThreads / 64];
    const int l = blockIdx.x, t = threadIdx.x;
    int less = 0, mine = 0;
    for (int m = t; m < a.M; m += kOrderThreads) {
        const int i = a.index[m];
        less += i >= 0 && i < l;
        mine += i == l;
    }
    int first, count;
    block_prefix<kOrderThreads>(less, scratch, &first);
    block_prefix<kOrderThreads>(mine, scratch, &count);
    int at = first;
    for (int m0 = 0; m0 < a.M; m0 += kOrderThreads) {
        const int m = m0 + t;
        const int hit = m < a.M && a.index[m] == l;
        int n;
        const int p = block_prefix<kOrderThreads>(hit, scratch, &n);
        if (hit) a.order[at + p] = m;
        at += n;
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

// One item, 64 columns per wave.  DIRECT: the item is the adapter, and its sums are the gradient.
template <class T, int RT, bool DIRECT>
__global__ void __launch_bounds__(kThreads) adapter_grad_kernel(GradArgs a, int cblocks0, int cblocks, int64_t columns,
                                                                int item0)
{
    __shared__ uint16_t zt[2][16 * RT * kPitch];  // [first, second number][rank][row]
    __shared__ int list[DIRECT ? kDirectRows : kChunkRows];
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
    auto z_at = [&](int row, int r) __attribute__((always_inline)) {
        const float* p = s.z + (int64_t)row * a.R + r0 + r;
        float v = *p;
        for (int k = 1; k < s.splits; ++k) v += p[(int64_t)k * a.M * a.R];
        return v;
    };
    if constexpr (!__is_same(T, Bf16)) {  // one power of two per rank for all of the item's rows
        if (threadIdx.x < 16 * RT) most[threadIdx.x] = 0u;
        __syncthreads();
        for (int j = threadIdx.x; j < count * ranks; j += kThreads) {
            atomicMax(&most[j % ranks], abs_bits(z_at(row_at(j / ranks), j % ranks)));
        }
        __syncthreads();
    }

    f32x4 acc[RT][4];
#pragma unroll
    for (int k = 0; k < RT; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[k][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int base = 0; base < count; base += kChunkRows) {
        const int n = min(kChunkRows, count - base);
        if (base) __syncthreads();
        if constexpr (!DIRECT) {
            if (threadIdx.x < kChunkRows) list[threadIdx.x] = order[base + min((int)threadIdx.x, n - 1)];
            __syncthreads();
        }
        const int lbase = DIRECT ? base : 0;
        const int padded = (n + 31) & ~31;
        for (int j = threadIdx.x; j < padded * 16 * RT; j += kThreads) {
            const int r = j % (16 * RT), i = j / (16 * RT);
            uint16_t hi = 0, lo = 0;
            if (i < n && r < ranks) {
                const float f = __is_same(T, Bf16) ? 1.0f : pow2_for<T>(most[r]).up;
                split16<T>(z_at(list[lbase + i], r) * f, hi, lo);
            }
            zt[0][r * kPitch + i] = hi;
            zt[1][r * kPitch + i] = lo;
        }
        __syncthreads();
        const T* v = static_cast<const T*>(s.v);
#pragma unroll 2
        for (int k = 0; k < n; k += 32) {
            raw4_t vf[4];
            const int i0 = k + 8 * q;
            load_columns<T, 4>([&](int i) { return v + list[lbase + min(i0 + i, n - 1)] * s.ldv + c; }, s.C - c, vf);
            if (k + 32 > n) {  // rows past the last are a row again: not even a NaN of theirs may count twice
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) vf[j][e] &= first_rows_mask(e, n - i0);
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const raw4_t hi = *reinterpret_cast<const raw4_t*>(&zt[0][(16 * t + i16) * kPitch + i0]);
                const raw4_t lo = *reinterpret_cast<const raw4_t*>(&zt[1][(16 * t + i16) * kPitch + i0]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[t][j] = mfma16<T>(hi, vf[j], acc[t][j]);
                    acc[t][j] = mfma16<T>(lo, vf[j], acc[t][j]);
                }
            }
        }
    }

    const float scale = DIRECT && a.scale ? a.scale[l] : 1.0f;
    const int64_t offset = which ? a.side[0].grad ? a.side[0].C : 0 : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * t + 4 * q + e;  // of this group of ranks
            if (r >= ranks) continue;
            const float f = __is_same(T, Bf16) ? 1.0f : pow2_for<T>(most[r]).down;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (c + j >= s.C) continue;
                const float sum = acc[t][j][e] * f;
                if constexpr (DIRECT) {
                    const int64_t at = s.rank_inner ? ((int64_t)l * s.C + c + j) * a.R + r0 + r
                                                    : ((int64_t)l * a.R + r0 + r) * s.C + c + j;
                    static_cast<T*>(s.grad)[at] = narrow<T>(count ? scale * sum : 0.0f);
                } else {
                    a.part[((int64_t)item * a.R + r0 + r) * columns + offset + c + j] = sum;
                }
            }
        }
    }
}

// The items' sums of 4 ranks and 4 columns of an adapter, in order, to the gradient
template <class T>
__global__ void __launch_bounds__(kThreads) adapter_join_kernel(GradArgs a, const int32_t* bounds, int64_t columns,
                                                                int quads, int64_t total, int64_t first_thread)
{
    const int64_t id = first_thread + (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int rquads = (a.R + 3) >> 2;
    const int cq = (int)(id % quads);
    const int rq = (int)(id / quads % rquads), l = (int)(id / quads / rquads);
    const int quads0 = a.side[0].grad ? (a.side[0].C + 3) >> 2 : 0;
    const int which = cq >= quads0 ? 1 : 0;
    const GradSide& s = a.side[which];
    const int c = 4 * (cq - (which ? quads0 : 0)), r = 4 * rq;
    const int64_t offset = which ? (a.side[0].grad ? a.side[0].C : 0) : 0;
    const int first = bounds[2 * l], count = bounds[2 * l + 1];
    const int base = first / a.rows + l, n = (count + a.rows - 1) / a.rows;
    float v[4][4] = {};
    const bool whole = r + 4 <= a.R && c + 4 <= s.C;
    for (int k = 0; k < n; ++k) {
        const float* p = a.part + ((int64_t)(base + k) * a.R + r) * columns + offset + c;
        if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const raw4_t d = *reinterpret_cast<const u32x4_any*>(p + i * columns);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] += __uint_as_float(d[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (r + i < a.R && c + j < s.C) v[i][j] += p[i * columns + j];
                }
            }
        }
    }
    const float scale = a.scale ? a.scale[l] : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (r + i >= a.R || c + j >= s.C) continue;
            const int64_t at = s.rank_inner ? ((int64_t)l * s.C + c + j) * a.R + r + i
                                            : ((int64_t)l * a.R + r + i) * s.C + c + j;
            static_cast<T*>(s.grad)[at] = narrow<T>(n ? scale * v[i][j] : 0.0f);
        }
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
    if (!direct) {
        hipLaunchKernelGGL(adapter_order_kernel, dim3(a.L), dim3(kOrderThreads), 0, stream, a, (int)items,
                           bounds_of(a, items));
    }
    const int cblocks = cblocks0 + cblocks1;
    if (a.R <= 16) grad_items<T, 1>(a, direct, items, cblocks0, cblocks, columns, stream);
    else if (a.R <= 32) grad_items<T, 2>(a, direct, items, cblocks0, cblocks, columns, stream);
    else grad_items<T, 4>(a, direct, items, cblocks0, cblocks, columns, stream);
    if (!direct) {
        const int quads = (int)((c0 + 3) / 4 + (c1 + 3) / 4);
        const int64_t total = (int64_t)a.L * ((a.R + 3) / 4) * quads;
        for (int64_t t = 0; t < total; t += kMaxBlocks * kThreads) {
            const int64_t blocks = (total - t + kThreads - 1) / kThreads;
            hipLaunchKernelGGL(adapter_join_kernel<T>, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)),
                               dim3(kThreads), 0, stream, a, bounds_of(a, items), columns, quads, total, t);
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
    int64_t rows = ((int64_t)M * cblocks / 1024 + kChunkRows - 1) / kChunkRows * kChunkRows;
    return (int)(rows < 2 * kChunkRows ? 2 * kChunkRows : rows > 4096 ? 4096 : rows);
}

int64_t adapter_grad_items(int M, int L, int rows) { return (int64_t)M / rows + L; }

hipError_t adapter_grad_launch(int dtype, const GradArgs& a, hipStream_t stream)
{
    return dtype == GLU_DTYPE_BF16 ? grad_launch<Bf16>(a, stream) : grad_launch<Fp16>(a, stream);
}

}  // namespace glu
