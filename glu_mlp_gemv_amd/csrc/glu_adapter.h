// Launch interface of the low-rank adapter kernels (glu_adapter.hip, glu_adapter_grad.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glu {

constexpr int64_t kMaxAdapterRow = (int64_t)1 << 23;  // columns and row strides of every operand: a tile's bytes fit 32 bits

// w: [L][rows][cols] of the operands' type, element (l, i, j) at w + l * stack + i * row + j
struct Stack {
    const void* w;
    int64_t stack, row;
};

// First product: z[split][mat][m][r] = sum over the split's c of v[m][c] w[r][c] (rows: w is [L][R][C]) or of v[m][c] w[c][r]
// (columns: w is [L][C][R]), w that of the row's adapter; zeros for rows without one.
struct LowArgs {
    const void* v;
    Stack w[2];
    const int32_t* index;
    float* z;
    int64_t ldv;
    int M, C, R, L, mats, splits;
};
// columns: the contraction runs down w's columns (else along its rows)
hipError_t adapter_low_launch(int dtype, bool columns, const LowArgs& a, hipStream_t stream);

int adapter_low_splits(int M, int C, int R, int L, int mats, bool columns);

// Second product: out[m][n] = T(y[m][n] + scale sum_r z[m][r] w[n][r]) (w [L][N][R]) or w[r][n] (w [L][R][N]), z the
// sum of its splits; with two mats silu of the first times the second.
struct OutArgs {
    const void* y[2];      // null: zeros
    const float* z;
    Stack w[2];
    const int32_t* index;
    const float* scale;    // [L] or null
    void* out;
    float* low;            // [M][R]: z is stored there too, or null
    int64_t ldy[2], ldo;
    int M, N, R, L, mats, splits;
};
hipError_t adapter_out_launch(int dtype, bool columns, const OutArgs& a, hipStream_t stream);

// Gradient of a stack: grad[l] = T(scale[l] sum over rows m of adapter l of z[m]^T v[m]), for one or two stacks at
// once: da [L][R][K] (z = d, v = x) and db [L][N][R] (z = t, v = dout).
struct GradSide {
    const void* v;     // [M][C], row stride ldv
    const float* z;    // [splits][M][R]
    void* grad;        // null: this side is not wanted
    int64_t ldv;
    int C, splits;
    bool rank_inner;   // grad is [L][C][R], else [L][R][C]
};
struct GradArgs {
    GradSide side[2];
    const int32_t* index;
    const float* scale;
    int32_t* order;    // [M] rows by adapter                     } not used while one item holds an adapter's rows
    int32_t* items;    // [items][4]: adapter, first, count        }
    float* part;       // [items][R][C of both sides]              }
    int M, R, L, rows;  // rows per item
};
int adapter_grad_rows(int M, int64_t C);           // rows per item
bool adapter_grad_direct(int M, int rows);         // one item per adapter, no order and no join
int64_t adapter_grad_items(int M, int L, int rows);
// to[l][r][c] = from[l][c][r], rows of `pitch`; C == 0: nothing
struct Turn {
    Stack from;
    uint16_t* to;
    int C;
    int64_t pitch;
};
// before the other launches, unless direct: the rows by adapter (list) and the second product's weights turned
hipError_t adapter_prepare_launch(const GradArgs& a, bool list, const Turn& w, hipStream_t stream);
hipError_t adapter_grad_launch(int dtype, const GradArgs& a, hipStream_t stream);

}  // namespace glu
