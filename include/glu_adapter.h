/*
 * glu_adapter.h -- low-rank adapters of many requests beside a shared projection (gfx950).
 *
 *   t[m]   = x[m] a[i]^T                         i = index[m], fp32, [R]
 *   out[m] = T(y[m] + scale[i] t[m] b[i]^T)      [N]
 *
 * y is what the shared projection gave (glu_grouped_gemv, glu_fp8_linear, any other).  Each row of the batch names its
 * adapter; a row whose index is not in [0, L) has none, and its out is y.  glu_adapter_glu is the pair of gate and up
 * projections with the activation behind it: out = T(silu(g) u), g and u the sums above before any rounding.  As in fp32's own g / (1 + exp(-g)),
 * silu(g) is 0 where exp(-g) passes its range, from g = -87 (2^-119) down.
 * Rows of one adapter may stand anywhere in the batch: a decode batch of many requests and a prefill, in which long
 * runs of rows share one, are the same call.  The rows that share one should be neighbours in batches of more than 1024 rows,
 * or of 16 rows per adapter of the stacks and more: others are as right, but slower.
 *
 * An infinity in b (in the gradients, in dout or x) gives infinite results or NaN, as it meets two numbers of which one may be 0.
 *
 * t stays fp32: it goes into the second product as two numbers of T, its rounding and the rounding of what that left, so
 * that at most 2^-17 of it is lost (FP16: 2^-23): a result that lies so close to a border between two numbers of T may be the
 * other one, about one in a thousand (BF16).  Rows do not touch each other: a NaN in one request's rows or
 * adapter stays there.
 *
 * T is BF16 or FP16 (GLU_DTYPE_*, glu_fp8.h) and is the type of every array but index (int32), scale and low (fp32).
 * Ranks of a stack are padded with zeros to the largest.
 *
 * Ownership, execution, determinism and errors are those of glu_gemv.h: all arrays are device memory of the caller,
 * calls are asynchronous on `stream`, may be captured into a HIP graph, allocate nothing, and validate their
 * arguments before any HIP call.  Row strides are in elements, at least the row length and at most 2^23, and so are N and
 * K; the elements of a row are contiguous; pointers need the alignment of one element.  index is read on the device: nothing is known of it before.
 */
#ifndef GLU_ADAPTER_H
#define GLU_ADAPTER_H

#include <stdint.h>

#include "glu_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GLU_ADAPTER_MAX_RANK 256

/* L adapters: element (l, r, k) of a [L, R, K] at a + l * a_stack + r * a_row + k, (l, n, r) of b [L, N, R] at
 * b + l * b_stack + n * b_row + r.  Rows and adapters do not overlap. */
typedef struct glu_adapter {
    const void* a;
    const void* b;
    int64_t a_stack, a_row, b_stack, b_row;
} glu_adapter;

typedef struct glu_adapter_sizes {
    int64_t M;  /* rows of x */
    int64_t N;  /* columns of y */
    int64_t K;  /* columns of x */
    int64_t R;  /* rank, 1 to GLU_ADAPTER_MAX_RANK */
    int64_t L;  /* adapters, at least 1 */
} glu_adapter_sizes;

/*
 * scale [L] may be NULL (all 1).  out may be exactly y (same pointer and stride), any other overlap of an output is
 * refused.  low [M, R] fp32 dense, may be NULL, receives t (zeros for rows without an adapter), which the backward
 * reads.  M == 0 or N == 0 without low: GLU_OK, nothing launched.  K == 0: t is zero.
 * workspace: glu_adapter_workspace(1, ...) bytes, 16-byte aligned (NULL if 0).
 */
glu_status glu_adapter_add(const void* y, int64_t ldy, const void* x, int64_t ldx, const glu_adapter* ab,
                           const int32_t* index, const float* scale, void* out, int64_t ldo, float* low,
                           const glu_adapter_sizes* sizes, int dtype, void* workspace, int64_t workspace_bytes,
                           void* stream);

/* gate and up [M, N]; one index and scale for both adapters of a row.  out may be exactly gate or up.
 * workspace: glu_adapter_workspace(2, ...) bytes. */
glu_status glu_adapter_glu(const void* gate, int64_t ldg, const void* up, int64_t ldu, const void* x, int64_t ldx,
                           const glu_adapter* gate_ab, const glu_adapter* up_ab, const int32_t* index,
                           const float* scale, void* out, int64_t ldo, const glu_adapter_sizes* sizes, int dtype,
                           void* workspace, int64_t workspace_bytes, void* stream);

/* mats: 1 (add) or 2 (GLU) */
glu_status glu_adapter_workspace(int mats, const glu_adapter_sizes* sizes, int64_t* bytes);

/*
 * Gradients of glu_adapter_add for dout [M, N] (y's gradient is dout itself), with d[m] = dout[m] b[i], fp32:
 *   dx[m]  = T(scale[i] d[m] a[i])                         zeros for rows without an adapter
 *   da[l]  = T(scale[l] sum_{m: i = l} d[m]^T x[m])        [L, R, K] dense
 *   db[l]  = T(scale[l] sum_{m: i = l} dout[m]^T t[m])     [L, N, R] dense
 * low is the forward's t.  Any of dx, da and db may be NULL: it is not computed.  The rows are summed in fp32 in an
 * order fixed by the sizes and index: deterministic.  An adapter without rows gets zeros.  The sum's operand d or t is two
 * numbers of T as above.  M <= 2^24 and L <= 65536: GLU_ERR_BAD_SHAPE beyond.
 * workspace: glu_adapter_backward_workspace() bytes, 16-byte aligned (NULL if 0).
 */
glu_status glu_adapter_backward(const void* dout, int64_t ldd, const void* x, int64_t ldx, const glu_adapter* ab,
                                const int32_t* index, const float* scale, const float* low, void* dx, int64_t lddx,
                                void* da, void* db, const glu_adapter_sizes* sizes, int dtype, void* workspace,
                                int64_t workspace_bytes, void* stream);
glu_status glu_adapter_backward_workspace(const glu_adapter_sizes* sizes, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GLU_ADAPTER_H */
