/*
 * glu_fp8.h -- the 8-bit decoder-MLP path around the GLU projection (gfx950):
 * residual addition + RMS norm, conversion to block-scaled e4m3, and products
 * on block-scaled e4m3 operands.
 *
 *   h   = T(x + residual)                      T: the input's type
 *   r   = 1 / sqrt(mean_k h^2 + eps)           fp32
 *   y   = h r w                                fp32, then T or scaled e4m3
 *
 * Block-scaled e4m3 (OCP e4m3fn, largest finite value 448): a stored value q
 * stands for q * s, s fp32.  A row of activations has one s per 128 columns;
 * a weight [N, K] one per block of 128 rows x 128 columns, the last of either
 * possibly partial.  Conversion: s = max(amax / 448, 2^-126) (an all-zero
 * group keeps finite quotients), q = e4m3(v / s), to nearest even; a NaN in a
 * group makes its s and all its q NaN, an infinity makes s infinite, the
 * group's finite values 0 and its infinite ones NaN.
 *
 * Products: out[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in block b} x[m, k] w[n, k],
 * glu_fp8_dual_glu gives silu(gate) * up of two such sums, evaluated in fp32
 * and rounded once to the output's type.  The sums are fp32, except that on the fast layout with more than 16 rows of x and
 * a 16-bit output they run on the matrix unit's 8-bit path, which within 8 neighbouring products drops what lies 13
 * to 14 bits below the largest and adds the eighths in fp32: a row's result can differ in that between a call of 16
 * rows and one of 17, and between layouts.
 *
 * Ownership, execution, determinism and errors are those of glu_gemv.h: all
 * arrays are device memory of the caller, calls are asynchronous on `stream`,
 * may be captured into a HIP graph, allocate nothing, and validate their
 * arguments before any HIP call.  Row strides are in elements and at least the row length; the elements of a
 * row are contiguous; pointers need the alignment of one element.
 */
#ifndef GLU_FP8_H
#define GLU_FP8_H

#include <stdint.h>

#include "glu_gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
enum {
    GLU_DTYPE_BF16 = 0,
    GLU_DTYPE_FP16 = 1,
    GLU_DTYPE_FP32 = 2,
    GLU_DTYPE_E4M3 = 3
};

/*
 * out [M, K] = T(h r w), with h = x, or with a residual h = T(x + residual),
 * which is stored to sum.  x, residual, weight [K], sum and out have type
 * `dtype` (BF16, FP16, FP32).  residual and sum are given together or both
 * NULL; sum may be exactly residual or x (same pointer and stride), any other overlap of an output is
 * refused.  rstd [M] (fp32, may be NULL) receives r, which the backward reads.
 * K >= 1 (GLU_ERR_BAD_SHAPE: the mean of an empty row is not defined); M == 0 is GLU_OK.
 * The mean of squares is fp32: a row whose sum of squares passes its range (an element above some 1.8e19) has r = 0.
 * eps negative or not finite, or an unknown dtype: GLU_ERR_BAD_ARGUMENT.
 */
glu_status glu_add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                            void* sum, int64_t lds, void* out, int64_t ldo, float* rstd, int64_t M, int64_t K,
                            float eps, int dtype, void* stream);

/* The same with y (not rounded to T) converted to e4m3: q [M, K] and scale,
 * fp32, group g of row m at scale[g * ld_scale + m] (ld_scale >= M). */
glu_status glu_add_rms_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                void* sum, int64_t lds, uint8_t* q, int64_t ldq, float* scale, int64_t ld_scale,
                                float* rstd, int64_t M, int64_t K, float eps, int dtype, void* stream);

/*
 * Gradients of the norm: with a = dy w and xhat = h r,
 *   dx = T(r (a - xhat mean_k(a xhat)) + dresidual)       (dresidual may be NULL)
 *   dweight = T(sum_m dy xhat)
 * dx is the gradient of x and of residual alike.  dx may be exactly dresidual.
 * M == 0 zero-fills dweight.  The rows are summed in an order fixed by (M, K): deterministic.
 * workspace: glu_add_rms_norm_backward_workspace(M, K) bytes, 16-byte aligned (NULL if 0).
 */
glu_status glu_add_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                                     const float* rstd, const void* dresidual, int64_t lddr, void* dx, int64_t lddx,
                                     void* dweight, int64_t M, int64_t K, int dtype, void* workspace,
                                     int64_t workspace_bytes, void* stream);
glu_status glu_add_rms_norm_backward_workspace(int64_t M, int64_t K, int64_t* bytes);

/* x [M, K] to e4m3 q and scale (group g of row m at scale[g * ld_scale + m]). */
glu_status glu_fp8_quantize(const void* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, int64_t ld_scale,
                            int64_t M, int64_t K, int dtype, void* stream);

/* w [N, K] to e4m3 q and one scale per 128 x 128 block, block (i, b) at scale[i * ld_scale + b]. */
glu_status glu_fp8_quantize_weight(const void* w, int64_t ldw, uint8_t* q, int64_t ldq, float* scale,
                                   int64_t ld_scale, int64_t N, int64_t K, int dtype, void* stream);

/* A block-scaled e4m3 operand: row r at data + r * ld; the scale of row (weights: row block) r and
 * column block b at scale[r * scale_row + b * scale_block] (weights: scale_block must be 1). */
typedef struct glu_fp8_matrix {
    const uint8_t* data;
    const float* scale;
    int64_t ld;
    int64_t scale_row;
    int64_t scale_block;
} glu_fp8_matrix;

/*
 * out [M, N] = x w^T, resp. silu(x gate^T) * (x up^T), in out_dtype: BF16,
 * FP16, FP32 (out_scale NULL) or E4M3, then out_scale receives the scales,
 * group g of row m at out_scale[g * ld_scale + m].  K == 0 writes the conversion of +0.  Fast layout: data
 * 16-byte aligned, K and the row strides multiples of 16, strides at most 2^23; any other layout takes a
 * slower kernel, or, with more than 16 rows of x, K at most 2^23 and glu_fp8_copy_workspace() bytes of workspace, is
 * copied to the fast one there first where that is expected to be faster; either way the sums are fp32.  workspace: glu_fp8_workspace() bytes, 16-byte
 * aligned (NULL if 0).
 */
glu_status glu_fp8_linear(const glu_fp8_matrix* x, const glu_fp8_matrix* w, void* out, int64_t ldo, float* out_scale,
                          int64_t ld_scale, int64_t M, int64_t N, int64_t K, int out_dtype, void* workspace,
                          int64_t workspace_bytes, void* stream);
glu_status glu_fp8_dual_glu(const glu_fp8_matrix* x, const glu_fp8_matrix* gate, const glu_fp8_matrix* up, void* out,
                            int64_t ldo, float* out_scale, int64_t ld_scale, int64_t M, int64_t N, int64_t K,
                            int out_dtype, void* workspace, int64_t workspace_bytes, void* stream);

/* Launch shape of a product, decided on the host alone. */
enum {
    GLU_FP8_KERNEL_NONE = 0,   /* M == 0 or N == 0 */
    GLU_FP8_KERNEL_ZERO = 1,   /* K == 0 */
    GLU_FP8_KERNEL_STREAM = 2, /* weights straight to the matrix cores: few rows of x */
    GLU_FP8_KERNEL_TILE = 3,   /* LDS tiles */
    GLU_FP8_KERNEL_ANY = 4     /* byte-aligned loads: any layout that is not fast */
};
typedef struct glu_fp8_plan {
    int kernel;                /* GLU_FP8_KERNEL_* */
    int tile;                  /* TILE: tile shape; STREAM: weight rows per workgroup */
    int width;                 /* TILE: threads per workgroup; STREAM: waves per workgroup */
    int splits;                /* parts of K summed by different workgroups */
    int launches;              /* 2: the parts are joined, or e4m3 converted, by a second kernel */
    int64_t workspace_bytes;
    int64_t columns;           /* TILE: > 0 (a multiple of 128): only the first columns by this shape,
                                  the others by launches shaped for as many columns; 0: all */
} glu_fp8_plan;

/* mats: 1 (linear) or 2 (dual GLU); `fast` states whether the layout is fast. */
glu_status glu_fp8_product_plan(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int fast,
                                glu_fp8_plan* plan);

/* Workspace bytes either product needs for these sizes, whatever its layout; glu_fp8_product_workspace with
 * plan NULL is what the fast layout needs, often less. */
glu_status glu_fp8_workspace(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int64_t* bytes);

/* Workspace bytes that serve a call on a layout that is not fast whether it copies its operands first or not; 0 where
 * none does (M <= 16, K > 2^23 or an empty product). */
glu_status glu_fp8_copy_workspace(int mats, int64_t M, int64_t N, int64_t K, int out_dtype, int64_t* bytes);

/*
 * Either product with the launch shape of `plan` (kernel, tile, width, splits, columns;
 * launches and workspace_bytes are ignored), for sweeps and tests: up NULL is the linear one.  A shape that the library
 * was not built with or that cannot serve the operands returns GLU_ERR_UNSUPPORTED, before any HIP call.  The
 * workspace is that of glu_fp8_product_workspace for the same plan (NULL: the one that the library chooses).
 */
glu_status glu_fp8_product_tuned(const glu_fp8_matrix* x, const glu_fp8_matrix* w, const glu_fp8_matrix* up,
                                 void* out, int64_t ldo, float* out_scale, int64_t ld_scale, int64_t M, int64_t N,
                                 int64_t K, int out_dtype, const glu_fp8_plan* plan, void* workspace,
                                 int64_t workspace_bytes, void* stream);
glu_status glu_fp8_product_workspace(int mats, int64_t M, int64_t N, int64_t K, int out_dtype,
                                     const glu_fp8_plan* plan, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GLU_FP8_H */
