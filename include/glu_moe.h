/*
 * glu_moe.h -- a mixture-of-experts GLU layer for a few tokens (gfx950).
 *
 *   experts of row m: the `top` largest of logits[m], of equal ones the lowest
 *   p = softmax of logits[m] over them (normalize), or over all experts
 *   out[m] = T( sum_e p_e down_e T(silu(gate_e x[m]) (up_e x[m])) )
 *
 * An expert's gate and up are read once per 64 rows of x in which some row needs it, and down once per 32 rows of its own (16
 * of FP16 or E4M3 weights; 2 in calls of up to 4 rows), again from the caches mostly.  That is what bounds the layer: it is
 * meant for the tokens of a decode step, and correct for any number of rows.  The products' sums, the activation, the softmax and the
 * sum over experts are fp32; as the operand of the second product the activation is two 16-bit numbers, its rounding and the
 * rounding of what that left, so that 2^-17 of it is lost at most (fp16 weights: 2^-23, and 2^-39 of the largest of 16
 * columns).  It has fp32's range for every T.
 *
 * A logit of -inf is an expert masked away: it is never chosen, and a row without any other has fewer experts, or none
 * and out = 0.  A NaN logit ranks above all others and makes its row NaN.  Experts that a row did not choose do not
 * touch it, whatever they hold.
 *
 * T, the type of x and out, is BF16 or FP16 (GLU_DTYPE_*, glu_fp8.h).  The weights are of T or block-scaled E4M3 (one
 * fp32 scale per 128 x 128 block of an expert's matrix), whose products with x are exact in fp32 sums.
 *
 * Ownership, execution, determinism and errors are those of glu_gemv.h: all arrays are device memory of the caller,
 * calls are asynchronous on `stream`, may be captured into a HIP graph, allocate nothing, and validate their
 * arguments before any HIP call.  Row strides are in elements and at least the row length; the elements of a row are
 * contiguous; pointers need the alignment of one element.
 */
#ifndef GLU_MOE_H
#define GLU_MOE_H

#include <stdint.h>

#include "glu_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GLU_MOE_MAX_EXPERTS 1024
#define GLU_MOE_MAX_TOP 32

/* E matrices: element (e, i, j) at data + e * stack + i * ld + j; for E4M3 the scale of block (i / 128, j / 128) at
 * scale[e * scale_stack + (i / 128) * scale_ld + j / 128], else scale is NULL.  Rows and matrices do not overlap. */
typedef struct glu_expert_matrix {
    const void* data;
    const float* scale;
    int64_t stack, ld, scale_stack, scale_ld;
} glu_expert_matrix;

typedef struct glu_moe_sizes {
    int64_t M;    /* rows of x */
    int64_t K;    /* columns of x and out */
    int64_t N;    /* an expert's inner width */
    int64_t E;    /* experts, 1 to GLU_MOE_MAX_EXPERTS */
    int64_t top;  /* experts per row, 1 to min(E, GLU_MOE_MAX_TOP) */
} glu_moe_sizes;

/*
 * x and out [M, K], logits [M, E] of logits_dtype (FP32 or dtype), gate and up [E, N, K], down [E, K, N] of weight_dtype
 * (dtype or E4M3).  An output that overlaps an input is refused.  M == 0 or K == 0: GLU_OK, nothing launched; N == 0
 * zeros out.
 * workspace: glu_moe_workspace() bytes, 16-byte aligned (NULL if 0).
 */
glu_status glu_moe_glu(const void* x, int64_t ldx, const void* logits, int64_t ldl, int logits_dtype,
                       const glu_expert_matrix* gate, const glu_expert_matrix* up, const glu_expert_matrix* down,
                       void* out, int64_t ldo, const glu_moe_sizes* sizes, int normalize, int dtype, int weight_dtype,
                       void* workspace, int64_t workspace_bytes, void* stream);
glu_status glu_moe_workspace(const glu_moe_sizes* sizes, int64_t* bytes);

/*
 * logits[m] = x[m] router^T, fp32 sums that are not rounded: what glu_moe_glu ranks.  Rounded to 16 bits, logits of neighbouring
 * experts become equal or change places, and the lowest of equal ones is taken.
 * x [M, K] and router [E, K] of dtype (BF16 or FP16), logits [M, E] dense.  M == 0: GLU_OK, nothing launched; K == 0: zeros.
 */
glu_status glu_moe_logits(const void* x, int64_t ldx, const void* router, int64_t ldr, float* logits, int64_t M, int64_t K,
                          int64_t E, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GLU_MOE_H */
