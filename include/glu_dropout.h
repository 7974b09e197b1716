/*
 * glu_dropout.h -- dropout with a mask that is computed and never stored (gfx950).
 *
 *   out[m, k] = T(residual[m, k] + (kept(m, k) ? x[m, k] * c : 0)),   c = 65536 / (65536 - drop) in fp32
 *
 * kept: draw(m, k) >= drop, drop = round(65536 p) of the caller, a whole number of 0 .. 65536.  The draws are 16 bits of
 * Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with key (seed low, seed
 * high) and counter (k / 8, m, offset low, offset high): its four words hold the draws of columns 8 (k / 8) .. + 7, the low
 * half of a word first.  So p is applied in steps of 2^-16, with c the reciprocal of what is kept, and the mask depends
 * on seed, offset and an element's place alone, not on types, strides or launches: the same call on a gradient is the
 * backward.  A dropped x does not show, NaN or infinite as it may be.
 *
 * Ownership, execution, determinism and errors are those of glu_gemv.h.  Row strides are in elements and at least the row length;
 * the elements of a row are contiguous; pointers need the alignment of one element.
 */
#ifndef GLU_DROPOUT_H
#define GLU_DROPOUT_H

#include <stdint.h>

#include "glu_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * x, residual (may be NULL: zeros) and out [M, K] of dtype (BF16, FP16, FP32).  out may be exactly x or residual.
 * seed_device (may be NULL): the seed is the 64-bit number there, read when the kernel runs (8-byte aligned), so that a
 * captured graph draws anew on each replay; else `seed`.  drop outside 0 .. 65536 or an unknown dtype:
 * GLU_ERR_BAD_ARGUMENT.
 */
glu_status glu_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* out, int64_t ldo, int64_t M,
                       int64_t K, int64_t drop, uint64_t seed, const uint64_t* seed_device, uint64_t offset, int dtype,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GLU_DROPOUT_H */
