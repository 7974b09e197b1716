// C ABI of dropout (include/glu_dropout.h): argument validation, before any HIP call, and launch.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/glu_dropout.h"
#include "glu_check.h"
#include "glu_dropout.h"
#include "glu_status.h"

extern "C" glu_status glu_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* out, int64_t ldo,
                                  int64_t M, int64_t K, int64_t drop, uint64_t seed, const uint64_t* seed_device,
                                  uint64_t offset, int dtype, void* stream)
{
    if (dtype != GLU_DTYPE_BF16 && dtype != GLU_DTYPE_FP16 && dtype != GLU_DTYPE_FP32) return GLU_ERR_BAD_ARGUMENT;
    if (drop < 0 || drop > 65536) return GLU_ERR_BAD_ARGUMENT;
    if (glu::bad_dim(M) || glu::bad_dim(K)) return GLU_ERR_BAD_SHAPE;
    if (M == 0 || K == 0) return GLU_OK;
    const int es = dtype == GLU_DTYPE_FP32 ? 4 : 2;
    const glu::Array arrays[] = {
        {x, M, K, ldx, es, false},
        {residual, residual ? M : 0, K, ldr, es, false},
        {out, M, K, ldo, es, true},
        {seed_device, seed_device ? 1 : 0, 1, 1, 8, false},
    };
    const glu_status st = glu::check_arrays(arrays, 4, 1u << 2, 3u);
    if (st != GLU_OK) return st;
    const float scale = drop == 65536 ? 0.0f : 65536.0f / (float)(65536 - drop);  // nothing is kept of 65536
    const glu::DropoutArgs a{x,   residual, out, seed_device, seed,   offset,         ldx,
                             ldr, ldo,      (int)M, (int)K,   (uint32_t)drop, scale};
    const hipError_t e = glu::dropout_launch(dtype, a, (hipStream_t)stream);
    return e == hipSuccess ? GLU_OK : glu::fail_launch(e);
}
