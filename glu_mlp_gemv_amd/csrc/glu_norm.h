// Launch interface of the RMS-norm kernels (glu_norm.hip).  Types are GLU_DTYPE_* of include/glu_fp8.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glu {

struct NormArgs {
    const void* x;        // [M][K], row stride ldx
    const void* res;      // residual, or null
    const void* weight;   // [K]
    void* sum;            // rounded x + residual (null without a residual)
    void* out;            // [M][K] in x's type, or e4m3
    float* scale;         // e4m3: [groups][lds]
    float* rstd;          // [M] or null
    int64_t ldx, ldr, ldsum, ldo, lds;
    int M, K;
    float eps;
};
hipError_t norm_launch(int dtype, bool e4m3, const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
    const void* dy;       // [M][K]
    const void* h;        // [M][K]: the rounded sum that was normalised
    const void* dres;     // gradient arriving on the residual stream, or null
    const void* weight;   // [K]
    const float* rstd;    // [M]
    void* dx;             // [M][K]
    void* dw;             // [K]
    float* part;          // [parts][K]: norm_grad_part_floats
    int64_t lddy, ldh, lddr, lddx;
    int M, K;
};
int64_t norm_grad_part_floats(int dtype, int M, int K);
hipError_t norm_grad_launch(int dtype, const NormGradArgs& a, hipStream_t stream);

}  // namespace glu
