// Launch interface of the e4m3 conversions (glu_quantize.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glu {

// q[m][k] = e4m3(x[m][k] / s[k / 128][m]) with s the rows' group scales, [groups][lds]
hipError_t quantize_rows_launch(int dtype, const void* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale,
                                int64_t lds, int M, int K, hipStream_t stream);
// one scale per block of 128 rows x 128 columns, s[n / 128][k / 128] at row stride lds
hipError_t quantize_blocks_launch(int dtype, const void* w, int64_t ldw, uint8_t* q, int64_t ldq, float* scale,
                                  int64_t lds, int N, int K, hipStream_t stream);

// e4m3 rows of any layout to rows of kp bytes, the K bytes and then zeros (kp and out: multiples of 16)
hipError_t copy_rows_launch(const uint8_t* x, int64_t ldx, uint8_t* out, int kp, int rows, int K, hipStream_t stream);

// The end of a product whose sums lie in fp32 planes [splits][mats][M][N]: the splits' sum in order, with two
// matrices silu(first) * second, then out (GLU_DTYPE_*; e4m3 with its scales).  splits == 0: the sums are +0.
struct FinishArgs {
    const float* part;
    void* out;
    float* scale;
    int64_t ldo, lds;
    int M, N, splits, mats;
};
hipError_t finish_launch(int out_dtype, const FinishArgs& a, hipStream_t stream);

}  // namespace glu
