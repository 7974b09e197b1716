// Launch interface of the block-scaled e4m3 products (glu_fp8_stream.hip, glu_fp8_tile.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glu {

// One or two products of the same rows: sum over K-blocks b of sx[m, b] sw[n / 128, b] sum_{k in b} x[m, k]
// w[n, k].
struct Fp8Args {
    const uint8_t* x;       // [M][K] e4m3, row stride ldx
    const float* sx;        // scale of row m, block b at m * sxm + b * sxg
    const uint8_t* w[2];    // [N][K] e4m3, row strides ldw; two: out = silu(first) * second
    const float* sw[2];     // scale of rows 128 i .., block b at i * ldsw + b
    void* out;              // [M][N] of out_dtype at row stride ldo
    float* scale;           // e4m3 out: scale of group i, row m at i * lds + m
    float* part;            // partial sums [splits][mats][M][N], when the plan asks for them
    int64_t ldx, sxm, sxg, ldw[2], ldsw[2], ldo, lds;
    int M, N, K;
    int out_dtype;          // GLU_DTYPE_*; kPartial: raw sums into part
};
constexpr int kPartial = -1;

// Weights straight from memory to the matrix cores; a workgroup of `waves` waves splits the K-blocks of
// `rows` weight rows (4, for x of up to 4 rows, or 16) among them.
struct StreamConfig {
    int rows, waves, splits;
    bool any;  // K or an address not a multiple of 16: byte-aligned loads (rows 16)
};
hipError_t fp8_stream_launch(int mats, const StreamConfig& c, const Fp8Args& a, hipStream_t stream);
bool fp8_stream_supported(const StreamConfig& c, int M);

// LDS-tiled product; shape: an index into kTileShapes
struct TileShape {
    int bm;       // rows of x per workgroup
    int br;       // weight rows per workgroup (bn = br / mats of each matrix)
    int threads;
    int stages;
};
constexpr int kTileShapeCount = 5;
extern const TileShape kTileShapes[kTileShapeCount];
struct TileConfig {
    int shape, splits;
    bool wide;  // fp32 sums on the bf16 unit, else the 8-bit unit's (glu_fp8_mfma.h); e4m3 out: always
};
// whether the kernel can finish e4m3 by itself: a workgroup holds whole groups of 128 columns
bool fp8_tile_owns_groups(int mats, int shape);
hipError_t fp8_tile_launch(int mats, const TileConfig& c, const Fp8Args& a, hipStream_t stream);

}  // namespace glu
