// Launch interface of dropout (glu_dropout.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glu {

struct DropoutArgs {
    const void* x;
    const void* res;             // or null
    void* out;
    const uint64_t* seed_at;     // or null: seed
    uint64_t seed, offset;
    int64_t ldx, ldr, ldo;
    int M, K;
    uint32_t drop;               // of 65536
    float scale;
};
hipError_t dropout_launch(int dtype, const DropoutArgs& a, hipStream_t stream);

}  // namespace glu
