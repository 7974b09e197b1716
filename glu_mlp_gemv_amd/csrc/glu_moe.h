// Launch interface of the expert-layer kernels (glu_moe.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glu {

constexpr int kMoeRows = 64;  // rows of x per set of launches: an expert's rows are a 64-bit mask

struct ExpertMatrix {
    const uint8_t* data;
    const float* scale;
    int64_t stack, ld, scale_stack, scale_ld;  // in elements
};

// An expert some row chose: its rows are slots first .. first + count - 1.
struct Active { int expert, first, count; };

struct MoeArgs {
    const void* x;         // [M][K]
    const void* logits;    // [M][E]
    ExpertMatrix w[3];     // gate, up [N][K]; down [K][N]
    void* out;             // [M][K]
    int64_t ldx, ldl, ldo;
    int M, K, N, E, top;   // M <= kMoeRows
    bool normalize;
    // workspace
    int* actives;          // how many experts are active
    Active* active;        // [E], ascending
    int* row;              // [M top] row of each slot
    float* weight;         // [M top] its weight
    uint16_t* act;         // [M top][2][ld_act] activations, two numbers each
    float* factor;         // [M top][ld_factor] what 16 columns of them are multiplied with, where they are fp16
    float* part;           // [splits][M][K] sums of the second product's parts, where splits > 1
    int64_t ld_act, ld_factor;
};

// How the second product is cut: `splits` sets of workgroups take the active experts in turn, and within a workgroup
// `parts` waves share one expert's columns; rows: weight rows per workgroup, 4 or 16.
struct MoePlan { int splits, parts, rows; };
MoePlan moe_plan(int M, int K, int N, int E, int top, bool e4m3);
hipError_t moe_launch(int dtype, int logits_dtype, bool e4m3, const MoeArgs& a, const MoePlan& p, hipStream_t stream);

struct LogitsArgs {
    const void* x;       // [M][K]
    const void* router;  // [E][K]
    float* logits;       // [M][E]
    int64_t ldx, ldr;
    int M, K, E;
};
hipError_t moe_logits_launch(int dtype, const LogitsArgs& a, hipStream_t stream);

}  // namespace glu
