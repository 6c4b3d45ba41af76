// The MoE layer on e4m3 weights (k_fp8_moe.cu).  Not part of the public interface.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8.cuh"

namespace mmoe {
namespace f8 {

constexpr int kFewTokens = 64;  // largest T of the two-launch path
constexpr int kRanks = 8;       // CTAs of a cluster, at most

struct MoePlan {
    int d, h, hs, E, k, gating, T;
    const float* w_router;
    const float* router_bias;  // null: none
    const uint8_t* gate_up;    // routed experts [E, 2h, d], scales [E, 2 ceil(h/128), ceil(d/128)]
    const float* s_gate_up;
    const uint8_t* down;       // [E, d, h], [E, ceil(d/128), ceil(h/128)]
    const float* s_down;
    const uint8_t* sh_gate_up; // shared expert [2hs, d], ...
    const float* sh_s_gate_up;
    const uint8_t* sh_down;
    const float* sh_s_down;
    const __nv_bfloat16* x;    // [T, d]
    void* y;                   // [T, d]
    bool y_bf16;
    int32_t* out_idx;          // optional outputs
    float* out_gate;
    int32_t* out_counts;
    int part_hidden, parts;    // the shared expert is taken in parts of that many hidden features
    // workspace
    int32_t* idx;              // [T, k]
    float* gate;               // [T, k]
    uint32_t* arrived;         // [T, kRanks] contributions of a token that are in, per rank of a cluster
    float* sx;                 // [T, ceil(d/128)]
    uint8_t* xq;               // [T, d]
    float* part;               // [T, k, d] expert outputs, then [parts, T, d] of the shared one
    Waits waits;
};

// Sets the parts of the shared expert, lays the workspace out from `base`, returns its size.
size_t carve_moe(MoePlan& p, unsigned char* base);
cudaError_t launch_moe_few(const MoePlan& p, cudaStream_t st);

}  // namespace f8
}  // namespace mmoe
