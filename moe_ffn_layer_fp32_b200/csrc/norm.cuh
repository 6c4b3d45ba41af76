// The norms after and before a block (k_norm.cu).  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mmoe {

constexpr int kNormMaxDim = 8192;

struct NormPlan {
    int64_t rows;
    int d;
    const void* r;         // residual stream, row stride ldr
    int64_t ldr;
    bool r_bf16;
    const void* y;         // block output (null: none), row stride ldy
    int64_t ldy;
    bool y_bf16;
    const float* w_post;   // null: y is not normalised
    const float* gate;     // null: 1
    int64_t gate_row;      // elements between rows and columns of the gate (0: the same for all)
    int gate_col;
    float scale;           // of the residual stream
    float eps;
    void* r_out;           // null: not wanted; r's type
    int64_t ldo;
    const float* w_pre;    // null: no norm before the next block
    uint16_t* x;           // [rows, d] BF16 (null: not wanted)
    uint8_t* xq;           // [rows, d] e4m3 codes and their scales (null: not wanted)
    float* sx;
};

cudaError_t launch_block_norm(const NormPlan& p, cudaStream_t st);

}  // namespace mmoe
