// The norms after and before a block, fused with the block's gate and the
// residual update:
//
//   z  = y rsqrt(mean(y^2) + eps) w_post        (or y)
//   r' = scale r + gate z
//   x' = r' rsqrt(mean(r'^2) + eps) w_pre       -> BF16, and e4m3 codes with a scale per 128 features
//
// All of it in FP32: r' is rounded where it is stored, x' is computed from the
// sum before that rounding, and the codes from x' before its rounding to BF16.
//
// Bound by memory: a row is read once, held in registers through both norms
// and written once.  kG threads share a row (a warp where the registers allow
// it: no barrier), 8 features of a thread at a time (16-byte accesses), 16
// lanes side by side on one block of 128 features.
#include "fp8.cuh"
#include "norm.cuh"

namespace mmoe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(f8::bf16x2(v[0], v[1]), f8::bf16x2(v[2], v[3]), f8::bf16x2(v[4], v[5]),
                                              f8::bf16x2(v[6], v[7]));
}

// Sum over the kG threads of a row; `part` holds one word a warp and is used once.
template <int kG>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (kG > 32) {
        const int warp = threadIdx.x >> 5, first = warp / (kG / 32) * (kG / 32);
        if ((threadIdx.x & 31) == 0) part[warp] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kG / 32; ++i) v += part[first + i];
    }
    return v;
}

// kG threads a row, kV vectors of 8 features a thread.
template <int kG, int kV, class R, class Y>
__global__ void __launch_bounds__(kThreads) block_norm_kernel(const NormPlan p)
{
    __shared__ float part[2][kThreads / 32];
    const int g = threadIdx.x % kG;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / kG) + threadIdx.x / kG;
    const bool live = row < p.rows;
    f8::dep_launch();
    f8::dep_wait();
    float r[kV][8], z[kV][8];
    const bool block = p.y != nullptr;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int c = (i * kG + g) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = z[i][j] = 0.0f;
        if (live && c < p.d) {
            if (block) f8::load8(static_cast<const Y*>(p.y) + row * p.ldy + c, z[i]);
            f8::load8(static_cast<const R*>(p.r) + row * p.ldr + c, r[i]);
        }
    }
    float s = 1.0f;
    if (p.w_post) {  // the same for every thread of the grid
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(z[i][j], z[i][j], sum);
        s = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(row_sum<kG>(sum, part[0]), (float)p.d) + p.eps));
    }
    const float g0 = (p.gate && p.gate_col == 0 && live) ? p.gate[row * p.gate_row] : 1.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int c = (i * kG + g) * 8;
        if (!(live && c < p.d)) continue;
        float w[8];
        if (p.w_post) {
            f8::load8(p.w_post + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = z[i][j] * s * w[j];
        }
        if (p.gate && p.gate_col) {
            f8::load8(p.gate + row * p.gate_row + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] *= w[j];
        } else if (p.gate) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] *= g0;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[i][j] = block ? fmaf(p.scale, r[i][j], z[i][j]) : p.scale * r[i][j];
            sum = fmaf(r[i][j], r[i][j], sum);
        }
        if (p.r_out) store8(static_cast<R*>(p.r_out) + row * p.ldo + c, r[i]);
    }
    if (!p.w_pre) return;
    s = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(row_sum<kG>(sum, part[1]), (float)p.d) + p.eps));
    const int kb = (p.d + f8::kBlk - 1) / f8::kBlk;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int c = (i * kG + g) * 8;
        const bool in = live && c < p.d;
        if (in) {
            float w[8];
            f8::load8(p.w_pre + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * s * w[j];
            if (p.x) store8(reinterpret_cast<__nv_bfloat16*>(p.x) + row * p.d + c, r[i]);
        }
        if (p.xq) {
            const float sc = f8::scale_of(f8::half_warp_max(in ? f8::amax8(r[i]) : 0u));
            if (in) {
                *reinterpret_cast<uint2*>(p.xq + row * p.d + c) =
                    make_uint2(f8::e4m3x4(r[i], sc), f8::e4m3x4(r[i] + 4, sc));
                if ((g & 15) == 0) p.sx[row * kb + c / f8::kBlk] = sc;
            }
        }
    }
}

template <int kG, int kV>
cudaError_t launch(const NormPlan& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.rows + kThreads / kG - 1) / (kThreads / kG)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    using B = __nv_bfloat16;
    if (p.r_bf16)
        return p.y_bf16 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, kV, B, B>, p)
                        : cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, kV, B, float>, p);
    return p.y_bf16 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, kV, float, B>, p)
                    : cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, kV, float, float>, p);
}

}  // namespace

cudaError_t launch_block_norm(const NormPlan& p, cudaStream_t st) {
    const int v = (p.d + 7) / 8;
    if (v <= 32) return launch<32, 1>(p, st);
    if (v <= 64) return launch<32, 2>(p, st);
    if (v <= 128) return launch<32, 4>(p, st);
    if (v <= 256) return launch<64, 4>(p, st);
    if (v <= 512) return launch<128, 4>(p, st);
    return launch<256, 4>(p, st);
}

}  // namespace mmoe
