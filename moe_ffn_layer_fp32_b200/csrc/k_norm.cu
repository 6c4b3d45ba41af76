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
// Bound by memory: a row is read once, held by its threads through both norms
// and written once.  kG threads take a row, 8 features each (16-byte accesses,
// 16 lanes side by side on one block of 128 features), and go on to other rows:
// the weights and a gate per feature are read once a thread, and the next row
// is on its way while this one is reduced.  Rows of 2048 features stay in
// registers and run at 90 % of the memory's rate (32768 rows with codes: 126
// us).  Above that a thread has 64 registers, 92 to 136 bytes of which spill,
// and the barriers of 16 or 32 warps weigh more: 8192 rows of 4096 take 98 us
// for 56 us of traffic, of 8192 237 us for 113.  (Rows of up to 256, a warp
// each, spill up to 76 bytes where r is FP32.)
#include <algorithm>

#include "fp8.cuh"
#include "norm.cuh"

namespace mmoe {
namespace {

// 8 features as they lie in memory.
template <class T>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const { f8::unpack8(u, v); }
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(f8::bf16x2(v[0], v[1]), f8::bf16x2(v[2], v[3]), f8::bf16x2(v[4], v[5]),
                                              f8::bf16x2(v[6], v[7]));
}

// 1 / sqrt(mean(v^2) + eps) of the row that kG threads hold.  `part` holds one word a warp; the next row uses another
// one, so that one barrier is enough.  Every thread does the last steps, so they are a product with 1 / d (inv_d) and
// rsqrtf (off by 2 ulp at most): with IEEE divisions and root the kernel issued 430 instructions a warp and row, and
// was bound by them.  Of 32768 x 2048 codes 66 differ
// from those of a 64-bit norm, 78 with torch's FP32 operations (IEEE root and quotient).
template <int kG>
__device__ __forceinline__ float inv_rms(const float (&v)[8], float* part, float inv_d, float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (kG > 32) {
        constexpr int kW = kG / 32;
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        if constexpr (kW % 4 == 0) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kW; i += 4) {
                const float4 p = *reinterpret_cast<const float4*>(part + i);
                sum += (p.x + p.y) + (p.z + p.w);
            }
        } else {
            sum = part[0] + part[1];
        }
    }
    return rsqrtf(fmaf(sum, inv_d, eps));
}

// kG threads a row; a CTA has one row, or eight of a warp each.
template <int kG>
constexpr int threads() {
    return kG == 32 ? 256 : kG;
}

// CTAs an SM: 768 threads of 80 registers, or 1024 of 64 where a row takes more.
template <int kG>
constexpr int resident() {
    return (kG <= 256 ? 768 : 1024) / threads<kG>();
}

template <int kG, class R, class Y>
__global__ void __launch_bounds__(threads<kG>(), resident<kG>()) block_norm_kernel(const NormPlan p)
{
    constexpr int kRows = threads<kG>() / kG;
    __shared__ alignas(16) float part[2][2][kG / 32];
    const int g = threadIdx.x % kG, c = g * 8;
    const bool mine = c < p.d;
    f8::dep_launch();
    f8::dep_wait();
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kG;
    const bool block = p.y != nullptr, per_row = p.gate && p.gate_col == 0, whole = p.gate && p.gate_col && p.gate_row;
    Raw<R> rr = {};
    Raw<Y> yy = {};
    Raw<float> post = {}, pre = {}, gate = {};
    float g0 = 1.0f;
    const auto fetch = [&](int64_t at) {
        if (mine) {
            rr.load(static_cast<const R*>(p.r) + at * p.ldr + c);
            if (block) yy.load(static_cast<const Y*>(p.y) + at * p.ldy + c);
            if (whole) gate.load(p.gate + at * p.gate_row + c);
        }
        if (per_row) g0 = p.gate[at * p.gate_row];
    };
    if (row < p.rows) fetch(row);
    if (mine) {
        if (p.gate && p.gate_col && !whole) gate.load(p.gate + c);
        if (p.w_post) post.load(p.w_post + c);
        if (p.w_pre) pre.load(p.w_pre + c);
    }
    const int kb = (p.d + f8::kBlk - 1) / f8::kBlk;
    const float inv_d = __fdiv_rn(1.0f, (float)p.d);
    for (int turn = 0; row < p.rows; row += step, turn ^= 1) {  // the same row for all kG threads
        float r[8], z[8], w[8];
        rr.get(r);
        yy.get(z);
        const float gr = g0;
        float gv[8];
        gate.get(gv);
        if (row + step < p.rows) fetch(row + step);
        if (p.w_post) {
            const float s = inv_rms<kG>(z, part[turn][0], inv_d, p.eps);
            post.get(w);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = z[j] * s * w[j];
        }
        if (per_row) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] *= gr;
        } else if (p.gate) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] *= gv[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = block ? fmaf(p.scale, r[j], z[j]) : p.scale * r[j];
        if (p.r_out && mine) store8(static_cast<R*>(p.r_out) + row * p.ldo + c, r);
        if (!p.w_pre) continue;
        const float s = inv_rms<kG>(r, part[turn][1], inv_d, p.eps);
        pre.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = r[j] * s * w[j];
        if (p.x && mine) store8(reinterpret_cast<__nv_bfloat16*>(p.x) + row * p.d + c, r);
        if (p.xq) {
            const float sc = f8::scale_of(f8::half_warp_max(mine ? f8::amax8(r) : 0u));
            if (mine) {
                *reinterpret_cast<uint2*>(p.xq + row * p.d + c) = f8::Coder(sc)(r);
                if ((g & 15) == 0) p.sx[row * kb + c / f8::kBlk] = sc;
            }
        }
    }
}

template <int kG>
cudaError_t launch(const NormPlan& p, cudaStream_t st) {
    constexpr int kT = threads<kG>(), kRows = kT / kG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((p.rows + kRows - 1) / kRows, (int64_t)f8::sm_count() * resident<kG>()));
    cfg.blockDim = dim3(kT);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    using B = __nv_bfloat16;
    if (p.r_bf16)
        return p.y_bf16 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, B, B>, p)
                        : cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, B, float>, p);
    return p.y_bf16 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, float, B>, p)
                    : cudaLaunchKernelEx(&cfg, block_norm_kernel<kG, float, float>, p);
}

}  // namespace

cudaError_t launch_block_norm(const NormPlan& p, cudaStream_t st) {
    const int v = (p.d + 7) / 8;
    if (v <= 32) return launch<32>(p, st);
    if (v <= 64) return launch<64>(p, st);
    if (v <= 128) return launch<128>(p, st);
    if (v <= 256) return launch<256>(p, st);
    if (v <= 512) return launch<512>(p, st);
    return launch<1024>(p, st);
}

}  // namespace mmoe
