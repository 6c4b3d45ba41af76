// e4m3 block-scaled operators: declarations and device helpers shared by their
// kernels (k_fp8_quant.cu, k_fp8_gemm.cu, k_fp8_moe.cu, k_norm.cu) and their C
// entries (mmoe_ops.cu).  Not part of the public interface.
//
// A quantised block holds codes q = e4m3(v / s), s = max|v| / 448 (both IEEE
// FP32 divisions, the code rounded to nearest even), all 0 for a block of
// zeros.  A block is 128 consecutive features of one activation row, or 128 x
// 128 values of a weight matrix.  NaN and infinities: the maximum is taken on
// the bit patterns, so that a NaN in the block makes s NaN and an infinity
// makes s infinite; either way every product with the block is NaN, as it is
// where the values themselves are multiplied.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mmoe.h"
#include "sm100_async.cuh"
#include "sm100_tc.cuh"

namespace mmoe {
namespace f8 {

constexpr int kBlk = 128;             // features (and weight rows) per scale
constexpr float kTop = 448.0f;        // largest finite e4m3 value
constexpr long long kWaitClk = 4000000000ll;  // about 2 s of SM clock: the limit of every device-side wait

inline int64_t blocks_of(int64_t n) { return (n + kBlk - 1) / kBlk; }

// --- device helpers ---------------------------------------------------------

// Programmatic dependent launch: the kernel may start before its predecessor in the stream has ended;
// everything it reads or writes in global memory comes after dep_wait (which returns when the
// predecessor has completed and its writes are visible).
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ float scale_of(uint32_t amax_bits) { return __fdiv_rn(__uint_as_float(amax_bits), kTop); }

__device__ __forceinline__ float coded(float v, float s) { return s > 0.0f ? __fdiv_rn(v, s) : 0.0f; }

// Two values to two e4m3 codes, `lo` in the low byte (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(const float* v, float s) {
    return e4m3x2(coded(v[0], s), coded(v[1], s)) | (e4m3x2(coded(v[2], s), coded(v[3], s)) << 16);
}

// Ordinary loads: the read-only path may be hoisted above dep_wait.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
}

// Maximum over the 16 lanes of a half warp.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// D (TMEM) = A * B (+ D when `accumulate`), e4m3 operands (32 of K), FP32 accumulator, M = 128,
// issued by one thread.  The descriptor's type fields of e4m3 are 0.
__host__ __device__ constexpr uint32_t idesc_e4m3(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Makes this thread's shared-memory stores visible to the tensor cores and the copy engine.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of the same shared variable in CTA `rank` of the cluster, and a load from there.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(async::su32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A bounded mbarrier wait.  Gives up after kWaitClk, or once another thread of the CTA has given up;
// then it sets the CTA's abort word and the host-visible flag and returns false.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort_word, int* err, int site) {
    if (async::mbar_try_wait(bar, parity)) return true;
    const long long t0 = async::clk();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (async::mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int*>(abort_word)) return false;
        if (async::clk() - t0 > kWaitClk) {
            atomicExch(abort_word, 1);
            *reinterpret_cast<volatile int*>(err) = site;
            __threadfence_system();
            return false;
        }
    }
}

// Signals an mbarrier of a peer CTA (this thread's earlier stores, and what it has seen of others', come before),
// and the bounded wait for such signals.
__device__ __forceinline__ void peer_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, int* abort_word, int* err, int site) {
    const long long t0 = async::clk();
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(async::su32(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        if (*reinterpret_cast<volatile int*>(abort_word)) return false;
        if (async::clk() - t0 > kWaitClk) {
            atomicExch(abort_word, 1);
            *reinterpret_cast<volatile int*>(err) = site;
            __threadfence_system();
            return false;
        }
    }
}

// The same by a whole warp, which decides as one.  Every lane polls: against one lane that polls and a shuffle that
// tells the others, a block of 128 of the promotion loops took 639 instead of 1042 clocks.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort_word, int* err, int site) {
    if (__all_sync(0xffffffffu, async::mbar_try_wait(bar, parity))) return true;
    const long long t0 = async::clk();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, async::mbar_try_wait(bar, parity))) return true;
        const bool late = async::clk() - t0 > kWaitClk;
        if (late) {
            atomicExch(abort_word, 1);
            *reinterpret_cast<volatile int*>(err) = site;
            __threadfence_system();
        }
        if (__any_sync(0xffffffffu, late || *reinterpret_cast<volatile int*>(abort_word))) return false;
    }
}

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// The wait used while draining: ignores the abort word.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
    const long long t0 = async::clk();
    while (!async::mbar_try_wait(bar, parity))
        if (async::clk() - t0 > kWaitClk) return;
}

// --- launchers ----------------------------------------------------------------

// cuTensorMap of a row-major byte matrix [rows, cols] (row stride in bytes), boxes of 128 bytes x
// box_rows in the 128-byte swizzle layout; bytes outside the matrix read as 0.
cudaError_t byte_map(void* map, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, int box_rows);
int sm_count();

cudaError_t launch_quantize_rows(const void* x, bool bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* q, float* s,
                                 cudaStream_t st);
cudaError_t launch_quantize_blocks(const void* w, bool bf16, int64_t batch, int64_t N, int64_t K, uint8_t* q, float* s,
                                   cudaStream_t st);

// y[M, N] = a * w^T.  a: codes [M, K] with scales sa, or BF16 values x [M, K] (then quantised on the way
// in; M <= kSmallRows only).  groups = 0: one weight matrix; else rows offsets[g] .. offsets[g+1] - 1 use
// weight matrix g.
constexpr int kSmallRows = 64;
constexpr int kMaxGroups = 1024;
struct Product {
    const uint8_t* a;
    const float* sa;
    const __nv_bfloat16* x;
    int64_t ldx;
    const uint8_t* w;
    const float* sw;
    int64_t M;
    int N, K;
    int groups;
    const int32_t* offsets;
    void* y;
    bool y_bf16;
    int64_t ldy;
    int* err;
};
cudaError_t launch_product(const Product& p, cudaStream_t st);
cudaError_t launch_product_small(const Product& p, cudaStream_t st);

}  // namespace f8
}  // namespace mmoe
