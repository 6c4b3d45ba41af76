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

#include <atomic>

#include "mmoe.h"
#include "sm100_async.cuh"
#include "sm100_tc.cuh"

namespace mmoe {
namespace f8 {

constexpr int kBlk = 128;             // features (and weight rows) per scale
constexpr float kTop = 448.0f;        // largest finite e4m3 value
constexpr long long kWaitClk = 4000000000ll;  // about 2 s of SM clock: how long a device-side wait lasts before it gives up
constexpr long long kDrainClk = 200000000ll;  // about 0.1 s: then a kernel that gives up no longer waits for its copies or MMAs

// How long the waits of a launch last, and where one that gives up says so.
struct Waits {
    int* err;         // host-visible word, set to the wait's site
    long long limit;  // SM clocks
    int stall;        // failure-detection tests: 1: in the first CTA the MMA warps' barriers expect an arrival more than there
                      // is, 2: in the first cluster's last CTA those of the promotion warps
    // What CTA `cta` adds to the arrivals that the barriers of 1: the MMA, 2: the promotion warps expect.
    __device__ __forceinline__ int missing(int who, unsigned cta) const { return stall == who && blockIdx.x == cta; }
};

constexpr int64_t blocks_of(int64_t n) { return (n + kBlk - 1) / kBlk; }

// --- device helpers ---------------------------------------------------------

// Programmatic dependent launch: the kernel may start before its predecessor in the stream has ended;
// everything it reads or writes in global memory comes after dep_wait (which returns when the
// predecessor has completed and its writes are visible).
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// max|v| / 448, the IEEE quotient.  Division by a constant after Brisebarre, Muller and Raina ("Accelerating correctly
// rounded floating-point division when the divisor is known in advance"): the product with the rounded reciprocal and
// one correction by its remainder.  Checked over every significand (tests/test_fp8_quotients.py); below 2^-100, for infinities and NaN it divides.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits), q = a * (1.0f / kTop);
    const float s = fmaf(fmaf(-kTop, q, a), 1.0f / kTop, q);
    return a >= 0x1p-100f && a <= 3.0e38f ? s : __fdiv_rn(a, kTop);
}

__device__ __forceinline__ float coded(float v, float s) { return s > 0.0f ? __fdiv_rn(v, s) : 0.0f; }

// Two values to two e4m3 codes, `lo` in the low byte (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | (e4m3x2(c, d) << 16); }

// A call: inlined, divisions would be most of a kernel's code, and a kernel of a few microseconds waits for its code.
static __device__ __noinline__ uint32_t divided4(float a, float b, float c, float d, float s) {
    return e4m3x4(coded(a, s), coded(b, s), coded(c, s), coded(d, s));
}

// The codes of a block's values, e4m3(v / s), from one reciprocal: y = RN(1 / s), the quotient v y and one correction
// by its remainder, RN(q + (v - q s) y).  Before that last rounding it is within 2^-46 of v / s, relative, so that it
// is the IEEE quotient unless v / s lies 2^-22 of an ulp or less from the middle of two FP32 numbers.  That matters
// for the code only beside a rounding border of e4m3, a number of four significant bits; with significands V, S <
// 2^24 the middle beside it, B 2^20 + 1 with B below 2^5, can be as near to V / S only where S is within 4 of a
// multiple of 2^20.  For those S (16 either way) every V is checked on the CPU, as is for every S the V beside each
// border (tests/test_fp8_quotients.py): always the IEEE quotient.  A code that is not 0 needs v >= s 2^-11, and the
// remainder is a multiple of v 2^-47, which must not underflow; blocks outside that range, of zeros, with NaN or
// infinities are divided.  (Bounding the quotient from both sides by two products costs less, but BF16 values lie on
// a border too often: one in 200.)  All of it is done for -v / s, whose codes have the other sign: there the
// correction adds zeros of one sign, while for v / s it made +0 of the code of -0.  Quantising 32768 x 2048 BF16
// values took 106 us with a division each, and takes 39 us.
struct Coder {
    float s, y;
    bool fast;
    __device__ __forceinline__ explicit Coder(float scale) : Coder(scale, inverse(scale)) {}
    static __device__ __forceinline__ float inverse(float scale) { return __fdiv_rn(1.0f, scale); }
    __device__ __forceinline__ Coder(float scale, float inv) : s(scale), y(inv) {
        fast = scale >= 0x1p-80f && scale <= 0x1p100f;
    }
    // the codes of -a and -b
    __device__ __forceinline__ uint32_t pair(float a, float b) const {
        const float2 v = make_float2(a, b), yy = make_float2(-y, -y), ss = make_float2(s, s);
        float2 q = __fmul2_rn(v, yy);
        q = __ffma2_rn(__ffma2_rn(ss, q, v), yy, q);
        return e4m3x2(q.x, q.y);
    }
    __device__ __forceinline__ uint2 operator()(const float (&v)[8]) const {
        if (!fast) return make_uint2(divided4(v[0], v[1], v[2], v[3], s), divided4(v[4], v[5], v[6], v[7], s));
        const uint32_t lo = pair(v[0], v[1]) | pair(v[2], v[3]) << 16, hi = pair(v[4], v[5]) | pair(v[6], v[7]) << 16;
        return make_uint2(lo ^ 0x80808080u, hi ^ 0x80808080u);
    }
};

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

// Largest magnitude of 8 BF16 values, as FP32 bits.
__device__ __forceinline__ uint32_t amax_bf16(const uint4& u) {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & k, u.y & k), __vmaxu2(u.z & k, u.w & k));
    return max(m << 16, m & 0xffff0000u);
}

// Scales and codes of the first n of U blocks, 8 lanes a block with 16 values each in two halves: peak(u) gives a lane's
// largest magnitude, get(u, half, values) the values.  All blocks side by side, for one after the other each waits for its
// own maximum, divisions and conversions; lane u of the 8 does block u's divisions.
template <int U, class Peak, class Get>
__device__ __forceinline__ void encode(int n, const Peak& peak, const Get& get, float (&s)[U], uint2 (&q)[U][2]) {
    uint32_t m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) m[u] = u < n ? peak(u) : 0u;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < n) m[u] = max(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
    uint32_t mine = m[0];
#pragma unroll
    for (int u = 1; u < U; ++u)
        if ((threadIdx.x & (U - 1)) == u) mine = m[u];
    const float scale = scale_of(mine), inv = Coder::inverse(scale);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u < n) {
            s[u] = __shfl_sync(0xffffffffu, scale, u, 8);
            const Coder code(s[u], __shfl_sync(0xffffffffu, inv, u, 8));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
                get(u, h, v);
                q[u][h] = code(v);
            }
        }
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

// The same for a pair of CTAs (M = 256, 128 rows and half of N in each one's shared memory, at the same addresses),
// issued in the pair's CTA 0.
__host__ __device__ constexpr uint32_t idesc_e4m3_pair(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on both CTAs' `bar` when the pair operations issued before have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            async::su32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// A tile into this CTA's shared memory, counted on a barrier (a cluster address) of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(async::su32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const void* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            async::su32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(async::su32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const void* map, int x, int y, int z, int u, int v, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
        "[%7];" ::"r"(async::su32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(async::su32(bar))
        : "memory");
}
// A tile from shared memory to global memory (one group of the issuing thread's).
__device__ __forceinline__ void tma_store_2d(const void* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(async::su32(src))
                 : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(async::su32(dst_smem)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t tmem, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
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

__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// A CTA's waits, in its shared memory (as kernel arguments in each wait they took registers: the product of 512 x 2048 x
// 2048 11.6 us instead of 10.7).
struct Stop {
    long long limit;
    int set;  // a wait has run out
    __device__ __forceinline__ void init(const Waits& w) {
        limit = w.limit;
        set = 0;
    }
    __device__ __forceinline__ bool is_set() const { return *reinterpret_cast<const volatile int*>(&set); }
    __device__ __forceinline__ bool late(long long t0) const {
        return async::clk() - t0 > *reinterpret_cast<const volatile long long*>(&limit);
    }
    // Tells the CTA's other threads, and the host.
    __device__ __forceinline__ void give_up(int* err, int site) {
        atomicExch(&set, 1);
        *reinterpret_cast<volatile int*>(err) = site;
        __threadfence_system();
    }
};

// A bounded mbarrier wait.  It ends without the barrier (and returns false) after the launch's limit, which it then reports,
// or once another thread of the CTA has given up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Stop* stop, int* err, int site) {
    if (async::mbar_try_wait(bar, parity)) return true;
    const long long t0 = async::clk();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (async::mbar_try_wait(bar, parity)) return true;
        if (stop->is_set()) return false;
        if (stop->late(t0)) {
            stop->give_up(err, site);
            return false;
        }
    }
}

// Signals an mbarrier of a peer CTA (this thread's earlier stores, and what it has seen of others', come before),
// and the bounded wait for such signals.
__device__ __forceinline__ void peer_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, Stop* stop, int* err, int site) {
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
        if (stop->is_set()) return false;
        if (stop->late(t0)) {
            stop->give_up(err, site);
            return false;
        }
    }
}

// The same by a whole warp, which decides as one.  Every lane polls: against one lane that polls and a shuffle that
// tells the others, a block of 128 of the promotion loops took 639 instead of 1042 clocks.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Stop* stop, int* err, int site) {
    if (__all_sync(0xffffffffu, async::mbar_try_wait(bar, parity))) return true;
    const long long t0 = async::clk();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, async::mbar_try_wait(bar, parity))) return true;
        const bool late = stop->late(t0);
        if (late) stop->give_up(err, site);
        if (__any_sync(0xffffffffu, late || stop->is_set())) return false;
    }
}

// Signals an mbarrier of a CTA of the cluster that this thread's tensor-memory loads are done (tcgen05.wait::ld and
// before_sync come first).  It orders nothing else: a release at cluster scope waits for the thread's stores, and made
// a block of 128 of the product take 2200 clocks.
__device__ __forceinline__ void peer_arrive_read(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Both of two barriers.
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, Stop* stop,
                                           int* err, int site) {
    const bool first = async::mbar_try_wait(a, pa), both = async::mbar_try_wait(b, pb) && first;
    if (__all_sync(0xffffffffu, both)) return true;
    return warp_wait(a, pa, stop, err, site) && warp_wait(b, pb, stop, err, site);
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

// The wait of a kernel that has given up, for its own copies and MMAs in flight: it does not look at the stop and has a limit of
// its own, long beside any copy.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
    const long long t0 = async::clk();
    while (!async::mbar_try_wait(bar, parity))
        if (async::clk() - t0 > kDrainClk) return;
}

// Lets a kernel have as much dynamic shared memory as a CTA can (asked for once a device: the call is not free).
template <auto kKernel>
cudaError_t allow_smem() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (done.load(std::memory_order_acquire) >> dev & 1)) return e;
    cudaFuncAttributes a;
    int most = 0;
    e = cudaFuncGetAttributes(&a, kKernel);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)a.sharedSizeBytes);
    if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return e;
}

// --- launchers ----------------------------------------------------------------

// cuTensorMap of a row-major byte matrix [rows, cols] (row stride in bytes), boxes of 128 bytes x
// box_rows in the 128-byte swizzle layout; bytes outside the matrix read as 0.
cudaError_t byte_map(void* map, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, int box_rows);
// The same of up to five dimensions (cols first; strides of the others in bytes), box as given.
cudaError_t byte_map_n(void* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box);
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
    Waits waits;
};
cudaError_t launch_product(const Product& p, cudaStream_t st);
cudaError_t launch_product_small(const Product& p, cudaStream_t st);

}  // namespace f8
}  // namespace mmoe
