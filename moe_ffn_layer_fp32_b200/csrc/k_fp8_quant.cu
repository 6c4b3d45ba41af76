// Quantisation to e4m3 codes with one FP32 scale per block of 128.
//
// Both kernels read every value once, keep it in registers between the
// maximum and the division, and write one byte a value: they are bound by
// memory (3 bytes a value for BF16 rows).
#include "fp8.cuh"

namespace mmoe {
namespace f8 {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;  // blocks a half warp holds at once: enough loads in flight to cover the latency

// 8 values as they lie in memory (zeros until loaded).
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
    float v[8] = {};
    __device__ __forceinline__ void load(const float* p) { load8(p, v); }
    __device__ __forceinline__ uint32_t amax() const { return amax8(v); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = v[j];
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u = {0u, 0u, 0u, 0u};
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ uint32_t amax() const { return amax_bf16(u); }
    __device__ __forceinline__ void get(float (&o)[8]) const { unpack8(u, o); }
};

// Rows: a half warp takes one (row, block) at a time, 8 values a lane (16 bytes of BF16).
template <class T>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const T* x, int64_t nblk, int kb, int K,
                                                                 int64_t ldx, uint8_t* q,
                                                                 float* s)
{
    const int hl = threadIdx.x & 15;
    dep_launch();
    dep_wait();
    constexpr int kPer = kThreads / 16 * kItems;  // blocks a CTA takes, kItems in a row a half warp
    const int64_t begin = (int64_t)blockIdx.x * kPer, row0 = begin / kb;
    const int b0 = (int)(begin - row0 * kb), mine = (threadIdx.x >> 4) * kItems;
    const int64_t first = begin + mine;
    Raw8<T> v[kItems];
    int64_t at[kItems];  // of the lane's values in q (-1: none)
    int64_t row = row0 + (b0 + mine) / kb;  // 64-bit divisions for each block took three times the copy's time
    int col = (b0 + mine) % kb * kBlk + hl * 8;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const bool in = first + i < nblk && col < K;
        at[i] = in ? row * K + col : -1;
        if (in) v[i].load(x + row * ldx + col);
        col += kBlk;
        if (col >= kb * kBlk) {
            col = hl * 8;
            ++row;
        }
    }
    float sc[kItems];
    uint2 code[kItems];
    encode<kItems>(kItems, [&](int i) { return v[i].amax(); }, [&](int i, float (&o)[8]) { v[i].get(o); }, sc, code);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (hl == 0 && first + i < nblk) s[first + i] = sc[i];
        if (at[i] >= 0) *reinterpret_cast<uint2*>(q + at[i]) = code[i];
    }
}

// Weights: one CTA per 128 x 128 block; a half warp takes a row at a time.
template <class T>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const T* w, int nb, int kb, int N,
                                                                   int K, uint8_t* q,
                                                                   float* s)
{
    constexpr int kRows = kBlk / (kThreads / 16);
    __shared__ uint32_t part[kThreads / 32];
    const int hl = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int64_t blk = blockIdx.x;  // (batch * nb + row block) * kb + column block
    const int64_t bn = blk / kb;
    const int col = (int)(blk - bn * kb) * kBlk + hl * 8;
    const int64_t batch = bn / nb;
    const int n0 = (int)(bn - batch * nb) * kBlk;
    dep_launch();
    dep_wait();
    float v[kRows][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int n = n0 + r0 + i * (kThreads / 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        if (n < N && col < K) load8(w + (batch * N + n) * K + col, v[i]);
        m = max(m, amax8(v[i]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    const float sc = scale_of(m);
    if (threadIdx.x == 0) s[blk] = sc;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int n = n0 + r0 + i * (kThreads / 16);
        if (n < N && col < K)
            *reinterpret_cast<uint2*>(q + (batch * N + n) * K + col) =
                Coder(sc)(v[i]);
    }
}

cudaLaunchConfig_t dependent(unsigned grid, cudaStream_t st, cudaLaunchAttribute* at) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* q, float* s,
                                 cudaStream_t st) {
    const int64_t kb = blocks_of(K), nblk = rows * kb, per = kThreads / 16 * kItems;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = dependent((unsigned)((nblk + per - 1) / per), st, &at);
    return bf16 ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<__nv_bfloat16>, (const __nv_bfloat16*)x, nblk, (int)kb,
                                     (int)K, ldx, q, s)
                : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<float>, (const float*)x, nblk, (int)kb, (int)K, ldx, q,
                                     s);
}

cudaError_t launch_quantize_blocks(const void* w, bool bf16, int64_t batch, int64_t N, int64_t K, uint8_t* q, float* s,
                                   cudaStream_t st) {
    const int64_t nb = blocks_of(N), kb = blocks_of(K);
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = dependent((unsigned)(batch * nb * kb), st, &at);
    return bf16 ? cudaLaunchKernelEx(&cfg, quantize_blocks_kernel<__nv_bfloat16>, (const __nv_bfloat16*)w, (int)nb,
                                     (int)kb, (int)N, (int)K, q, s)
                : cudaLaunchKernelEx(&cfg, quantize_blocks_kernel<float>, (const float*)w, (int)nb, (int)kb, (int)N,
                                     (int)K, q, s);
}

}  // namespace f8
}  // namespace mmoe
