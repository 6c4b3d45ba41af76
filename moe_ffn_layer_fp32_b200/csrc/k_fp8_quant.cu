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
constexpr int kItems = 2;  // blocks that 8 lanes hold at once: 64 bytes of BF16 a lane in flight

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

// Rows: 8 lanes take a (row, block), 16 values a lane in two halves of 8.  Issue slots bound it beside the memory (24 us
// for 16384 x 2048 BF16 values with 16 lanes a block, whose copy takes 16), so what is done once a block or once a thread
// is shared, and where the rows' blocks can be counted in 32 bits they are.
template <class T>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const T* x, int64_t nblk, int kb, int K,
                                                                 int64_t ldx, uint8_t* q,
                                                                 float* s)
{
    constexpr int kPer = kThreads / 8 * kItems;  // blocks a CTA takes, kItems in a row 8 lanes
    const int l = threadIdx.x & 7;
    const int64_t first = (int64_t)blockIdx.x * kPer + (threadIdx.x >> 3) * kItems;
    const int64_t row = nblk < (int64_t(1) << 31) ? (int64_t)((uint32_t)first / (uint32_t)kb) : first / kb;
    int col = (int)(first - row * kb) * kBlk + l * 8;
    const T* from = x + row * ldx + col;
    uint8_t* to = q + row * K + col;
    dep_launch();
    dep_wait();
    Raw8<T> v[kItems][2];
    uint8_t* at[kItems][2];  // where the lane's codes go (null: nowhere)
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            at[i][h] = nullptr;
            if (first + i < nblk && col + 64 * h < K) {
                v[i][h].load(from + 64 * h);
                at[i][h] = to + 64 * h;
            }
        }
        col += kBlk;
        from += kBlk;
        to += kBlk;
        if (col >= kb * kBlk) {  // on to the next row
            col -= kb * kBlk;
            from += ldx - (int64_t)kb * kBlk;
            to += K - kb * kBlk;
        }
    }
    float sc[kItems];
    uint2 code[kItems][2];
    encode<kItems>(kItems, [&](int i) { return max(v[i][0].amax(), v[i][1].amax()); },
                   [&](int i, int h, float (&o)[8]) { v[i][h].get(o); }, sc, code);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (l == 0 && first + i < nblk) s[first + i] = sc[i];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (at[i][h]) *reinterpret_cast<uint2*>(at[i][h]) = code[i][h];
    }
}

// Weights: one CTA per 128 x 128 block; a half warp takes a row at a time.  60 x 2048 x 2048 FP32 values take 190 us, the
// time of their traffic; BF16 ones take 379 us for 115 us of traffic, and have not been made faster (weights are quantised
// once).
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
    const int64_t kb = blocks_of(K), nblk = rows * kb, per = kThreads / 8 * kItems;
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
