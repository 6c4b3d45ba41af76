// Matrix product in e4m3 with a scale per block of 128, dense or grouped.
//
//   y[m, n] = sum_b sa[m, b] sw[n / 128, b] P_b[m, n],   P_b = sum_{k in block b} a[m, k] w[n, k]
//
// P_b leaves the tensor cores (tcgen05 kind::f8f6f4, FP32 accumulators) after
// each block of 128 and is added in FP32 with its scales by the CUDA cores:
// acc = fma(P_b, sa sw, acc).  One rounding, at the store of a BF16 y.
//
// product_kernel (many rows).  A persistent CTA per SM walks over tiles of 128
// rows x 128 H columns (H halves of 128 weight rows).  The rows are the MMA's
// M: each thread of the promotion warps owns one row, so a scale is one
// register per half and block, and its 64 columns of each half stay in
// registers.  Warps:
//   0      producer: per block of 128 the activation tile and the H weight tiles (TMA, 128-byte swizzle)
//   1      TMEM (two buffers of 128 H columns); one lane issues the MMAs, a commit per block
//   2, 3   idle (they complete warpgroup 0, whose registers go to the promotion)
//   4..11  promotion and epilogue: warp w reads TMEM lanes 32 (w % 4).. and columns 64 ((w - 4) / 4)..
//          of each half
//
// product_small_kernel (up to 64 rows).  Bound by one pass over the weights,
// so these are the MMA's M (128 weight rows) and the few activation rows its
// N; a cluster splits the blocks of 128 along K so that every SM streams, and
// adds its partial sums through distributed shared memory in a fixed order.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "fp8.cuh"

namespace mmoe {
namespace f8 {

cudaError_t byte_map(void* map, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, int box_rows) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {stride};
    const cuuint32_t box[2] = {(cuuint32_t)kBlk, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = encode(static_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base),
                              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        n = 148;
    return n;
}

namespace {

using async::mbar_arrive;
using async::mbar_expect_tx;
using async::mbar_init;

constexpr int kTileBytes = kBlk * kBlk;  // one 128 x 128 operand tile: 16 KB

// ------------------------------------------------------------------- many rows

constexpr int kBufs = 2;                 // TMEM buffers
constexpr int kTInfo = 4;                // tiles published ahead
constexpr int kPromoWarps = 8;
constexpr int kThreads = 128 + 32 * kPromoWarps;
// Register split (setmaxnreg): 168 a thread at launch; warpgroup 0 drops to 32, the promotion rises to 232.
constexpr int kRegsLow = 32, kRegsHigh = 232;
static_assert(128 * kRegsLow + 32 * kPromoWarps * kRegsHigh <= kThreads * 168, "register split");
constexpr int kStageRow = 80;            // bytes of an output row in the staging buffer: 64 + 16 against bank conflicts
constexpr int kStageBytes = 32 * kStageRow;

struct TileInfo {
    int end;
    int nr;        // valid rows
    int n0;        // first output column
    int sw0;       // index of the first half's weight scales (of block 0)
    int64_t row0;
};

template <int H>
constexpr int stages() {
    return H == 2 ? 4 : 5;
}

template <int H>
struct Smem {
    alignas(1024) uint8_t ring[stages<H>()][(1 + H) * kTileBytes];
    uint8_t out[kPromoWarps][kStageBytes];
    uint64_t full[stages<H>()], empty[stages<H>()];
    uint64_t accf[kBufs], acce[kBufs];
    uint64_t tfull[kTInfo], tempty[kTInfo];
    TileInfo ti[kTInfo];
    uint32_t tmem;
    int abort;
    int off[kMaxGroups + 1];     // grouped: first row of each group
    int tiles[kMaxGroups + 1];   // grouped: row tiles before each group
};

// Offsets of the groups, made harmless: within [0, M] and not decreasing, whatever the array holds.
// Warp 0 of the CTA; 32 groups a step.
template <int H>
__device__ __forceinline__ void load_groups(const Product& p, Smem<H>* sm, int lane) {
    int prev = 0, base = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        const int g = g0 + lane;
        int o = g < p.groups ? p.offsets[g + 1] : 0;
        if (g0 == 0) {
            int first = p.offsets[0];
            first = min(max(first, 0), (int)p.M);
            prev = first;
            if (lane == 0) {
                sm->off[0] = first;
                sm->tiles[0] = 0;
            }
        }
        o = min(max(o, prev), (int)p.M);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, o, d);
            if (lane >= d) o = max(o, u);
        }
        int before = __shfl_up_sync(0xffffffffu, o, 1);
        if (lane == 0) before = prev;
        int t = g < p.groups ? (o - before + kBlk - 1) / kBlk : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += u;
        }
        if (g < p.groups) {
            sm->off[g + 1] = o;
            sm->tiles[g + 1] = base + t;
        }
        prev = __shfl_sync(0xffffffffu, o, 31);
        base += __shfl_sync(0xffffffffu, t, 31);
    }
    __syncwarp();
}

// 64 bytes of an output row: a staging row, written by the thread that owns the row ...
__device__ __forceinline__ void stage_row(uint8_t* row, const float2* acc, __nv_bfloat16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(row + 16 * i) =
            make_uint4(bf16x2(acc[4 * i].x, acc[4 * i].y), bf16x2(acc[4 * i + 1].x, acc[4 * i + 1].y),
                       bf16x2(acc[4 * i + 2].x, acc[4 * i + 2].y), bf16x2(acc[4 * i + 3].x, acc[4 * i + 3].y));
}
__device__ __forceinline__ void stage_row(uint8_t* row, const float2* acc, float) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(row + 16 * i) = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
}

// ... and the warp's 32 such rows on to global memory, 4 lanes a row (16 bytes each) where the row of y
// and the columns allow it, else element by element.
template <class T>
__device__ __forceinline__ void store_rows(const uint8_t* st, T* y, int64_t ldy, int nr, int col, int N, bool wide,
                                           int lane) {
    constexpr int kCols = 64 / (int)sizeof(T);
    if (col >= N) return;
    if (wide && col + kCols <= N) {
        const int c = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r < nr)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(y + r * ldy + col) + 16 * c) =
                    *reinterpret_cast<const uint4*>(st + r * kStageRow + 16 * c);
        }
        return;
    }
    const int c = lane % kCols;
    for (int r = lane / kCols; r < nr; r += 32 / kCols)
        if (col + c < N) y[r * ldy + col + c] = *reinterpret_cast<const T*>(st + r * kStageRow + c * (int)sizeof(T));
}

template <int H, class T>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap, const Product p)
{
    constexpr int S = stages<H>();
    constexpr int kTx = (1 + H) * kTileBytes;
    constexpr int kCols = 64;  // columns of each half a promotion thread owns
    extern __shared__ uint8_t smem_raw[];
    Smem<H>* sm = reinterpret_cast<Smem<H>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int KB = (p.K + kBlk - 1) / kBlk, nb = (p.N + kBlk - 1) / kBlk, ntiles = (nb + H - 1) / H;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sm->accf[i], 1);
            mbar_init(&sm->acce[i], kPromoWarps);
        }
        for (int i = 0; i < kTInfo; ++i) {
            mbar_init(&sm->tfull[i], 1);
            mbar_init(&sm->tempty[i], 1 + kPromoWarps);
        }
        sm->abort = 0;
        async::fence_barrier_init();
    }
    if (warp == 1) {
        tc5::tmem_alloc(&sm->tmem, kBufs * H * kBlk);
        tc5::before_sync();
    }
    dep_wait();
    __syncthreads();
    tc5::after_sync();
    dep_launch();  // not before this CTA has its TMEM: a dependent that waits for this grid may take the rest
    const uint32_t tmem = sm->tmem;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0) {
            int64_t total;
            if (p.groups) {
                load_groups<H>(p, sm, lane);
                total = (int64_t)sm->tiles[p.groups] * ntiles;
            } else {
                total = (p.M + kBlk - 1) / kBlk * ntiles;
            }
            int sc = 0, tc = 0;
            bool ok = true;
            for (int64_t L = blockIdx.x; ok; L += gridDim.x, ++tc) {
                const int b = tc % kTInfo;
                if (tc >= kTInfo && !warp_wait(&sm->tempty[b], (tc / kTInfo - 1) & 1, &sm->abort, p.err, 1)) break;
                TileInfo& ti = sm->ti[b];
                if (L >= total) {
                    if (lane == 0) {
                        ti.end = 1;
                        mbar_arrive(&sm->tfull[b]);
                    }
                    break;
                }
                // column tiles innermost: the CTAs that run together share activation tiles in L2
                const int64_t mt = L / ntiles;
                const int nt = (int)(L - mt * ntiles);
                int g = 0;
                int64_t row0 = mt * kBlk, rows = p.M;
                if (p.groups) {
                    int lo = 0, hi = p.groups - 1;  // the last group with tiles[g] <= mt
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (sm->tiles[mid] <= mt) lo = mid;
                        else hi = mid - 1;
                    }
                    g = lo;
                    row0 = sm->off[g] + (mt - sm->tiles[g]) * kBlk;
                    rows = sm->off[g + 1];
                }
                const int n0 = nt * H * kBlk;
                if (lane == 0) {
                    ti.end = 0;
                    ti.nr = (int)min((int64_t)kBlk, rows - row0);
                    ti.n0 = n0;
                    ti.sw0 = (g * nb + nt * H) * KB;
                    ti.row0 = row0;
                    mbar_arrive(&sm->tfull[b]);
                }
                const int w0 = g * p.N + n0;
                for (int kb = 0; kb < KB; ++kb, ++sc) {
                    const int s = sc % S;
                    if (sc >= S && !warp_wait(&sm->empty[s], (sc / S - 1) & 1, &sm->abort, p.err, 2)) {
                        ok = false;
                        break;
                    }
                    if (elect()) {
                        mbar_expect_tx(&sm->full[s], kTx);
                        tc5::tma_load_2d(sm->ring[s], &amap, kb * kBlk, (int)row0, &sm->full[s]);
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            tc5::tma_load_2d(sm->ring[s] + (1 + h) * kTileBytes, &wmap, kb * kBlk, w0 + h * kBlk,
                                             &sm->full[s]);
                    }
                    __syncwarp();
                }
            }
            // every copy has landed before the CTA may exit
            for (int i = max(sc - S, 0); i < sc; ++i) wait_drain(&sm->full[i % S], (i / S) & 1);
        } else if (warp == 1) {
            // the warp walks together and one lane issues: in a branch of one lane the same loop starves beside the
            // promotion warps
            int sc = 0, tc = 0;
            bool ok = true;
            while (ok) {
                const int b = tc % kTInfo;
                if (!warp_wait(&sm->tfull[b], (tc / kTInfo) & 1, &sm->abort, p.err, 3)) break;
                const int end = sm->ti[b].end;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->tempty[b]);
                ++tc;
                if (end) break;
                for (int kb = 0; kb < KB; ++kb, ++sc) {
                    const int s = sc % S, d = sc % kBufs;
                    if (!warp_wait(&sm->full[s], (sc / S) & 1, &sm->abort, p.err, 4) ||
                        !warp_wait(&sm->acce[d], (sc / kBufs) & 1, &sm->abort, p.err, 5)) {
                        ok = false;
                        break;
                    }
                    tc5::after_sync();
                    const uint64_t ad = tc5::smem_desc_sw128(sm->ring[s]);
                    const uint64_t wd = tc5::smem_desc_sw128(sm->ring[s] + kTileBytes);
                    const uint32_t dt = tmem + d * H * kBlk;
                    if (elect()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 of K (32 bytes, 2 descriptor units) each
                            mma_e4m3(dt, ad + 2 * k, wd + 2 * k, idesc_e4m3(H * kBlk), k > 0);
                        tc5::commit(&sm->empty[s]);
                        tc5::commit(&sm->accf[d]);
                    }
                    __syncwarp();
                }
            }
            // every MMA has completed before TMEM is released
            if (sc > 0) wait_drain(&sm->accf[(sc - 1) % kBufs], ((sc - 1) / kBufs) & 1);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        const int quarter = warp & 3, cg = (warp - 4) >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + cg * kCols;
        uint8_t* stage = sm->out[warp - 4];
        const bool wide = ((reinterpret_cast<uintptr_t>(p.y) | (uintptr_t)(p.ldy * (int)sizeof(T))) & 15) == 0;
        if (lane == 0)
            for (int b = 0; b < kBufs; ++b) mbar_arrive(&sm->acce[b]);
        int sc = 0, tc = 0;
        bool ok = true;
        while (ok) {
            const int tb = tc % kTInfo;
            if (!warp_wait(&sm->tfull[tb], (tc / kTInfo) & 1, &sm->abort, p.err, 6)) break;
            const TileInfo ti = sm->ti[tb];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->tempty[tb]);
            ++tc;
            if (ti.end) break;
            const float* sa = p.sa + (ti.row0 + min(row, ti.nr - 1)) * KB;
            const float* sw = p.sw + ti.sw0;
            const int second = (H == 2 && ti.n0 + kBlk < p.N) ? KB : 0;  // a last half past the matrix: unused columns
            float2 acc[H][kCols / 2];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int c = 0; c < kCols / 2; ++c) acc[h][c] = make_float2(0.0f, 0.0f);
            float a1 = sa[0], w0 = sw[0], w1 = sw[second];
            for (int kb = 0; kb < KB; ++kb, ++sc) {
                const int d = sc % kBufs;
                const float s[2] = {a1 * w0, a1 * w1};
                if (kb + 1 < KB) {
                    a1 = sa[kb + 1];
                    w0 = sw[kb + 1];
                    w1 = sw[second + kb + 1];
                }
                if (!warp_wait(&sm->accf[d], (sc / kBufs) & 1, &sm->abort, p.err, 7)) {
                    ok = false;
                    break;
                }
                tc5::after_sync();
                const uint32_t ta = tl + d * H * kBlk;
                // 32 columns at a time, each load under the additions of the one before; the buffer goes
                // back to the MMA when the last has landed
                uint32_t v[2][32];
                tc5::tmem_ld32(ta, v[0]);
#pragma unroll
                for (int i = 0; i < 2 * H; ++i) {
                    tc5::tmem_wait_ld(v[i & 1]);
                    if (i + 1 < 2 * H) {
                        tc5::tmem_ld32(ta + ((i + 1) >> 1) * kBlk + ((i + 1) & 1) * 32, v[(i + 1) & 1]);
                    } else {
                        tc5::before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm->acce[d]);
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float2& to = acc[i >> 1][(i & 1) * 16 + c];
                        to.x = fmaf(__uint_as_float(v[i & 1][2 * c]), s[i >> 1], to.x);
                        to.y = fmaf(__uint_as_float(v[i & 1][2 * c + 1]), s[i >> 1], to.y);
                    }
                }
            }
            if (!ok || *reinterpret_cast<volatile int*>(&sm->abort)) break;
            constexpr int kChunk = 64 / (int)sizeof(T);
            T* y = static_cast<T*>(p.y) + (ti.row0 + quarter * 32) * p.ldy;
            const int nr = min(ti.nr - quarter * 32, 32);
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int c = 0; c < kCols / kChunk; ++c) {
                    stage_row(stage + lane * kStageRow, &acc[h][c * kChunk / 2], T());
                    __syncwarp();
                    store_rows<T>(stage, y, p.ldy, nr, ti.n0 + h * kBlk + cg * kCols + c * kChunk, p.N, wide, lane);
                    __syncwarp();
                }
        }
    }
    tc5::before_sync();
    __syncthreads();
    tc5::after_sync();
    if (warp == 1) tc5::tmem_dealloc(tmem, kBufs * H * kBlk);
}

// -------------------------------------------------------------------- few rows

constexpr int kRing = 8;                     // weight tiles in flight: 128 KB of the about 66 KB an SM needs
constexpr int kOperand = 64 * 1024;          // codes of the activation rows, as many blocks of K as fit
constexpr int kSBufs = 4;                    // TMEM buffers
constexpr int kSThreads = 192;               // producer, MMA, four promotion warps

template <int NT>
struct SmallSmem {
    alignas(1024) uint8_t ring[kRing][kTileBytes];
    alignas(1024) uint8_t b[kOperand];       // [block][NT rows][128 bytes], swizzled; then the partial sums [NT][128]
    float sx[kOperand / (NT * kBlk)][NT];
    uint64_t full[kRing], empty[kRing], accf[kSBufs], acce[kSBufs], ready, drained;
    uint32_t tmem;
    int abort;
};

// NT: rows rounded up to 16, 32 or 64.  The cluster's CTA r takes the blocks kb = r, r + C, ...
template <int NT, class T>
__global__ void __launch_bounds__(kSThreads, 1)
product_small_kernel(const __grid_constant__ CUtensorMap wmap, const Product p, const int C)
{
    constexpr int kRound = kOperand / (NT * kBlk);  // blocks of K the operand buffer holds
    constexpr uint32_t kCols = NT * kSBufs;
    extern __shared__ uint8_t smem_raw[];
    SmallSmem<NT>* sm = reinterpret_cast<SmallSmem<NT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int nt = blockIdx.x / C;
    const int KB = (p.K + kBlk - 1) / kBlk;
    const int mine = (KB - rank + C - 1) / C;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(&sm->accf[i], 1);
            mbar_init(&sm->acce[i], 4);
        }
        mbar_init(&sm->ready, 128);
        mbar_init(&sm->drained, 4);
        sm->abort = 0;
        async::fence_barrier_init();
    }
    if (warp == 1) {
        tc5::tmem_alloc(&sm->tmem, kCols);
        tc5::before_sync();
    }
    dep_wait();
    __syncthreads();
    tc5::after_sync();
    dep_launch();  // not before this CTA has its TMEM: a dependent that waits for this grid may take the rest
    const uint32_t tmem = sm->tmem;
    const int m = (int)p.M;

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < mine; ++i) {
                const int s = i % kRing;
                if (i >= kRing && !wait(&sm->empty[s], (i / kRing - 1) & 1, &sm->abort, p.err, 11)) break;
                mbar_expect_tx(&sm->full[s], kTileBytes);
                tc5::tma_load_2d(sm->ring[s], &wmap, (rank + i * C) * kBlk, nt * kBlk, &sm->full[s]);
            }
            for (int j = max(i - kRing, 0); j < i; ++j) wait_drain(&sm->full[j % kRing], (j / kRing) & 1);
        }
    } else if (warp == 1) {
        int i = 0;
        for (; i < mine; ++i) {
            const int s = i % kRing, d = i % kSBufs, r = i % kRound;
            if (r == 0 && !warp_wait(&sm->ready, (i / kRound) & 1, &sm->abort, p.err, 12)) break;
            if (!warp_wait(&sm->full[s], (i / kRing) & 1, &sm->abort, p.err, 13) ||
                !warp_wait(&sm->acce[d], (i / kSBufs) & 1, &sm->abort, p.err, 14))
                break;
            tc5::after_sync();
            const uint64_t wd = tc5::smem_desc_sw128(sm->ring[s]);
            const uint64_t bd = tc5::smem_desc_sw128(sm->b + r * NT * kBlk);
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3(tmem + d * NT, wd + 2 * k, bd + 2 * k, idesc_e4m3(NT), k > 0);
                tc5::commit(&sm->empty[s]);
                tc5::commit(&sm->accf[d]);
            }
            __syncwarp();
        }
        if (i > 0) wait_drain(&sm->accf[(i - 1) % kSBufs], ((i - 1) / kSBufs) & 1);
    } else {
        const int pt = tid - 64, quarter = warp & 3;
        const int row = quarter * 32 + lane;  // weight row of the tile
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        if (lane == 0)
            for (int b = 0; b < kSBufs; ++b) mbar_arrive(&sm->acce[b]);
        float2 acc[NT / 2];
#pragma unroll
        for (int c = 0; c < NT / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
        const float* sw = p.sw + (int64_t)nt * KB + rank;
        for (int i0 = 0; i0 < mine; i0 += kRound) {
            if (i0 > 0) {  // the operand buffer and its scales are free once every warp has added the last round
                if (lane == 0) mbar_arrive(&sm->drained);
                if (!warp_wait(&sm->drained, (i0 / kRound - 1) & 1, &sm->abort, p.err, 17)) break;
            }
            // operand rows of this round: a half warp per (row, block)
            const int n = min(kRound, mine - i0);
            const int hl = pt & 15;
            for (int j = pt >> 4; j < n * m; j += 8) {
                const int r = j / m, t = j - r * m;
                const int kb = rank + (i0 + r) * C, col = kb * kBlk + hl * 8;
                uint2 code = make_uint2(0u, 0u);
                if (p.x) {
                    float v[8] = {};
                    if (col < p.K) load8(p.x + t * p.ldx + col, v);
                    // the half warps of a warp may part at the end of the loop
                    uint32_t am = amax8(v);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1)
                        am = max(am, __shfl_xor_sync(0xffffu << (threadIdx.x & 16), am, o));
                    const float sc = scale_of(am);
                    code = make_uint2(e4m3x4(v, sc), e4m3x4(v + 4, sc));
                    if (hl == 0) sm->sx[r][t] = sc;
                } else {
                    if (col < p.K) code = *reinterpret_cast<const uint2*>(p.a + (int64_t)t * p.K + col);
                    if (hl == 0) sm->sx[r][t] = p.sa[(int64_t)t * KB + kb];
                }
                // 128-byte swizzle: 16-byte chunk c of row t lies at chunk c ^ (t & 7)
                *reinterpret_cast<uint2*>(sm->b + (r * NT + t) * kBlk + (((hl >> 1) ^ (t & 7)) << 4) + (hl & 1) * 8) = code;
            }
            fence_async_smem();
            mbar_arrive(&sm->ready);
            if (!warp_wait(&sm->ready, (i0 / kRound) & 1, &sm->abort, p.err, 15)) break;
            float ws = sw[(int64_t)i0 * C];
            bool ok = true;
            for (int r = 0; r < n; ++r) {
                const int i = i0 + r, d = i % kSBufs;
                const float w = ws;
                if (r + 1 < n) ws = sw[(int64_t)(i + 1) * C];
                if (!warp_wait(&sm->accf[d], (i / kSBufs) & 1, &sm->abort, p.err, 16)) {
                    ok = false;
                    break;
                }
                tc5::after_sync();
#pragma unroll
                for (int c0 = 0; c0 < NT; c0 += 16) {
                    uint32_t v[16];
                    tc5::tmem_ld16(tl + d * NT + c0, v);
                    tc5::tmem_wait_ld(v);
                    if (c0 + 16 == NT) {
                        tc5::before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm->acce[d]);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float2 x2 = *reinterpret_cast<const float2*>(&sm->sx[r][c0 + 2 * c]);
                        acc[c0 / 2 + c] = __ffma2_rn(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])),
                                                     make_float2(x2.x * w, x2.y * w), acc[c0 / 2 + c]);
                    }
                }
            }
            if (!ok) break;
        }
        // every MMA of this CTA has been read: the operand buffer takes the partial sums
        float* part = reinterpret_cast<float*>(sm->b);
        if (C > 1) {
#pragma unroll
            for (int c = 0; c < NT / 2; ++c) {
                part[(2 * c) * kBlk + row] = acc[c].x;
                part[(2 * c + 1) * kBlk + row] = acc[c].y;
            }
        } else {
            T* y = static_cast<T*>(p.y) + nt * kBlk + row;
            if (nt * kBlk + row < p.N && !sm->abort) {
#pragma unroll
                for (int c = 0; c < NT / 2; ++c) {
                    if (2 * c < m) y[(2 * c) * p.ldy] = (T)acc[c].x;
                    if (2 * c + 1 < m) y[(2 * c + 1) * p.ldy] = (T)acc[c].y;
                }
            }
        }
    }
    if (C > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp >= 2) {
            const int row = (warp & 3) * 32 + lane;
            T* y = static_cast<T*>(p.y) + nt * kBlk + row;
            for (int t = rank; t < m; t += C) {
                float sum = 0.0f;
#pragma unroll 4
                for (int c = 0; c < C; ++c)
                    sum += peer_load(peer_addr(reinterpret_cast<const float*>(sm->b) + t * kBlk + row, (uint32_t)c));
                if (nt * kBlk + row < p.N && !sm->abort) y[t * p.ldy] = (T)sum;
            }
        }
        // the partial sums stay until every CTA has read them
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    tc5::before_sync();
    __syncthreads();
    tc5::after_sync();
    if (warp == 1) tc5::tmem_dealloc(tmem, kCols);
}

template <class K, class... A>
cudaError_t launch(K kern, unsigned grid, unsigned threads, size_t smem, int cluster, cudaStream_t st, A... args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int H>
cudaError_t launch_many(const Product& p, const CUtensorMap& am, const CUtensorMap& wm, int64_t tiles, cudaStream_t st) {
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, sm_count());
    const size_t smem = sizeof(Smem<H>) + 1024;
    return p.y_bf16 ? launch(product_kernel<H, __nv_bfloat16>, grid, kThreads, smem, 1, st, am, wm, p)
                    : launch(product_kernel<H, float>, grid, kThreads, smem, 1, st, am, wm, p);
}

template <int NT>
cudaError_t launch_few(const Product& p, const CUtensorMap& wm, int C, cudaStream_t st) {
    const unsigned grid = (unsigned)(blocks_of(p.N) * C);
    const size_t smem = sizeof(SmallSmem<NT>) + 1024;
    return p.y_bf16 ? launch(product_small_kernel<NT, __nv_bfloat16>, grid, kSThreads, smem, C, st, wm, p, C)
                    : launch(product_small_kernel<NT, float>, grid, kSThreads, smem, C, st, wm, p, C);
}

}  // namespace

cudaError_t launch_product(const Product& p, cudaStream_t st) {
    CUtensorMap am, wm;
    const int64_t G = p.groups ? p.groups : 1;
    cudaError_t e = byte_map(&am, p.a, (uint64_t)p.K, (uint64_t)p.M, (uint64_t)p.K, kBlk);
    if (e == cudaSuccess) e = byte_map(&wm, p.w, (uint64_t)p.K, (uint64_t)(G * p.N), (uint64_t)p.K, kBlk);
    if (e != cudaSuccess) return e;
    // tiles at most: each group may end inside a tile of rows
    const int64_t mt = p.groups ? std::min<int64_t>(p.M / kBlk + p.groups, p.M) : blocks_of(p.M);
    const int64_t nb = blocks_of(p.N);
    // 256 columns a tile read the activations half as often; 128 where that leaves SMs without a tile
    if (nb > 1 && mt * ((nb + 1) / 2) >= sm_count()) return launch_many<2>(p, am, wm, mt * ((nb + 1) / 2), st);
    return launch_many<1>(p, am, wm, mt * nb, st);
}

cudaError_t launch_product_small(const Product& p, cudaStream_t st) {
    CUtensorMap wm;
    cudaError_t e = byte_map(&wm, p.w, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.K, kBlk);
    if (e != cudaSuccess) return e;
    // CTAs along K: as many as there are SMs for
    int C = 1;
    while (C < 8 && 2 * C <= blocks_of(p.K) && blocks_of(p.N) * 2 * C <= sm_count()) C *= 2;
    return p.M <= 16 ? launch_few<16>(p, wm, C, st) : p.M <= 32 ? launch_few<32>(p, wm, C, st) : launch_few<64>(p, wm, C, st);
}

}  // namespace f8
}  // namespace mmoe
