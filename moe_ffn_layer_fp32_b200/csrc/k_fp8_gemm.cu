// Matrix product in e4m3 with a scale per block of 128, dense or grouped.
//
//   y[m, n] = sum_b sa[m, b] sw[n / 128, b] P_b[m, n],   P_b = sum_{k in block b} a[m, k] w[n, k]
//
// P_b leaves the tensor cores (tcgen05 kind::f8f6f4, FP32 accumulators) after
// each block of 128 and is added in FP32 with its scales by the CUDA cores:
// acc = fma(P_b, sa sw, acc).  One rounding, at the store of a BF16 y.
//
// product_kernel (many rows).  Persistent CTAs, or pairs of CTAs (cta_group::2: each loads its own 128 rows and half of the
// weight rows, so that a block of 128 brings 32 KB instead of 48 KB into an SM's shared memory), walk over tiles of C x 128
// rows x H x 128 columns.  The rows are the MMA's M: each thread of the promotion warps owns one row, so a scale is one
// register a block, and its columns stay in registers.  Warps:
//   0      producer: per block of 128 the activation and the weight tile (TMA, 128-byte swizzle)
//   1, 2   issue the MMAs, a block in turn, into 512 / (128 H) buffers of TMEM (tiles of 128 x 256: warp 1 alone)
//   3      idle (it completes warpgroup 0, whose registers go to the promotion; so is warp 2 there)
//   4..11  promotion and epilogue: warp w reads TMEM lanes 32 (w % 4).. and half of the columns; y goes out through
//          shared memory by the copy engine, while the next tile is on its way
// What bounds it: the handoffs, and the ends of tiles.  16384 x 2048 x 2048 takes 70 us (1.96 PFLOP/s) at 1.67 GHz, 117,800
// clocks a CTA, by clocks read in the promotion warps: seven tiles of 16 blocks at 750 clocks (of which a block's MMAs run
// 515) and 2,150 to stage and store y, while the MMAs run only as far ahead as there are buffers, then 300 to the next
// tile's first block; 3,700 before the first tile and 3,000 after the last; the rest is the wait for the launch before.
// Without the additions a block took 725 of then 800 clocks, without the TMEM loads 550, without the copies no less.  More
// buffers of half the width, four promotion warps a half, FFMA2, a poll of the next buffer ahead of time and 16-byte stores
// by the warps themselves were all slower or no faster.
//
// product_small_kernel (up to 64 rows).  Bound by one pass over the weights and its own latencies, so these are the MMA's M
// (128 weight rows) and the few activation rows its N; a cluster splits the blocks of 128 along K so that every SM streams,
// and adds its partial sums through distributed shared memory in a fixed order.  1 x 2048 x 1024: 3.6 us a launch in a
// chain (with 200 KB of shared memory instead of half, which keeps the next launch off the SM, 7.5 us), 3.8 us where each
// launch's weights come from HBM; 64 x 4096 x 2048: 11.0 and 11.3 us, half of it for the codes of the rows, which every
// cluster makes for itself.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "fp8.cuh"

namespace mmoe {
namespace f8 {

namespace {
cudaError_t encode_map(void* map, CUtensorMapDataType type, const void* base, int rank, const uint64_t* dims,
                       const uint64_t* strides, const uint32_t* box) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return cudaErrorNotSupported;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], step[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        step[i] = 1;
        if (i + 1 < rank) s[i] = strides[i];
    }
    const CUresult r = encode(static_cast<CUtensorMap*>(map), type, (cuuint32_t)rank, const_cast<void*>(base), d, s, b, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// y in boxes of 32 rows x 128 bytes
cudaError_t out_map(void* map, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, bool bf16) {
    const uint64_t dims[2] = {cols, rows};
    const uint32_t box[2] = {bf16 ? 64u : 32u, 32u};
    return encode_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, 2, dims, &stride, box);
}
}  // namespace

cudaError_t byte_map_n(void* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rank, dims, strides, box);
}

cudaError_t byte_map(void* map, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, int box_rows) {
    const uint64_t dims[2] = {cols, rows};
    const uint32_t box[2] = {(uint32_t)kBlk, (uint32_t)box_rows};
    return byte_map_n(map, base, 2, dims, &stride, box);
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

constexpr int kTmemCols = 512;            // two or four buffers of a tile's width
constexpr int kMaxBufs = 4;
constexpr int kTInfo = 4;                // tiles published ahead
constexpr long long kLandClk = 2000000;  // what a copy is given to land where no barrier tells
constexpr int kPromoWarps = 8;
constexpr int kThreads = 128 + 32 * kPromoWarps;
// Register split (setmaxnreg): 168 a thread at launch; warpgroup 0 drops to 40, the promotion rises to 232.
constexpr int kRegsLow = 40, kRegsHigh = 232;
static_assert(128 * kRegsLow + 32 * kPromoWarps * kRegsHigh <= kThreads * 168, "register split");

struct TileInfo {
    int end;
    int nr;        // valid rows
    int n0;        // first output column
    int sw0;       // index of the first half's weight scales (of block 0)
    int64_t row0;
};

// A tile is C x 128 rows and H x 128 columns, by a pair of CTAs (C = 2, each with 128 rows, and with half of the weight
// rows in its shared memory) or by one.
template <int C, int H>
struct Smem {
    static constexpr int kWeights = H / C * kTileBytes;            // of a block of K, in a CTA
    // (Four stages and two issuers of 128 x 256, with half the staging, are faster in short runs, 103 us instead of 110 for
    // 32768 expert rows, and slower under the power cap, 133 us instead of 129.)
    static constexpr int kStages = H > C ? 3 : 4;
    static constexpr int kOut = 8192;                              // staging of a promotion warp: 32 rows x 128 bytes, once or twice
    alignas(1024) uint8_t ring[kStages][kTileBytes + kWeights];    // 128 activation rows, the weight rows
    alignas(1024) uint8_t out[kPromoWarps][kOut];
    uint64_t full[kStages], empty[kStages];
    uint64_t accf[kMaxBufs], acce[kMaxBufs];
    uint64_t tfull[kTInfo], tempty[kTInfo];
    TileInfo ti[kTInfo];
    uint32_t tmem;
    Stop stop;
};

// Walks over the groups of a grouped product in a warp's registers, 32 groups at a time (a lane a group).  The offsets are
// made harmless on the way: within [0, M] and not decreasing, whatever the array holds.
template <int kRows>
struct Groups {
    int g0 = -32, prev = 0, end = 0;  // first group held, first row behind them, tiles up to there
    int first = 0, last = 0, tiles = 0, upto = 0;  // of the lane's group: rows [first, last), tiles, tiles up to its last

    __device__ __forceinline__ void next(const Product& p, int lane) {
        if (g0 < 0) prev = min(max(p.offsets[0], 0), (int)p.M);
        g0 += 32;
        const int g = g0 + lane;
        last = min(max(g < p.groups ? p.offsets[g + 1] : 0, prev), (int)p.M);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, last, d);
            if (lane >= d) last = max(last, u);
        }
        first = __shfl_up_sync(0xffffffffu, last, 1);
        if (lane == 0) first = prev;
        tiles = g < p.groups ? (last - first + kRows - 1) / kRows : 0;
        upto = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += u;
        }
        upto += end;
        prev = __shfl_sync(0xffffffffu, last, 31);
        end = __shfl_sync(0xffffffffu, upto, 31);
    }
    // Row tile mt (not below an earlier one): its group and rows; false behind the last.
    __device__ __forceinline__ bool find(const Product& p, int lane, int64_t mt, int& g, int64_t& row0, int64_t& rows) {
        while (mt >= end) {
            if (g0 + 32 >= p.groups) return false;
            next(p, lane);
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, upto > mt)) - 1;
        g = g0 + at;
        row0 = __shfl_sync(0xffffffffu, first, at) + (mt - __shfl_sync(0xffffffffu, upto - tiles, at)) * kRows;
        rows = __shfl_sync(0xffffffffu, last, at);
        return true;
    }
};

// A box of the staging buffer: 32 rows of 128 bytes, 16-byte chunk c of row r at chunk c ^ (r & 7) (the 128-byte
// swizzle of the copy engine, and no bank conflict).  The thread that owns row r writes it from its accumulators ...
__device__ __forceinline__ void stage_row(uint8_t* box, int r, const float2* acc, __nv_bfloat16) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(box + r * 128 + ((i ^ (r & 7)) << 4)) =
            make_uint4(bf16x2(acc[4 * i].x, acc[4 * i].y), bf16x2(acc[4 * i + 1].x, acc[4 * i + 1].y),
                       bf16x2(acc[4 * i + 2].x, acc[4 * i + 2].y), bf16x2(acc[4 * i + 3].x, acc[4 * i + 3].y));
}
__device__ __forceinline__ void stage_row(uint8_t* box, int r, const float2* acc, float) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(box + r * 128 + ((i ^ (r & 7)) << 4)) =
            make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
}

// ... and where the copy engine may not write it (rows behind the tile's that belong to another group, rows of y that
// are not whole 16 bytes) the warp does: 16 bytes a lane, or element by element.
template <class T>
__device__ __forceinline__ void store_box(const uint8_t* box, T* y, int64_t ldy, int nr, int col, int N, bool wide, int lane) {
    if (wide) {  // N is whole 16 bytes too
        const int c = lane & 7, at = col + c * (16 / (int)sizeof(T));
        if (at >= N) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (r < nr)
                *reinterpret_cast<uint4*>(y + r * ldy + at) = *reinterpret_cast<const uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4));
        }
        return;
    }
    constexpr int kCols = 128 / (int)sizeof(T);
    for (int c = lane; c < kCols; c += 32) {
        if (col + c >= N) break;
        const int byte = c * (int)sizeof(T);
        for (int r = 0; r < nr; ++r)
            y[r * ldy + col + c] = *reinterpret_cast<const T*>(box + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
    }
}

template <int C, int H, class T>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
               const __grid_constant__ CUtensorMap ymap, const bool wide, const Product p)
{
    using Sm = Smem<C, H>;
    constexpr bool kPair = C == 2;
    constexpr int kRows = C * kBlk, S = Sm::kStages;
    constexpr int kBuf = H * kBlk, kBufs = kTmemCols / kBuf;  // a block's product, and how many of them TMEM holds
    constexpr int kCols = H * 64;                             // columns that a promotion thread owns
    constexpr int kIssuers = H > C ? 1 : 2;
    extern __shared__ uint8_t smem_raw[];
    Sm* sm = reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kPair ? (int)cluster_rank() : 0;
    const int KB = (p.K + kBlk - 1) / kBlk, nb = (p.N + kBlk - 1) / kBlk, ntiles = (nb + H - 1) / H;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sm->accf[i], 1 + p.waits.missing(2, C - 1));
            mbar_init(&sm->acce[i], C * kPromoWarps + p.waits.missing(1, 0));
        }
        for (int i = 0; i < kTInfo; ++i) {
            mbar_init(&sm->tfull[i], 1);
            mbar_init(&sm->tempty[i], kIssuers + kPromoWarps);
        }
        sm->stop.init(p.waits);
        async::fence_barrier_init();
    }
    if (warp == 1) {
        if (kPair) tmem_alloc_pair(&sm->tmem, kTmemCols);
        else tc5::tmem_alloc(&sm->tmem, kTmemCols);
        tc5::before_sync();
    }
    __syncthreads();
    if (kPair) {  // the barriers of both CTAs exist before either is signalled
        cluster_arrive();
        cluster_wait();
    }
    tc5::after_sync();
    dep_wait();
    dep_launch();  // not before this CTA has its TMEM: a dependent that waits for this grid may take the rest
    const uint32_t tmem = sm->tmem;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0) {
            const int64_t total = (p.M + kRows - 1) / kRows * ntiles;  // of a dense product
            Groups<kRows> groups;
            int sc = 0, tc = 0;
            bool ok = true;
            for (int64_t L = blockIdx.x / C; ok; L += gridDim.x / C, ++tc) {
                const int b = tc % kTInfo;
                if (tc >= kTInfo && !warp_wait(&sm->tempty[b], (tc / kTInfo - 1) & 1, &sm->stop, p.waits.err, 1)) break;
                TileInfo& ti = sm->ti[b];
                // column tiles innermost: the CTAs that run together share activation tiles in L2
                const int64_t mt = L / ntiles;
                const int nt = (int)(L - mt * ntiles);
                int g = 0;
                int64_t row0 = mt * kRows, rows = p.M;
                if (!kPair && p.groups ? !groups.find(p, lane, mt, g, row0, rows) : L >= total) {  // (groups go to single CTAs)
                    if (lane == 0) {
                        ti.end = 1;
                        mbar_arrive(&sm->tfull[b]);
                    }
                    break;
                }
                const int n0 = nt * H * kBlk;
                // CTA 1 of a pair may have no rows: then it loads none, and its half of the product is not used
                const bool second = row0 + kBlk < rows;
                row0 += rank * kBlk;
                const int nr = (int)min((int64_t)kBlk, max(rows - row0, (int64_t)0));
                if (lane == 0) {
                    ti.end = 0;
                    ti.nr = nr;
                    ti.n0 = n0;
                    ti.sw0 = (g * nb + nt * H) * KB;
                    ti.row0 = row0;
                    mbar_arrive(&sm->tfull[b]);
                }
                const int w0 = g * p.N + n0 + rank * kBlk;
                const uint32_t tx = kPair ? (second ? 4 : 3) * kTileBytes : kTileBytes + Sm::kWeights;
                for (int kb = 0; kb < KB; ++kb, ++sc) {
                    const int s = sc % S;
                    if (sc >= S && !warp_wait(&sm->empty[s], (sc / S - 1) & 1, &sm->stop, p.waits.err, 2)) {
                        ok = false;
                        break;
                    }
                    if (elect()) {
                        if (kPair) {
                            const uint32_t bar = peer_addr(&sm->full[s], 0);
                            if (rank == 0) mbar_expect_tx(&sm->full[s], tx);
                            if (nr > 0) tma_load_2d_pair(sm->ring[s], &amap, kb * kBlk, (int)row0, bar);
                            tma_load_2d_pair(sm->ring[s] + kTileBytes, &wmap, kb * kBlk, w0, bar);
                        } else {
                            mbar_expect_tx(&sm->full[s], tx);
                            tc5::tma_load_2d(sm->ring[s], &amap, kb * kBlk, (int)row0, &sm->full[s]);
#pragma unroll
                            for (int h = 0; h < H; ++h)
                                tc5::tma_load_2d(sm->ring[s] + (1 + h) * kTileBytes, &wmap, kb * kBlk, w0 + h * kBlk, &sm->full[s]);
                        }
                    }
                    __syncwarp();
                }
            }
            // every copy has landed before the CTA may exit; CTA 0's barriers count those of both
            if (rank == 0)
                for (int i = max(sc - S, 0); i < sc; ++i) wait_drain(&sm->full[i % S], (i / S) & 1);
        } else if (warp <= kIssuers) {
            // Two warps issue in turn, a block of K each: its MMAs run for 515 clocks (a pair) or 288, but what one warp
            // does for it (two waits, four MMAs, two commits) takes about 600.  (The MMAs of a single CTA's wide tile wait
            // for shared memory longer than that: one warp.)  A warp walks together and one lane issues: in a
            // branch of one lane the same loop takes half as long again.  Each warp keeps to its own buffers and ring
            // stages, so that no phase of a barrier passes unseen.
            static_assert(S % kIssuers == 0 && kBufs % kIssuers == 0, "ownership");
            const uint64_t ring_desc = tc5::smem_desc_sw128(sm->ring[0]);
            int sc = 0, mine = warp - 1, tc = 0, last = -1;  // blocks of K so far, this warp's next; its last buffer
            bool ok = true;
            while (ok) {
                const int b = tc % kTInfo;
                if (!warp_wait(&sm->tfull[b], (tc / kTInfo) & 1, &sm->stop, p.waits.err, 3)) break;
                const int end = sm->ti[b].end;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->tempty[b]);
                ++tc;
                if (end) break;
                if (rank != 0) continue;  // CTA 0 issues for both
                sc += KB;
                for (; mine < sc && ok; mine += kIssuers) {
                    const int s = mine % S, d = mine % kBufs;
                    ok = warp_wait2(&sm->full[s], (mine / S) & 1, &sm->acce[d], (mine / kBufs) & 1, &sm->stop, p.waits.err, 4);
                    if (!ok) break;
                    tc5::after_sync();
                    const uint64_t ad = ring_desc + (uint64_t)(s * ((kTileBytes + Sm::kWeights) >> 4)), wd = ad + (kTileBytes >> 4);
                    const uint32_t dt = tmem + d * kBuf;
                    if (elect()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // 32 of K (32 bytes, 2 descriptor units) each
                            if (kPair) mma_e4m3_pair(dt, ad + 2 * k, wd + 2 * k, idesc_e4m3_pair(kBuf), k > 0);
                            else mma_e4m3(dt, ad + 2 * k, wd + 2 * k, idesc_e4m3(kBuf), k > 0);
                        }
                        if (kPair) {
                            commit_pair(&sm->accf[d]);
                            commit_pair(&sm->empty[s]);
                        } else {
                            tc5::commit(&sm->accf[d]);
                            tc5::commit(&sm->empty[s]);
                        }
                    }
                    __syncwarp();
                    last = mine;
                }
            }
            // every MMA has completed before TMEM is released, and the last commits have arrived before the CTA may exit
            if (last >= 0) {
                wait_drain(&sm->accf[last % kBufs], (last / kBufs) & 1);
                wait_drain(&sm->empty[last % S], (last / S) & 1);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        // warps 4..7 take the first half of the tile's columns and 8..11 the second
        const int quarter = warp & 3, set = (warp - 4) >> 2, half = H == 2 ? set : 0;
        const int row = quarter * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + set * kCols;
        const uint32_t acce = peer_addr(&sm->acce[0], 0);  // of the CTA that issues
        uint8_t* out = sm->out[warp - 4];
        if (lane == 0)
            for (int b = 0; b < kBufs; ++b) peer_arrive_read(acce + b * 8);
        int n = 0, tc = 0;
        // the next tile, and its first two blocks' scales on their way
        TileInfo ti;
        const float *sa, *sw;
        float a[2], w[2];
        const auto scales = [&](int i, int kb) {
            a[i] = sa[kb];
            w[i] = sw[kb];
        };
        const auto next = [&]() -> bool {
            const int tb = tc % kTInfo;
            if (!warp_wait(&sm->tfull[tb], (tc / kTInfo) & 1, &sm->stop, p.waits.err, 6)) return false;
            ti = sm->ti[tb];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->tempty[tb]);
            ++tc;
            if (ti.end) return false;
            sa = p.sa + min(ti.row0 + row, p.M - 1) * KB;  // rows past the tile's: not used
            // a half past the matrix (its columns are not used) takes the first one's scales
            sw = p.sw + ti.sw0 + (ti.n0 + half * kBlk < p.N ? half * KB : 0);
            scales(0, 0);
            scales(1, KB > 1 ? 1 : 0);
            return true;
        };
        bool more = next();
        while (more) {
            float2 acc[kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            uint32_t v[2][32];
            bool ok = warp_wait(&sm->accf[n % kBufs], (n / kBufs) & 1, &sm->stop, p.waits.err, 7);
            if (ok) {
                tc5::after_sync();
                tc5::tmem_ld32(tl + n % kBufs * kBuf, v[0]);
            }
            for (int kb = 0; kb < KB && ok; ++kb) {
                const float s = a[0] * w[0];
                a[0] = a[1];
                w[0] = w[1];
                if (kb + 2 < KB) scales(1, kb + 2);
                const int d = n % kBufs;
                ++n;
                uint64_t* const after = &sm->accf[n % kBufs];
                // 32 columns at a time, each load under the additions of the one before; a buffer goes back to the MMA
                // when its last load has landed
#pragma unroll
                for (int i = 0; i < kCols / 32; ++i) {
                    tc5::tmem_wait_ld(v[i & 1]);
                    if (i + 1 < kCols / 32) {
                        tc5::tmem_ld32(tl + d * kBuf + (i + 1) * 32, v[(i + 1) & 1]);
                    } else {
                        tc5::before_sync();
                        __syncwarp();
                        if (lane == 0) peer_arrive_read(acce + d * 8);
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float2& to = acc[i * 16 + c];
                        to.x = fmaf(__uint_as_float(v[i & 1][2 * c]), s, to.x);
                        to.y = fmaf(__uint_as_float(v[i & 1][2 * c + 1]), s, to.y);
                    }
                }
                if (kb + 1 < KB) {
                    ok = warp_wait(after, (n / kBufs) & 1, &sm->stop, p.waits.err, 8);
                    if (ok) {
                        tc5::after_sync();
                        tc5::tmem_ld32(tl + n % kBufs * kBuf, v[0]);
                    }
                }
            }
            if (!ok || __any_sync(0xffffffffu, sm->stop.is_set())) break;
            constexpr int kBox = 128 / (int)sizeof(T);           // columns of a box
            constexpr int kRound = Sm::kOut / (32 * 128);        // boxes staged at once
            const int64_t y0 = ti.row0 + quarter * 32;
            const int nr = min(ti.nr - quarter * 32, 32), n0 = ti.n0 + set * kCols;
            more = next();
            if (nr <= 0) continue;
            // a box whose rows are all the tile's, or behind the matrix, is left to the copy engine
            const bool engine = wide && (nr == 32 || y0 + nr == p.M);
#pragma unroll
            for (int b0 = 0; b0 < kCols / kBox; b0 += kRound) {
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int b = b0; b < b0 + kRound && b < kCols / kBox; ++b)
                    stage_row(out + (b - b0) * 32 * 128, lane, &acc[b * kBox / 2], T());
                fence_async_smem();
                __syncwarp();
#pragma unroll
                for (int b = b0; b < b0 + kRound && b < kCols / kBox; ++b) {
                    const int col = n0 + b * kBox;
                    if (!engine) store_box<T>(out + (b - b0) * 32 * 128, static_cast<T*>(p.y) + y0 * p.ldy, p.ldy, nr, col, p.N, wide, lane);
                    else if (lane == 0 && col < p.N) tma_store_2d(&ymap, out + (b - b0) * 32 * 128, col, (int)y0);
                }
                if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                __syncwarp();
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the writes are done, not only read
        __syncwarp();
    }
    tc5::before_sync();
    __syncthreads();
    if (kPair) {  // neither CTA leaves while the other may signal its barriers or the pair's MMAs read its operands
        // after a wait that gave up CTA 1 may have sent copies that CTA 0 did not, which no barrier tells of: they get about 1 ms
        if (rank != 0 && sm->stop.is_set()) {
            const long long t0 = async::clk();
            while (async::clk() - t0 < kLandClk) {
            }
            __syncwarp();
        }
        cluster_arrive();
        cluster_wait();
    }
    tc5::after_sync();
    if (warp == 1) {
        if (kPair) tmem_dealloc_pair(tmem, kTmemCols);
        else tc5::tmem_dealloc(tmem, kTmemCols);
    }
}

// -------------------------------------------------------------------- few rows

// A ring of 64 KB (an SM needs about 66 KB in flight) and the codes of 32 KB of activation rows, as many blocks of K as
// fit: less than half an SM's shared memory, so that the next launch of a chain gets ready beside this one.
constexpr int kRing = 4;
constexpr int kOperand = 32 * 1024;
constexpr int kSBufs = 4;                    // TMEM buffers

// Warps that encode the activation rows; the first four go on as the promotion warps.
template <int NT>
constexpr int quant_warps() {
    return NT == 16 ? 4 : NT == 32 ? 8 : 12;
}
template <int NT>
constexpr int small_threads() {
    return 64 + 32 * quant_warps<NT>();      // with a producer and an MMA warp
}

template <int NT>
struct SmallSmem {
    alignas(1024) uint8_t ring[kRing][kTileBytes];
    alignas(1024) uint8_t b[kOperand];       // [block][NT rows][128 bytes], swizzled; then the partial sums [NT][128]
    float sx[kOperand / (NT * kBlk)][NT];
    uint64_t full[kRing], empty[kRing], accf[kSBufs], acce[kSBufs], ready, drained;
    uint32_t tmem;
    Stop stop;
};

// Codes and scales of the activation rows of n blocks of K, those of this CTA from its i0-th on, into the operand buffer: 8
// lanes per (row, block), 16 values a lane.
template <int NT>
__device__ __forceinline__ void encode_rows(const Product& p, SmallSmem<NT>* sm, int rank, int C, int KB, int i0, int n, int pt) {
    constexpr int kBatch = NT == 16 ? 1 : 2;      // items in flight of 8 lanes
    constexpr int kStep = 4 * quant_warps<NT>();  // such groups of 8 lanes
    const int m = (int)p.M, l = pt & 7;
    const float inv = __fdividef(1.0f, (float)m);
    // (the four groups of a warp make the same turns: they meet in the shuffles)
    for (int jw = pt >> 5 << 2; jw < n * m; jw += kStep * kBatch) {
        const int j0 = jw + (pt >> 3 & 3);
        uint4 raw[kBatch][2] = {};
        float sc[kBatch];
        uint2 code[kBatch][2];
        int at[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (jw + kStep * u >= n * m) continue;
            const int j = min(j0 + kStep * u, n * m - 1);                 // the last one may be read by several
            const int r = (int)(((float)j + 0.5f) * inv), t = j - r * m;  // exact: j is below 2^12
            const int kb = rank + (i0 + r) * C;
            at[u] = r * NT + t;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = kb * kBlk + h * 64 + l * 8;
                if (col >= p.K) continue;
                if (p.x) {
                    raw[u][h] = *reinterpret_cast<const uint4*>(p.x + t * p.ldx + col);
                } else {
                    const uint2 q = *reinterpret_cast<const uint2*>(p.a + (int64_t)t * p.K + col);
                    raw[u][h].x = q.x;
                    raw[u][h].y = q.y;
                }
            }
            if (!p.x) sc[u] = p.sa[(int64_t)t * KB + kb];
        }
        if (p.x) {
            encode<kBatch>((n * m - jw + kStep - 1) / kStep, [&](int u) { return max(amax_bf16(raw[u][0]), amax_bf16(raw[u][1])); },
                           [&](int u, int h, float (&v)[8]) { unpack8(raw[u][h], v); }, sc, code);
        } else {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) code[u][h] = make_uint2(raw[u][h].x, raw[u][h].y);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (jw + kStep * u >= n * m) continue;
            if (l == 0) (&sm->sx[0][0])[at[u]] = sc[u];
            // 128-byte swizzle: 16-byte chunk c of row t lies at chunk c ^ (t & 7) (NT is a multiple of 8)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint2*>(sm->b + at[u] * kBlk + (((4 * h + (l >> 1)) ^ (at[u] & 7)) << 4) + (l & 1) * 8) = code[u][h];
        }
    }
    fence_async_smem();
    mbar_arrive(&sm->ready);
}

// NT: rows rounded up to 16, 32 or 64.  The cluster's CTA r takes the blocks kb = r, r + C, ...
template <int NT, class T>
__global__ void __launch_bounds__(small_threads<NT>(), NT == 64 ? 1 : 2)
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
            mbar_init(&sm->accf[i], 1 + p.waits.missing(2, C - 1));
            mbar_init(&sm->acce[i], 4 + p.waits.missing(1, 0));
        }
        mbar_init(&sm->ready, 32 * quant_warps<NT>());
        mbar_init(&sm->drained, 4);
        sm->stop.init(p.waits);
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
                if (i >= kRing && !wait(&sm->empty[s], (i / kRing - 1) & 1, &sm->stop, p.waits.err, 11)) break;
                mbar_expect_tx(&sm->full[s], kTileBytes);
                tc5::tma_load_2d(sm->ring[s], &wmap, (rank + i * C) * kBlk, nt * kBlk, &sm->full[s]);
            }
            for (int j = max(i - kRing, 0); j < i; ++j) wait_drain(&sm->full[j % kRing], (j / kRing) & 1);
        }
    } else if (warp == 1) {
        int i = 0;
        for (; i < mine; ++i) {
            const int s = i % kRing, d = i % kSBufs, r = i % kRound;
            if (r == 0 && !warp_wait(&sm->ready, (i / kRound) & 1, &sm->stop, p.waits.err, 12)) break;
            if (!warp_wait(&sm->full[s], (i / kRing) & 1, &sm->stop, p.waits.err, 13) ||
                !warp_wait(&sm->acce[d], (i / kSBufs) & 1, &sm->stop, p.waits.err, 14))
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
        if (i > 0) {  // the last commits have arrived
            wait_drain(&sm->accf[(i - 1) % kSBufs], ((i - 1) / kSBufs) & 1);
            wait_drain(&sm->empty[(i - 1) % kRing], ((i - 1) / kRing) & 1);
        }
    } else if (warp >= 6) {
        for (int i0 = 0; i0 < mine; i0 += kRound) {
            if (i0 > 0 && !warp_wait(&sm->drained, (i0 / kRound - 1) & 1, &sm->stop, p.waits.err, 18)) break;
            encode_rows<NT>(p, sm, rank, C, KB, i0, min(kRound, mine - i0), tid - 64);
        }
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
                if (!warp_wait(&sm->drained, (i0 / kRound - 1) & 1, &sm->stop, p.waits.err, 17)) break;
            }
            const int n = min(kRound, mine - i0);
            encode_rows<NT>(p, sm, rank, C, KB, i0, n, pt);
            if (!warp_wait(&sm->ready, (i0 / kRound) & 1, &sm->stop, p.waits.err, 15)) break;
            float ws = sw[(int64_t)i0 * C];
            bool ok = true;
            for (int r = 0; r < n; ++r) {
                const int i = i0 + r, d = i % kSBufs;
                const float w = ws;
                if (r + 1 < n) ws = sw[(int64_t)(i + 1) * C];
                if (!warp_wait(&sm->accf[d], (i / kSBufs) & 1, &sm->stop, p.waits.err, 16)) {
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
            if (nt * kBlk + row < p.N && !sm->stop.is_set()) {
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
        if (warp >= 2 && !sm->stop.is_set()) {
            // every C-th row is this CTA's: a warp a row, two rows and all the peers' sums in flight
            const int c4 = lane * 4, col = nt * kBlk + c4;
            for (int i0 = warp - 2; rank + C * i0 < m; i0 += 2 * quant_warps<NT>()) {
                float4 v[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = rank + C * (i0 + quant_warps<NT>() * u);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < C && t < m)
                            v[u][c] = peer_load4(peer_addr(reinterpret_cast<const float*>(sm->b) + t * kBlk + c4, (uint32_t)c));
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = rank + C * (i0 + quant_warps<NT>() * u);
                    if (t >= m) continue;
                    float4 sum = v[u][0];
#pragma unroll
                    for (int c = 1; c < 8; ++c)
                        if (c < C) {
                            sum.x += v[u][c].x;
                            sum.y += v[u][c].y;
                            sum.z += v[u][c].z;
                            sum.w += v[u][c].w;
                        }
                    T* y = static_cast<T*>(p.y) + t * p.ldy + col;
                    if (col < p.N) y[0] = (T)sum.x;
                    if (col + 1 < p.N) y[1] = (T)sum.y;
                    if (col + 2 < p.N) y[2] = (T)sum.z;
                    if (col + 3 < p.N) y[3] = (T)sum.w;
                }
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

template <auto kKernel, class... A>
cudaError_t launch(unsigned grid, unsigned threads, size_t smem, int cluster, cudaStream_t st, A... args) {
    const cudaError_t e = allow_smem<kKernel>();
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
    return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

template <int C, int H>
cudaError_t launch_many(const Product& p, const CUtensorMap& am, const CUtensorMap& wm, int64_t tiles, cudaStream_t st) {
    // y for the copy engine, where it is laid out for it: it writes whole 16 bytes, past the last column too
    const int64_t es = p.y_bf16 ? 2 : 4;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.y) | (uintptr_t)(p.ldy * es) | (uintptr_t)(p.N * es)) & 15) == 0;
    CUtensorMap ym = {};
    if (wide) {
        const cudaError_t e = out_map(&ym, p.y, (uint64_t)p.N, (uint64_t)p.M, (uint64_t)(p.ldy * es), p.y_bf16);
        if (e != cudaSuccess) return e;
    }
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, sm_count() / C) * C;
    const size_t smem = sizeof(Smem<C, H>) + 1024;
    return p.y_bf16 ? launch<product_kernel<C, H, __nv_bfloat16>>(grid, kThreads, smem, C, st, am, wm, ym, wide, p)
                    : launch<product_kernel<C, H, float>>(grid, kThreads, smem, C, st, am, wm, ym, wide, p);
}

template <int NT>
cudaError_t launch_few(const Product& p, const CUtensorMap& wm, int C, cudaStream_t st) {
    const unsigned grid = (unsigned)(blocks_of(p.N) * C);
    const size_t smem = sizeof(SmallSmem<NT>) + 1024;
    return p.y_bf16 ? launch<product_small_kernel<NT, __nv_bfloat16>>(grid, small_threads<NT>(), smem, C, st, wm, p, C)
                    : launch<product_small_kernel<NT, float>>(grid, small_threads<NT>(), smem, C, st, wm, p, C);
}

}  // namespace

cudaError_t launch_product(const Product& p, cudaStream_t st) {
    CUtensorMap am, wm;
    const int64_t G = p.groups ? p.groups : 1;
    cudaError_t e = byte_map(&am, p.a, (uint64_t)p.K, (uint64_t)p.M, (uint64_t)p.K, kBlk);
    if (e != cudaSuccess) return e;
    // tiles at most: each group may end inside a tile of rows
    const auto row_tiles = [&](int64_t rows) {
        return p.groups ? std::min<int64_t>(p.M / rows + p.groups, p.M) : (p.M + rows - 1) / rows;
    };
    const int64_t nb = blocks_of(p.N), wide = (nb + 1) / 2, pairs = row_tiles(2 * kBlk) * wide, singles = row_tiles(kBlk) * wide;
    e = byte_map(&wm, p.w, (uint64_t)p.K, (uint64_t)(G * p.N), (uint64_t)p.K, kBlk);
    if (e != cudaSuccess) return e;
    // Dense rows go to pairs of CTAs where there are tiles for all of them (32768 x 2048 x 2048 with its quantisation: 175
    // us, 186 us with tiles of 128 x 256, 207 us with 128 x 128).  Groups fill 256 rows less often, and go to tiles of 128 x
    // 256 (8192 rows in 60 groups, 1024 x 1024: 23.7 us, 25.8 us with 128 x 128, and 30 us with pairs when those still
    // walked over groups; 32768 rows, 1536 x 1536: 105 and 119 us).  The number of their tiles is known as an upper bound
    // only, but from a few rows up the wide tiles are the better ones (256 rows: 17.1 and 18.9 us, 64 rows: 15.4 and 16.4 us,
    // 16 rows the same).  Where there are too few of either, tiles of 128 x 128, more of them (777 x 1000 x 784: 9.4 us, 12.5
    // us with 128 x 256 and 11.8 us with pairs; 512 x 2048 x 2048: 10.5 us and 14.2 us with either).  K does not enter, and
    // no tile's K is split: between the two, at 1200 to 2048 x 2048 x 2048, the smaller tiles are up to 7 % behind.
    if (nb > 1 && !p.groups && p.M > kBlk && 2 * pairs >= sm_count()) return launch_many<2, 2>(p, am, wm, pairs, st);
    if (nb > 1 && singles >= sm_count()) return launch_many<1, 2>(p, am, wm, singles, st);
    return launch_many<1, 1>(p, am, wm, row_tiles(kBlk) * nb, st);
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
