// The whole MoE layer on e4m3 weights for up to 64 tokens, in two launches.
//
//   y = FFN_s(x) + sum_j gate_j FFN_{idx_j}(x),  FFN(x) = down(Q(silu(gate Q(x)) * (up Q(x))))
//
// Q is the quantisation to e4m3 in blocks of 128 features.  The work is one
// pass over the weights of the experts that some token selects, so everything
// is arranged to keep that stream running on every SM.
//
// moe_route_kernel: a cluster of 8 CTAs takes 8 tokens.  Each CTA sums an
// eighth of the FP32 router products of all 8 tokens, then finishes one token:
// the eight partial logits through distributed shared memory in a fixed order,
// gating, top-k; it also quantises that token's x.
//
// moe_experts_kernel: a cluster of S CTAs takes one expert and up to 8 of its
// tokens (half of the tensor cores' smallest N: wider clusters are the last to end).  A shared expert wider than the routed
// ones is taken in parts of its hidden features, a cluster each, so that it is
// not what the others wait for.  Weights are the MMA's M: a tile is up to 128
// weight rows x 128 of K, one copy, one step of a ring that runs from the first
// gate row to the last down row without a stop.
//   gate/up: the CTA owns 1/S of the hidden features, over all of K.  A tile
//     holds for each of the four TMEM lane quarters 16 gate rows and the 16 up
//     rows of the same features, so SwiGLU needs one shuffle.
//   exchange: once every peer has signalled its part, each CTA reads all hidden
//     features of its tokens through distributed shared memory and quantises
//     them for itself (a cluster barrier would also wait for the warps that
//     keep the ring running).
//   down: the CTA owns 1/S of the output rows, over all hidden features.
// Each (token, expert) row goes to the workspace; of the clusters that a token
// takes part in, the last one (per rank: it owns the same output rows in every
// cluster) adds the rows in the order of the formula.  No cluster waits for
// another one, and no sum depends on the order of arrival.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "fp8.cuh"
#include "fp8_moe.cuh"
#include "mmoe_internal.cuh"

namespace mmoe {
namespace f8 {
namespace {

using async::mbar_arrive;
using async::mbar_expect_tx;
using async::mbar_init;

constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 512;
constexpr int kRouteParts = kRouteThreads / 64;  // K parts within a CTA
constexpr int kRouteAhead = 32;                  // router weights a thread has in flight

// ------------------------------------------------------------------ router

__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads) moe_route_kernel(const MoePlan p)
{
    extern __shared__ float route_smem[];          // x slice [ks][8]
    __shared__ float red[kRouteParts][kRouteCluster][kMaxExperts];
    __shared__ float part[kRouteCluster][kMaxExperts];
    __shared__ int32_t top_idx[kMaxTopK];
    __shared__ float top_gate[kMaxTopK];
    const int tid = threadIdx.x, rank = (int)cluster_rank();
    const int t0 = (blockIdx.x / kRouteCluster) * kRouteCluster;
    const int nt = min(kRouteCluster, p.T - t0);
    // the dependent kernel may read weights before it waits for this one: it starts only once
    // everything before this kernel has completed
    dep_wait();
    dep_launch();
    const int ks = 32 * ((p.d / 32 + kRouteCluster - 1) / kRouteCluster);
    const int k0 = min(rank * ks, p.d), n = min(ks, p.d - k0);
    // thread: expert tid % 64, K part tid / 64; the first weights set out before x is read
    const int e = tid & 63, kp = tid >> 6;
    const float* w = p.w_router + (int64_t)k0 * p.E + e;
    float wv[kRouteAhead];
#pragma unroll
    for (int i = 0; i < kRouteAhead; ++i) {
        const int k = kp + i * kRouteParts;
        wv[i] = e < p.E && k < n ? w[(int64_t)k * p.E] : 0.0f;
    }
    for (int i = tid; i < kRouteCluster * (n / 8); i += kRouteThreads) {
        const int t = i & (kRouteCluster - 1), c = i / kRouteCluster * 8;
        float v[8] = {};
        if (t < nt) load8(p.x + (int64_t)(t0 + t) * p.d + k0 + c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) route_smem[(c + j) * kRouteCluster + t] = v[j];
    }
    const int mt = t0 + rank;
    __syncthreads();
    float acc[kRouteCluster] = {};
    for (int i0 = 0; i0 < n; i0 += kRouteAhead * kRouteParts) {
        float cur[kRouteAhead];
#pragma unroll
        for (int i = 0; i < kRouteAhead; ++i) {
            cur[i] = wv[i];
            const int k = i0 + kp + (i + kRouteAhead) * kRouteParts;
            wv[i] = e < p.E && k < n ? w[(int64_t)k * p.E] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kRouteAhead; ++i) {
            const int k = i0 + kp + i * kRouteParts;
            if (k >= n) break;
            const float4 a = *reinterpret_cast<const float4*>(route_smem + k * kRouteCluster);
            const float4 b = *reinterpret_cast<const float4*>(route_smem + k * kRouteCluster + 4);
            acc[0] = fmaf(a.x, cur[i], acc[0]);
            acc[1] = fmaf(a.y, cur[i], acc[1]);
            acc[2] = fmaf(a.z, cur[i], acc[2]);
            acc[3] = fmaf(a.w, cur[i], acc[3]);
            acc[4] = fmaf(b.x, cur[i], acc[4]);
            acc[5] = fmaf(b.y, cur[i], acc[5]);
            acc[6] = fmaf(b.z, cur[i], acc[6]);
            acc[7] = fmaf(b.w, cur[i], acc[7]);
        }
    }
#pragma unroll
    for (int t = 0; t < kRouteCluster; ++t) red[kp][t][e] = acc[t];
    __syncthreads();
    for (int i = tid; i < kRouteCluster * kMaxExperts; i += kRouteThreads) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kRouteParts; ++q) s += red[q][i >> 6][i & 63];
        part[i >> 6][i & 63] = s;
    }
    cluster_arrive();
    cluster_wait();
    if (tid < 32 && rank < nt) {
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int r = 0; r < kRouteCluster; ++r) {
            l0 += peer_load(peer_addr(&part[rank][tid], (uint32_t)r));
            l1 += peer_load(peer_addr(&part[rank][tid + 32], (uint32_t)r));
        }
        Plan g{};
        g.E = p.E;
        g.k = p.k;
        g.gating = p.gating;
        g.router_bias = p.router_bias;
        l0 = tid < p.E ? biased_logit(g, l0, tid) : -INFINITY;
        l1 = tid + 32 < p.E ? biased_logit(g, l1, tid + 32) : -INFINITY;
        gate_topk_warp(g, p.router_bias, 0, l0, l1, tid, top_idx, top_gate, nullptr);
        __syncwarp();
        if (tid < p.k) {
            p.idx[mt * p.k + tid] = top_idx[tid];
            p.gate[mt * p.k + tid] = top_gate[tid];
            if (p.out_idx) p.out_idx[mt * p.k + tid] = top_idx[tid];
            if (p.out_gate) p.out_gate[mt * p.k + tid] = top_gate[tid];
        }
    } else if (rank < nt) {
        // beside the top-k, the other warps: codes and scales of token t0 + rank, and its counters
        constexpr int kHalfWarps = kRouteThreads / 16 - 2;
        const int KB = (p.d + kBlk - 1) / kBlk, hl = tid & 15;
        for (int b0 = 0; b0 < KB; b0 += kHalfWarps) {
            const int b = b0 + (tid >> 4) - 2, c = b * kBlk + hl * 8;
            float v[8] = {};
            if (b < KB && c < p.d) load8(p.x + (int64_t)mt * p.d + c, v);
            const float s = scale_of(half_warp_max(amax8(v)));
            if (b < KB && c < p.d) *reinterpret_cast<uint2*>(p.xq + (int64_t)mt * p.d + c) = Coder(s)(v);
            if (b < KB && hl == 0) p.sx[mt * KB + b] = s;
        }
        if (tid < 32 + kRanks) p.arrived[mt * kRanks + tid - 32] = 0;
    }
    // the partial logits stay until every CTA has read them
    cluster_arrive();
    cluster_wait();
}

// ----------------------------------------------------------------- experts

constexpr int kN = 8;                  // tokens of a cluster
constexpr int kCols = 16;              // the tokens' side of an MMA, its smallest: the other half is not used
constexpr int kThreads = 224;          // producer, MMA, four promotion warps, MMA: each MMA warp has every second slot and buffer
constexpr int kSlot = kBlk * kBlk;     // a ring slot: 16 KB
constexpr int kMaxRing = 12;           // at least 4, and even (below)
constexpr int kBufs = 8;               // TMEM buffers of 16 columns
constexpr int kTmemCols = kBufs * kCols;
constexpr int kUnit = 16;              // hidden features of a lane quarter
constexpr int kAlone = 16;             // (token, block) items that each CTA quantises for itself

// Dynamic shared memory: ring | operand codes (x, then the hidden features: 8 rows a block of 128; the MMA's other 8 rows
// are the next block's, or the 1 KB behind the last) | own hidden features [8][features of a rank] | scales of x | scales
// of the hidden features.
struct Layout {
    int ring;              // slots
    int nu[2], no;         // units of 16 features (routed, shared) and of 32 output rows in a tile
    int operand;           // byte offsets
    int hidden, hidden_ld;
    int sx, sh;
    int bytes;
};

struct ExpertShared {
    uint64_t full[kMaxRing], empty[kMaxRing], accf[kBufs], acce[kBufs], xready, hready, stored, counted, peers, codes;  // from xready on: one phase each
    uint32_t tmem;
    Stop stop;
    int count[kMaxExperts];
    uint8_t slot[kFewTokens * kMaxTopK];  // the expert of each (token, choice)
    int expert, first, n;    // the cluster's expert (E + i: part i of the shared one; -1: none), its first token in the expert's list, tokens
    int list[kN];            // slot t * k + j (shared: (k + part) * T + t)
    int token[kN];
    int last[kN];
};

__device__ __forceinline__ void peer_store8(uint32_t addr, uint2 v) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// 16-byte chunk c of operand row t lies at chunk c ^ (t & 7) (128-byte swizzle); `row` counts over all blocks.
__device__ __forceinline__ uint8_t* operand_at(uint8_t* base, int row, int byte) {
    return base + row * kBlk + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
}

// Thread pt (of 128) of one TMEM tile: adds the 8 columns of its row, scaled.
__device__ __forceinline__ void add_scaled(float2 (&acc)[kN / 2], const uint32_t (&v)[kN], const float* s, float w) {
#pragma unroll
    for (int c = 0; c < kN / 2; ++c) {
        const float2 s2 = *reinterpret_cast<const float2*>(s + 2 * c);
        acc[c] = __ffma2_rn(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])),
                            make_float2(s2.x * w, s2.y * w), acc[c]);
    }
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

__device__ __forceinline__ float2 first_two(const float* w, int KB) { return make_float2(w[0], w[KB > 1 ? 1 : 0]); }

// acc = the sum of KB blocks of the tile whose first step is i: w[kb] s[kb][column] times the step's buffer, w01 being
// first_two(w, KB), read ahead.  The next buffer's load runs under this one's additions.
__device__ __forceinline__ bool add_blocks(float2 (&acc)[kN / 2], ExpertShared* sm, uint32_t tl, int i, int KB, const float* w,
                                           float2 w01, const float* s, int* err, int site) {
#pragma unroll
    for (int c = 0; c < kN / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
    float w0 = w01.x, w1 = w01.y;
    uint32_t v[2][kN];
    if (!warp_wait(&sm->accf[i % kBufs], (i / kBufs) & 1, &sm->stop, err, site)) return false;
    tc5::after_sync();
    tmem_ld8(tl + i % kBufs * kCols, v[0]);
    for (int kb0 = 0; kb0 < KB; kb0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kb = kb0 + u;
            if (kb >= KB) break;
            tmem_wait_ld8(v[u]);
            tc5::before_sync();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(&sm->acce[(i + kb) % kBufs]);
            const float wc = w0;
            w0 = w1;
            if (kb + 2 < KB) w1 = w[kb + 2];
            if (kb + 1 < KB) {
                const int n = i + kb + 1;
                if (!warp_wait(&sm->accf[n % kBufs], (n / kBufs) & 1, &sm->stop, err, site)) return false;
                tc5::after_sync();
                tmem_ld8(tl + n % kBufs * kCols, v[u ^ 1]);
            }
            add_scaled(acc, v[u], s + kb * kN, wc);
        }
    }
    return true;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

// The cluster's expert, tokens and slots (every CTA for itself).
__device__ __forceinline__ void find_work(const MoePlan& p, ExpertShared* sm, int work, int tid) {
    const int chunks = (p.T + kN - 1) / kN, chunks_sh = chunks * p.parts;
    if (work < chunks_sh) {  // the shared expert first: the longest clusters
        const int part = work / chunks, first = (work - part * chunks) * kN;
        if (tid < kN) {
            sm->token[tid] = first + tid;
            sm->list[tid] = (p.k + part) * p.T + first + tid;
        }
        if (tid == 0) {
            sm->expert = p.E + part;
            sm->n = min(kN, p.T - first);
        }
    }
    const bool counts = p.out_counts && blockIdx.x == 0;
    if (work < chunks_sh && !counts) {
        __syncthreads();
        return;
    }
    const int S = p.T * p.k;
    if (S <= 32 && p.T <= kN && !counts) {
        // a lane a choice: cluster j takes the j-th expert in the order of their first choice (no more than kN tokens
        // have it)
        if (tid < 32) {
            const int e = tid < S ? p.idx[tid] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            unsigned firsts = __ballot_sync(0xffffffffu, e >= 0 && __ffs(same) - 1 == tid);
            for (int j = work - chunks_sh; j > 0 && firsts; --j) firsts &= firsts - 1;
            const int pick = __ffs(firsts) - 1;
            const int expert = __shfl_sync(0xffffffffu, e, max(pick, 0));
            const unsigned mine = __shfl_sync(0xffffffffu, same, max(pick, 0));
            if (pick >= 0 && (mine >> tid & 1)) {
                const int at = __popc(mine & ((1u << tid) - 1u));
                sm->list[at] = tid;
                sm->token[at] = tid / p.k;
            }
            if (tid == 0) {
                sm->expert = pick >= 0 ? expert : -1;
                sm->n = __popc(mine);
            }
        }
        __syncthreads();
        return;
    }
    for (int i = tid; i < S; i += kThreads) {
        const int e = p.idx[i];
        sm->slot[i] = (uint8_t)e;
        atomicAdd(&sm->count[e], 1);
    }
    __syncthreads();
    if (counts) {
        for (int e = tid; e < p.E; e += kThreads) p.out_counts[e] = sm->count[e];
        if (tid == 0) p.out_counts[p.E] = p.T;
    }
    if (work < chunks_sh) return;
    if (tid < 32) {
        const int c0 = tid < p.E ? (sm->count[tid] + kN - 1) / kN : 0;
        const int c1 = tid + 32 < p.E ? (sm->count[tid + 32] + kN - 1) / kN : 0;
        int s0 = c0, s1 = c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u0 = __shfl_up_sync(0xffffffffu, s0, o), u1 = __shfl_up_sync(0xffffffffu, s1, o);
            if (tid >= o) {
                s0 += u0;
                s1 += u1;
            }
        }
        s1 += __shfl_sync(0xffffffffu, s0, 31);
        const int j = work - chunks_sh;
        if (tid == 0) sm->expert = -1;
        __syncwarp();
        if (s0 - c0 <= j && j < s0) {
            sm->expert = tid;
            sm->first = (j - (s0 - c0)) * kN;
            sm->n = min(kN, sm->count[tid] - sm->first);
        }
        if (s1 - c1 <= j && j < s1) {
            sm->expert = tid + 32;
            sm->first = (j - (s1 - c1)) * kN;
            sm->n = min(kN, sm->count[tid + 32] - sm->first);
        }
        __syncwarp();
        const int e = sm->expert;
        if (e >= 0) {
            const int first = sm->first;
            int seen = 0;
            for (int i0 = 0; i0 < S && seen < first + kN; i0 += 32) {
                const int i = i0 + tid;
                const bool hit = i < S && sm->slot[i] == e;
                const unsigned m = __ballot_sync(0xffffffffu, hit);
                const int at = seen + __popc(m & ((1u << tid) - 1u)) - first;
                if (hit && at >= 0 && at < kN) {
                    sm->list[at] = i;
                    sm->token[at] = i / p.k;
                }
                seen += __popc(m);
            }
        }
    }
    __syncthreads();
}

template <int S>
__global__ void __launch_bounds__(kThreads)
moe_experts_kernel(const __grid_constant__ CUtensorMap gu_map, const __grid_constant__ CUtensorMap dn_map,
                   const __grid_constant__ CUtensorMap sgu_map, const __grid_constant__ CUtensorMap sdn_map,
                   const MoePlan p, const Layout lay)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ ExpertShared shared;
    ExpertShared* sm = &shared;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* operand = base + lay.operand;
    float* hidden = reinterpret_cast<float*>(base + lay.hidden);
    float* sx = reinterpret_cast<float*>(base + lay.sx);
    float* sh = reinterpret_cast<float*>(base + lay.sh);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), work = blockIdx.x / S;
    if (tid == 0) {
        for (int i = 0; i < lay.ring; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sm->accf[i], 1 + p.waits.missing(2, S - 1));
            mbar_init(&sm->acce[i], 4 + p.waits.missing(1, 0));
        }
        mbar_init(&sm->xready, 128);
        mbar_init(&sm->hready, 128);
        mbar_init(&sm->stored, 4);
        mbar_init(&sm->counted, 4);
        mbar_init(&sm->peers, S * 4);
        mbar_init(&sm->codes, S * 4);
        sm->stop.init(p.waits);
        async::fence_barrier_init();
    }
    if (tid < kMaxExperts) sm->count[tid] = 0;
    if (tid == 64) {
        prefetch_map(&gu_map);
        prefetch_map(&dn_map);
        prefetch_map(&sgu_map);
        prefetch_map(&sdn_map);
    }
    if (warp == 1) {
        tc5::tmem_alloc(&sm->tmem, kTmemCols);
        tc5::before_sync();
    }
    __syncthreads();
    tc5::after_sync();
    dep_launch();  // not before this CTA has its TMEM (a dependent that waits for this grid may take the rest)
    cluster_arrive();  // the peers' barriers exist before anyone signals them
    cluster_wait();
    const uint32_t tmem = sm->tmem;
    dep_wait();
    find_work(p, sm, work, tid);
    const int expert = sm->expert;
    if (expert < 0) {  // so for the whole cluster: nothing left to do
        if (warp == 1) tc5::tmem_dealloc(tmem, kTmemCols);
        return;
    }
    const bool is_shared = expert >= p.E;
    const int n = sm->n, d = p.d;
    const int part0 = is_shared ? (expert - p.E) * p.part_hidden : 0;  // first hidden feature
    const int H = is_shared ? min(p.part_hidden, p.hs - part0) : p.h;
    const int KBd = (d + kBlk - 1) / kBlk, KBh = (H + kBlk - 1) / kBlk;
    const int KBw = is_shared ? (p.hs + kBlk - 1) / kBlk : KBh;        // of the whole expert
    // this rank's hidden features (units of 16) and output rows (units of 32)
    const int u0 = H / kUnit * rank / S, u1 = H / kUnit * (rank + 1) / S;
    const int o0 = d / 32 * rank / S, o1 = d / 32 * (rank + 1) / S;
    const int nu = lay.nu[is_shared], no = lay.no;
    const int gt = (u1 - u0 + nu - 1) / nu, dt = (o1 - o0 + no - 1) / no;  // gate/up and down tiles
    const int ngu = gt * KBd, steps = ngu + dt * KBh;

    if (warp == 0) {
        const CUtensorMap* gm = is_shared ? &sgu_map : &gu_map;
        const CUtensorMap* dm = is_shared ? &sdn_map : &dn_map;
        const int e = is_shared ? 0 : expert, unit0 = part0 / kUnit + u0;
        int i = 0;
        for (int t = 0, kb = 0; i < steps; ++i) {
            const int s = i % lay.ring;
            if (i >= lay.ring && !warp_wait(&sm->empty[s], (i / lay.ring - 1) & 1, &sm->stop, p.waits.err, 21)) break;
            const bool down = i >= ngu;
            if (i == ngu) t = kb = 0;
            if (elect()) {
                // the rows of a last tile that are another rank's, or past the matrix, come along unused
                if (down) {
                    mbar_expect_tx(&sm->full[s], (uint32_t)(no * 32 * kBlk));
                    tma_load_3d(base + s * kSlot, dm, part0 + kb * kBlk, (o0 + t * no) * 32, e, &sm->full[s]);
                } else {
                    mbar_expect_tx(&sm->full[s], (uint32_t)(nu * 2 * kUnit * kBlk));
                    tma_load_5d(base + s * kSlot, gm, kb * kBlk, 0, 0, unit0 + t * nu, e, &sm->full[s]);
                }
            }
            __syncwarp();
            if (++kb == (down ? KBh : KBd)) {
                kb = 0;
                ++t;
            }
        }
        for (int j = max(i - lay.ring, 0); j < i; ++j) wait_drain(&sm->full[j % lay.ring], (j / lay.ring) & 1);
    } else if (warp == 1 || warp == 6) {
        int last = -1;
        for (int i = warp == 1 ? 0 : 1; i < steps; i += 2) {
            const int s = i % lay.ring, b = i % kBufs;
            if ((i < 2 && gt > 0 && !warp_wait(&sm->xready, 0, &sm->stop, p.waits.err, 22)) ||
                ((i == ngu || i == ngu + 1) && !warp_wait(&sm->hready, 0, &sm->stop, p.waits.err, 23)) ||
                !warp_wait2(&sm->full[s], (i / lay.ring) & 1, &sm->acce[b], (i / kBufs) & 1, &sm->stop, p.waits.err, 24))
                break;
            tc5::after_sync();
            const int kb = i < ngu ? i % KBd : (i - ngu) % KBh;
            const uint64_t wd = tc5::smem_desc_sw128(base + s * kSlot);
            const uint64_t bd = tc5::smem_desc_sw128(operand + kb * kN * kBlk);
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3(tmem + b * kCols, wd + 2 * k, bd + 2 * k, idesc_e4m3(kCols), k > 0);
                tc5::commit(&sm->empty[s]);
                tc5::commit(&sm->accf[b]);
            }
            __syncwarp();
            last = i;
        }
        if (last >= 0) {  // the last commits have arrived
            wait_drain(&sm->accf[last % kBufs], (last / kBufs) & 1);
            wait_drain(&sm->empty[last % lay.ring], (last / lay.ring) & 1);
        }
    } else {
        const int pt = tid - 64, quarter = warp & 3, hl = pt & 15;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        if (lane == 0)
            for (int b = 0; b < kBufs; ++b) mbar_arrive(&sm->acce[b]);
        // where this thread's weight scales lie, the first of them read before anything else
        const float* sgu = is_shared ? p.sh_s_gate_up + (int64_t)(part0 / kBlk) * KBd : p.s_gate_up + (int64_t)expert * 2 * KBh * KBd;
        const auto gate_up_scales = [&](int t) {
            const int unit = u0 + nu * t + quarter;
            const bool mine = quarter < nu && unit < u1;
            return sgu + (int64_t)((lane < 16 ? 0 : KBw) + (mine ? unit * kUnit / kBlk : 0)) * KBd;
        };
        const float* sdn = is_shared ? p.sh_s_down + part0 / kBlk : p.s_down + (int64_t)expert * KBd * KBh;
        const auto down_scales = [&](int t) {
            const int og = o0 + no * t + quarter;
            return sdn + (int64_t)(quarter < no && og < o1 ? og * 32 / kBlk : 0) * KBw;
        };
        float2 gate_up_w = first_two(gate_up_scales(0), KBd), down_w = first_two(down_scales(0), KBh);
        // the tokens' codes and scales; features past d are zeros
        if ((pt >> 3 & 7) < n) {
            const int t = pt >> 3 & 7, c = pt & 7;  // a 16-byte chunk of every second block of a token, eight in flight
            const uint8_t* from = p.xq + (int64_t)sm->token[t] * d + c * 16;
            for (int kb0 = pt >> 6; kb0 < KBd; kb0 += 16) {
                uint4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    v[u] = make_uint4(0u, 0u, 0u, 0u);
                    if ((kb0 + 2 * u) * kBlk + c * 16 < d) v[u] = *reinterpret_cast<const uint4*>(from + (kb0 + 2 * u) * kBlk);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (kb0 + 2 * u < KBd) *reinterpret_cast<uint4*>(operand_at(operand, (kb0 + 2 * u) * kN + t, c * 16)) = v[u];
            }
        }
        if ((pt & 7) < n) {
            const float* from = p.sx + sm->token[pt & 7] * KBd;
#pragma unroll 4
            for (int kb = pt >> 3; kb < KBd; kb += 16) sx[kb * kN + (pt & 7)] = from[kb];
        }
        fence_async_smem();
        mbar_arrive(&sm->xready);
        bool ok = warp_wait(&sm->xready, 0, &sm->stop, p.waits.err, 26);
        int i = 0;
        // gate and up: a lane holds one weight row; lanes l and l + 16 the gate and up rows of a feature
        for (int t = 0; t < gt && ok; ++t) {
            const int unit = u0 + nu * t + quarter;
            const bool mine = quarter < nu && unit < u1;
            float2 acc[kN / 2];
            const float2 w01 = gate_up_w;
            if (t + 1 < gt) gate_up_w = first_two(gate_up_scales(t + 1), KBd);
            ok = add_blocks(acc, sm, tl, i, KBd, gate_up_scales(t), w01, sx, p.waits.err, 27);
            i += KBd;
            if (!ok) break;
            // lanes below 16 finish the even tokens, the others the odd ones
            const int f = (unit - u0) * kUnit + (lane & 15);
#pragma unroll
            for (int c = 0; c < kN / 2; ++c) {
                const float got = __shfl_xor_sync(0xffffffffu, lane < 16 ? acc[c].y : acc[c].x, 16);
                const int tok = 2 * c + (lane >> 4);
                if (mine && tok < n)
                    hidden[tok * lay.hidden_ld + f] = lane < 16 ? silu_mul(acc[c].x, got) : silu_mul(got, acc[c].y);
            }
        }
        // this warp's hidden features are in place: tell every peer, then wait for all of theirs
        __syncwarp();
        if (lane < S) peer_arrive(peer_addr(&sm->peers, (uint32_t)lane));
        if (ok) {
            if (lane == 0) ok = wait_cluster(&sm->peers, 0, &sm->stop, p.waits.err, 32);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            wait_cluster(&sm->peers, 0, &sm->stop, p.waits.err, 32);  // each lane's own acquire
        }
        if (ok) {
            // A half warp per (token, block).  With few of them each CTA quantises all for itself; with more, 1 / S of
            // them for all, at the price of another signal (about 1 us): 128 items took 8.6 us alone and take 4.0 us
            // shared.  (Four at a time hide more of the peers' latency, but four times the code comes from L2: 2.9 us
            // for a single item instead of 1.3 us.)
            const int U = H / kUnit, items = n * KBh, stride = items > kAlone ? S : 1, first = items > kAlone ? rank : 0;
            const int own = (items - first + stride - 1) / stride;
            // (both half warps of a warp make the same turns: they meet in the shuffles)
#pragma unroll 1
            for (int jw = pt >> 5 << 1; jw < own; jw += 8) {
                const int j = first + stride * min(jw + (pt >> 4 & 1), own - 1);  // the last one may be done by both
                const int t = j / KBh, kb = j - t * KBh, f = kb * kBlk + hl * 8;
                float v[8] = {};
                if (f < H) {
                    // the rank that owns unit f / 16: the last one that starts at or before it
                    const int r = (S * (f / kUnit + 1) - 1) / U;
                    const uint32_t from = peer_addr(hidden + t * lay.hidden_ld + (f - U * r / S * kUnit), (uint32_t)r);
                    const float4 a = peer_load4(from), b = peer_load4(from + 16);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                }
                const float s = scale_of(half_warp_max(amax8(v)));
                const uint2 code = Coder(s)(v);
                uint8_t* to = operand_at(operand, kb * kN + t, hl * 8);
                float* st = sh + kb * kN + t;
                if (stride == 1) {
                    *reinterpret_cast<uint2*>(to) = code;
                    if (hl == 0) *st = s;
                } else {
                    for (int r = 0; r < S; ++r) peer_store8(peer_addr(to, (uint32_t)r), code);
                    if (hl < S) peer_store(peer_addr(st, (uint32_t)hl), s);
                }
            }
            if (stride != 1) {
                __syncwarp();
                if (lane < S) peer_arrive(peer_addr(&sm->codes, (uint32_t)lane));
                if (lane == 0) ok = wait_cluster(&sm->codes, 0, &sm->stop, p.waits.err, 33);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                wait_cluster(&sm->codes, 0, &sm->stop, p.waits.err, 33);  // each lane's own acquire
            }
        }
        fence_async_smem();
        mbar_arrive(&sm->hready);
        ok = warp_wait(&sm->hready, 0, &sm->stop, p.waits.err, 28) && ok;
        for (int t = 0; t < dt && ok; ++t) {
            const int og = o0 + no * t + quarter;
            const bool mine = quarter < no && og < o1;
            float2 acc[kN / 2];
            const float2 w01 = down_w;
            if (t + 1 < dt) down_w = first_two(down_scales(t + 1), KBh);
            ok = add_blocks(acc, sm, tl, i, KBh, down_scales(t), w01, sh, p.waits.err, 29);
            i += KBh;
            if (!ok || !mine) continue;
            const int col = og * 32 + lane;
#pragma unroll
            for (int c = 0; c < kN / 2; ++c) {
                if (2 * c < n) p.part[(int64_t)sm->list[2 * c] * d + col] = acc[c].x;
                if (2 * c + 1 < n) p.part[(int64_t)sm->list[2 * c + 1] * d + col] = acc[c].y;
            }
        }
        // a token's last contribution to this rank's output rows adds them all up
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->stored);
        ok = warp_wait(&sm->stored, 0, &sm->stop, p.waits.err, 30) && ok;
        if (ok && o1 > o0) {
            if (pt < n) sm->last[pt] = atomicAdd(&p.arrived[sm->token[pt] * kRanks + rank], 1u) == (uint32_t)(p.k + p.parts - 1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->counted);
        }
    }
    // every warp helps with these sums
    if (o1 > o0) {
        __syncwarp();
        if (warp_wait(&sm->counted, 0, &sm->stop, p.waits.err, 31)) {
            __threadfence();
            const int quads = (o1 - o0) * 8;  // four columns a thread
            const bool wide = (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
#pragma unroll 1
            for (int at = tid; at < n * quads; at += kThreads) {
                const int j = at / quads, col = o0 * 32 + (at - j * quads) * 4;
                if (!sm->last[j]) continue;
                const int t = sm->token[j];
                const float* row = p.part + (int64_t)t * p.k * d + col;
                const float* gate = p.gate + t * p.k;
                const float* shr = p.part + ((int64_t)p.T * p.k + t) * d + col;
                float4 v[kMaxTopK];
                float g[kMaxTopK];
#pragma unroll
                for (int q = 0; q < kMaxTopK; ++q)
                    if (q < p.k) {
                        v[q] = __ldcg(reinterpret_cast<const float4*>(row + (int64_t)q * d));
                        g[q] = gate[q];
                    }
                float4 sum = __ldcg(reinterpret_cast<const float4*>(shr));
                for (int q = 1; q < p.parts; ++q) {
                    const float4 more = __ldcg(reinterpret_cast<const float4*>(shr + (int64_t)q * p.T * d));
                    sum = make_float4(sum.x + more.x, sum.y + more.y, sum.z + more.z, sum.w + more.w);
                }
#pragma unroll
                for (int q = 0; q < kMaxTopK; ++q)
                    if (q < p.k)
                        sum = make_float4(fmaf(g[q], v[q].x, sum.x), fmaf(g[q], v[q].y, sum.y), fmaf(g[q], v[q].z, sum.z),
                                          fmaf(g[q], v[q].w, sum.w));
                const float o[4] = {sum.x, sum.y, sum.z, sum.w};
                const int64_t to = (int64_t)t * d + col;
                if (p.y_bf16) {
                    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + to;
                    if (wide) *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2(o[0], o[1]), bf16x2(o[2], o[3]));
                    else
                        for (int i = 0; i < 4; ++i) y[i] = __float2bfloat16_rn(o[i]);
                } else {
                    float* y = static_cast<float*>(p.y) + to;
                    if (wide) *reinterpret_cast<float4*>(y) = sum;
                    else
                        for (int i = 0; i < 4; ++i) y[i] = o[i];
                }
            }
        }
    }
    // no CTA leaves while a peer may still read its hidden features
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    tc5::before_sync();
    __syncthreads();
    tc5::after_sync();
    if (warp == 1) tc5::tmem_dealloc(tmem, kTmemCols);
}

// Of `all` units, dealt to S ranks: how many a tile takes (4 at most, none more than a rank needs).
constexpr int tile_units(int all, int S) {
    const int most = (all + S - 1) / S, tiles = (most + 3) / 4;
    return (most + tiles - 1) / tiles;
}

// Ring slots and offsets for a cluster of S.
constexpr Layout layout_for(const MoePlan& p, int S) {
    const int ph = std::min(p.part_hidden, p.hs), hm = std::max(p.h, ph), KBd = (int)blocks_of(p.d), KBh = (int)blocks_of(hm);
    Layout l = {};
    l.nu[0] = tile_units(p.h / kUnit, S);
    l.nu[1] = tile_units(ph / kUnit, S);
    l.no = tile_units(p.d / 32, S);
    l.hidden_ld = (hm / kUnit + S - 1) / S * kUnit;
    const int operand = std::max(KBd, KBh) * kN * kBlk + 1024, hidden = kN * l.hidden_ld * 4;
    const int rest = operand + hidden + (KBd + KBh) * kN * 4;
    // two CTAs an SM where that leaves four slots each; less static shared memory and alignment
    const int half = 113 * 1024 - 4096, whole = 226 * 1024 - 4096;
    const int room = (half - rest) / kSlot >= 4 ? half : whole;
    l.ring = std::min((room - rest) / kSlot, kMaxRing) & ~1;
    l.operand = l.ring * kSlot;
    l.hidden = l.operand + operand;
    l.sx = l.hidden + hidden;
    l.sh = l.sx + KBd * kN * 4;
    l.bytes = l.sh + KBh * kN * 4;
    return l;
}

// The largest layer that the entry takes leaves six slots; a smaller one takes less beside the ring.
constexpr MoePlan largest_plan() {
    MoePlan p = {};
    p.d = 8192;
    p.h = p.hs = p.part_hidden = 4096;
    return p;
}
static_assert(layout_for(largest_plan(), 4).ring == 6 && layout_for(largest_plan(), 8).ring >= 6, "ring slots");

// Gate and up rows: (k, row of a unit, gate or up, unit, expert), so that one copy brings a tile as the kernel wants it.
cudaError_t gate_up_map(CUtensorMap* m, const uint8_t* w, int d, int H, int E, int nu) {
    const uint64_t D = (uint64_t)d;
    const uint64_t dims[5] = {D, kUnit, 2, (uint64_t)(H / kUnit), (uint64_t)E};
    const uint64_t strides[4] = {D, (uint64_t)H * D, kUnit * D, 2 * (uint64_t)H * D};
    const uint32_t box[5] = {kBlk, kUnit, 2, (uint32_t)nu, 1};
    return byte_map_n(m, w, 5, dims, strides, box);
}
cudaError_t down_map(CUtensorMap* m, const uint8_t* w, int d, int H, int E, int no) {
    const uint64_t dims[3] = {(uint64_t)H, (uint64_t)d, (uint64_t)E};
    const uint64_t strides[2] = {(uint64_t)H, (uint64_t)d * (uint64_t)H};
    const uint32_t box[3] = {kBlk, (uint32_t)(32 * no), 1};
    return byte_map_n(m, w, 3, dims, strides, box);
}

template <int S>
cudaError_t launch_experts(const MoePlan& p, int clusters, cudaStream_t st) {
    static_assert(S <= kRanks, "one counter a rank");
    const Layout l = layout_for(p, S);
    CUtensorMap m[4];
    cudaError_t e = gate_up_map(&m[0], p.gate_up, p.d, p.h, p.E, l.nu[0]);
    if (e == cudaSuccess) e = down_map(&m[1], p.down, p.d, p.h, p.E, l.no);
    if (e == cudaSuccess) e = gate_up_map(&m[2], p.sh_gate_up, p.d, p.hs, 1, l.nu[1]);
    if (e == cudaSuccess) e = down_map(&m[3], p.sh_down, p.d, p.hs, 1, l.no);
    if (e != cudaSuccess) return e;
    e = allow_smem<moe_experts_kernel<S>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)l.bytes + 1024;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_experts_kernel<S>, m[0], m[1], m[2], m[3], p, l);
}

}  // namespace

size_t carve_moe(MoePlan& p, unsigned char* base) {
    // the shared expert in parts no wider than a routed one, of whole quantisation blocks
    p.part_hidden = (int)blocks_of(p.h) * kBlk;
    p.parts = (p.hs + p.part_hidden - 1) / p.part_hidden;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char* q = base ? base + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return static_cast<void*>(q);
    };
    const size_t T = (size_t)p.T, k = (size_t)p.k, d = (size_t)p.d;
    p.idx = static_cast<int32_t*>(take(T * k * 4));
    p.gate = static_cast<float*>(take(T * k * 4));
    p.arrived = static_cast<uint32_t*>(take(T * kRanks * 4));
    p.sx = static_cast<float*>(take(T * (size_t)blocks_of(p.d) * 4));
    p.xq = static_cast<uint8_t*>(take(T * d));
    p.part = static_cast<float*>(take(T * (k + (size_t)p.parts) * d * 4));
    return off;
}

cudaError_t launch_moe_few(const MoePlan& p, cudaStream_t st) {
    const int ks = 32 * ((p.d / 32 + kRouteCluster - 1) / kRouteCluster);
    const size_t smem = (size_t)kRouteCluster * ks * 4;
    cudaError_t e = allow_smem<moe_route_kernel>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.T + kRouteCluster - 1) / kRouteCluster * kRouteCluster));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, moe_route_kernel, p);
    if (e != cudaSuccess) return e;
    // clusters: the shared expert's chunks, an expert per slot, and at most a chunk more per 8 slots.  Of 8 CTAs where
    // all of them are on the GPU at once (two CTAs an SM), else of 4: a second round of CTAs starts with its latencies
    // (64 tokens of 2048 features: 104 us with 8, 81 us with 4).
    const int slots = p.T * p.k;
    const int busy = (p.T + kN - 1) / kN * p.parts + std::min(p.E, slots), clusters = busy + slots / kN;
    if (8 * busy <= 2 * sm_count()) return launch_experts<8>(p, clusters, st);
    return launch_experts<4>(p, clusters, st);
}

}  // namespace f8
}  // namespace mmoe
