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
// moe_experts_kernel: a cluster of S CTAs takes one expert and up to 16 of its
// tokens (the tensor cores' smallest N).  Weights are the MMA's M: a tile is
// 128 weight rows x 128 of K, 16 KB, one or two of them in each step of a
// ring that runs from the first gate row to the last down row without a stop.
//   gate/up: the CTA owns 1/S of the hidden features, over all of K.  A tile
//     holds for each of the four TMEM lane quarters 16 gate rows and the 16 up
//     rows of the same features, so SwiGLU needs one shuffle.
//   exchange: once every peer has signalled its part, each CTA reads all hidden
//     features of its tokens through distributed shared memory and quantises
//     them for itself (a cluster barrier would also wait for the two warps that
//     keep the ring running).
//   down: the CTA owns 1/S of the output rows, over all hidden features.
// Each (token, expert) row goes to the workspace; of the k + 1 clusters that
// a token takes part in, the last one (per rank: it owns the same output rows
// in every cluster) adds the rows in the order of the formula.  No cluster
// waits for another one, and no sum depends on the order of arrival.
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
constexpr int kRouteThreads = 256;
constexpr int kRouteParts = kRouteThreads / 64;  // K parts within a CTA

// ------------------------------------------------------------------ router

__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads) moe_route_kernel(const MoePlan p)
{
    extern __shared__ float route_smem[];          // x slice [8][ks]
    __shared__ float red[kRouteParts][kRouteCluster][kMaxExperts];
    __shared__ float part[kRouteCluster][kMaxExperts];
    const int tid = threadIdx.x, rank = (int)cluster_rank();
    const int t0 = (blockIdx.x / kRouteCluster) * kRouteCluster;
    const int nt = min(kRouteCluster, p.T - t0);
    // the dependent kernel may read weights before it waits for this one: it starts only once
    // everything before this kernel has completed
    dep_wait();
    dep_launch();
    const int ks = 32 * ((p.d / 32 + kRouteCluster - 1) / kRouteCluster);
    const int k0 = min(rank * ks, p.d), n = min(ks, p.d - k0);
    for (int i = tid; i < nt * (n / 8); i += kRouteThreads) {
        const int t = i / (n / 8), c = (i - t * (n / 8)) * 8;
        float v[8];
        load8(p.x + (int64_t)(t0 + t) * p.d + k0 + c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) route_smem[t * ks + c + j] = v[j];
    }
    for (int i = tid; i < (kRouteCluster - nt) * ks; i += kRouteThreads) route_smem[nt * ks + i] = 0.0f;
    // codes and scales of token t0 + rank, and its counters
    const int mt = t0 + rank;
    const int KB = (p.d + kBlk - 1) / kBlk;
    if (rank < nt) {
        const int hl = tid & 15;
        for (int b0 = 0; b0 < KB; b0 += kRouteThreads / 16) {
            const int b = b0 + (tid >> 4), c = b * kBlk + hl * 8;
            float v[8] = {};
            if (b < KB && c < p.d) load8(p.x + (int64_t)mt * p.d + c, v);
            const float s = scale_of(half_warp_max(amax8(v)));
            if (b < KB && c < p.d)
                *reinterpret_cast<uint2*>(p.xq + (int64_t)mt * p.d + c) = Coder(s)(v);
            if (b < KB && hl == 0) p.sx[mt * KB + b] = s;
        }
        if (tid < 16) p.arrived[mt * 16 + tid] = 0;
    }
    __syncthreads();
    // thread: expert tid % 64, K part tid / 64
    const int e = tid & 63, kp = tid >> 6;
    float acc[kRouteCluster] = {};
    if (e < p.E) {
        const float* w = p.w_router + (int64_t)k0 * p.E + e;
#pragma unroll 8
        for (int k = kp; k < n; k += kRouteParts) {
            const float wv = w[(int64_t)k * p.E];
#pragma unroll
            for (int t = 0; t < kRouteCluster; ++t) acc[t] = fmaf(route_smem[t * ks + k], wv, acc[t]);
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
        gate_topk_warp(g, p.router_bias, mt, l0, l1, tid, p.idx, p.gate, nullptr);
        __syncwarp();
        if (tid < p.k) {
            if (p.out_idx) p.out_idx[mt * p.k + tid] = p.idx[mt * p.k + tid];
            if (p.out_gate) p.out_gate[mt * p.k + tid] = p.gate[mt * p.k + tid];
        }
    }
    // the partial logits stay until every CTA has read them
    cluster_arrive();
    cluster_wait();
}

// ----------------------------------------------------------------- experts

constexpr int kN = 16;                 // tokens of a cluster
constexpr int kThreads = 192;          // producer, MMA, four promotion warps
constexpr int kSlot = kBlk * kBlk;     // a ring slot: 16 KB
constexpr int kMinRing = 2, kMaxRing = 12;
constexpr int kBufs = 8;               // TMEM buffers of 16 columns
constexpr int kTmemCols = kBufs * kN;
constexpr int kUnit = 16;              // hidden features of a lane quarter

// Dynamic shared memory: ring | operand codes (x, then the hidden features) | own hidden features
// [16][features of a rank] | scales of x | scales of the hidden features.
struct Layout {
    int ring;        // slots
    int operand;     // byte offsets
    int hidden, hidden_ld;
    int sx, sh;
    int bytes;
};

struct ExpertShared {
    uint64_t full[kMaxRing], empty[kMaxRing], accf[kBufs], acce[kBufs], xready, hready, pbar, peers;
    uint32_t tmem;
    int abort;
    int count[kMaxExperts];
    int expert, first, n;    // the cluster's expert (E: shared; -1: none), its first token in the expert's list, tokens
    int list[kN];            // slot t * k + j (shared: T * k + t)
    int token[kN];
    int last[kN];
};

__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 16-byte chunk c of operand row t lies at chunk c ^ (t & 7) (128-byte swizzle).
__device__ __forceinline__ uint8_t* operand_at(uint8_t* base, int kb, int t, int byte) {
    return base + (kb * kN + t) * kBlk + (((byte >> 4) ^ (t & 7)) << 4) + (byte & 15);
}

// Thread pt (of 128) of one TMEM tile: adds the 16 columns of its row, scaled.
__device__ __forceinline__ void add_scaled(float2 (&acc)[kN / 2], const uint32_t (&v)[kN], const float* s, float w) {
#pragma unroll
    for (int c = 0; c < kN / 2; ++c) {
        const float2 s2 = *reinterpret_cast<const float2*>(s + 2 * c);
        acc[c] = __ffma2_rn(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])),
                            make_float2(s2.x * w, s2.y * w), acc[c]);
    }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

// The cluster's expert, tokens and slots (every CTA for itself).
__device__ __forceinline__ void find_work(const MoePlan& p, ExpertShared* sm, int work, int tid) {
    const int chunks_sh = (p.T + kN - 1) / kN;
    if (work < chunks_sh) {  // the shared expert first: the longest clusters
        if (tid < kN) {
            sm->token[tid] = work * kN + tid;
            sm->list[tid] = p.T * p.k + work * kN + tid;
        }
        if (tid == 0) {
            sm->expert = p.E;
            sm->n = min(kN, p.T - work * kN);
        }
    }
    const bool counts = p.out_counts && blockIdx.x == 0;
    if (work < chunks_sh && !counts) {
        __syncthreads();
        return;
    }
    const int S = p.T * p.k;
    for (int i = tid; i < S; i += kThreads) atomicAdd(&sm->count[p.idx[i]], 1);
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
                const bool hit = i < S && p.idx[i] == e;
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
            mbar_init(&sm->accf[i], 1);
            mbar_init(&sm->acce[i], 4);
        }
        mbar_init(&sm->xready, 128);
        mbar_init(&sm->hready, 128);
        mbar_init(&sm->pbar, 4);
        mbar_init(&sm->peers, S * 4);
        sm->abort = 0;
        async::fence_barrier_init();
    }
    if (tid < kMaxExperts) sm->count[tid] = 0;
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
    const bool is_shared = expert == p.E;
    const int n = sm->n, d = p.d, H = is_shared ? p.hs : p.h;
    const int KBd = (d + kBlk - 1) / kBlk, KBh = (H + kBlk - 1) / kBlk;
    // this rank's hidden features (units of 16) and output rows (units of 32)
    const int u0 = H / kUnit * rank / S, u1 = H / kUnit * (rank + 1) / S;
    const int o0 = d / 32 * rank / S, o1 = d / 32 * (rank + 1) / S;
    const int gt = (u1 - u0 + 3) / 4, dt = (o1 - o0 + 3) / 4;  // gate/up and down tiles
    const int ngu = gt * KBd, steps = ngu + dt * KBh;

    if (warp == 0) {
        if (lane == 0) {
            const CUtensorMap* gm = is_shared ? &sgu_map : &gu_map;
            const CUtensorMap* dm = is_shared ? &sdn_map : &dn_map;
            const int grow = is_shared ? 0 : expert * 2 * H, drow = is_shared ? 0 : expert * d;
            int i = 0;
            for (; i < steps; ++i) {
                const int s = i % lay.ring;
                if (i >= lay.ring && !wait(&sm->empty[s], (i / lay.ring - 1) & 1, &sm->abort, p.err, 21)) break;
                uint8_t* slot = base + s * kSlot;
                if (i < ngu) {
                    const int t = i / KBd, kb = i - t * KBd, nu = min(4, u1 - u0 - 4 * t);
                    mbar_expect_tx(&sm->full[s], (uint32_t)(nu * 2 * kUnit * kBlk));
                    for (int q = 0; q < nu; ++q) {
                        const int f = (u0 + 4 * t + q) * kUnit;
                        tc5::tma_load_2d(slot + q * 2 * kUnit * kBlk, gm, kb * kBlk, grow + f, &sm->full[s]);
                        tc5::tma_load_2d(slot + (q * 2 + 1) * kUnit * kBlk, gm, kb * kBlk, grow + H + f, &sm->full[s]);
                    }
                } else {
                    const int j = i - ngu, t = j / KBh, kb = j - t * KBh, nu = min(4, o1 - o0 - 4 * t);
                    mbar_expect_tx(&sm->full[s], (uint32_t)(nu * 32 * kBlk));
                    for (int q = 0; q < nu; ++q)
                        tc5::tma_load_2d(slot + q * 32 * kBlk, dm, kb * kBlk, drow + (o0 + 4 * t + q) * 32, &sm->full[s]);
                }
            }
            for (int j = max(i - lay.ring, 0); j < i; ++j) wait_drain(&sm->full[j % lay.ring], (j / lay.ring) & 1);
        }
    } else if (warp == 1) {
        int i = 0;
        for (; i < steps; ++i) {
            const int s = i % lay.ring, b = i % kBufs;
            if ((i == 0 && gt > 0 && !warp_wait(&sm->xready, 0, &sm->abort, p.err, 22)) ||
                (i == ngu && !warp_wait(&sm->hready, 0, &sm->abort, p.err, 23)) ||
                !warp_wait(&sm->full[s], (i / lay.ring) & 1, &sm->abort, p.err, 24) ||
                !warp_wait(&sm->acce[b], (i / kBufs) & 1, &sm->abort, p.err, 25))
                break;
            tc5::after_sync();
            const int kb = i < ngu ? i % KBd : (i - ngu) % KBh;
            const uint64_t wd = tc5::smem_desc_sw128(base + s * kSlot);
            const uint64_t bd = tc5::smem_desc_sw128(operand + kb * kN * kBlk);
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3(tmem + b * kN, wd + 2 * k, bd + 2 * k, idesc_e4m3(kN), k > 0);
                tc5::commit(&sm->empty[s]);
                tc5::commit(&sm->accf[b]);
            }
            __syncwarp();
        }
        if (i > 0) wait_drain(&sm->accf[(i - 1) % kBufs], ((i - 1) / kBufs) & 1);
    } else {
        const int pt = tid - 64, quarter = warp & 3, hl = pt & 15;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        if (lane == 0)
            for (int b = 0; b < kBufs; ++b) mbar_arrive(&sm->acce[b]);
        // the tokens' codes and scales; features past d are zeros
        for (int i = pt; i < n * KBd * 8; i += 128) {
            const int t = i / (KBd * 8), c = i - t * KBd * 8;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (c * 16 < d) v = *reinterpret_cast<const uint4*>(p.xq + (int64_t)sm->token[t] * d + c * 16);
            *reinterpret_cast<uint4*>(operand_at(operand, c >> 3, t, (c & 7) * 16)) = v;
        }
        for (int i = pt; i < n * KBd; i += 128) {
            const int t = i / KBd, kb = i - t * KBd;
            sx[kb * kN + t] = p.sx[sm->token[t] * KBd + kb];
        }
        fence_async_smem();
        mbar_arrive(&sm->xready);
        bool ok = warp_wait(&sm->xready, 0, &sm->abort, p.err, 26);
        int i = 0;
        // gate and up: a lane holds one weight row; lanes l and l + 16 the gate and up rows of a feature
        const float* sgu = is_shared ? p.sh_s_gate_up : p.s_gate_up + (int64_t)expert * 2 * KBh * KBd;
        for (int t = 0; t < gt && ok; ++t) {
            const int unit = u0 + 4 * t + quarter;
            const bool mine = unit < u1;
            const float* sw = sgu + (int64_t)((lane < 16 ? 0 : KBh) + (mine ? unit * kUnit / kBlk : 0)) * KBd;
            float2 acc[kN / 2];
#pragma unroll
            for (int c = 0; c < kN / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            float w = sw[0];
            for (int kb = 0; kb < KBd; ++kb, ++i) {
                const int b = i % kBufs;
                const float wc = w;
                if (kb + 1 < KBd) w = sw[kb + 1];
                ok = warp_wait(&sm->accf[b], (i / kBufs) & 1, &sm->abort, p.err, 27);
                if (!ok) break;
                tc5::after_sync();
                uint32_t v[kN];
                tc5::tmem_ld16(tl + b * kN, v);
                tc5::tmem_wait_ld(v);
                tc5::before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->acce[b]);
                add_scaled(acc, v, sx + kb * kN, wc);
            }
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
            if (lane == 0) ok = wait_cluster(&sm->peers, 0, &sm->abort, p.err, 32);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            wait_cluster(&sm->peers, 0, &sm->abort, p.err, 32);  // each lane's own acquire
        }
        if (dt > 0 && ok) {
            for (int j = pt >> 4; j < n * KBh; j += 8) {
                const int t = j / KBh, kb = j - t * KBh, f = kb * kBlk + hl * 8;
                float v[8] = {};
                if (f < H) {
                    // the rank that owns unit f / 16: the last one that starts at or before it
                    const int u = f / kUnit, r = (S * (u + 1) - 1) / (H / kUnit);
                    const uint32_t at = peer_addr(hidden + t * lay.hidden_ld + (f - H / kUnit * r / S * kUnit), (uint32_t)r);
                    const float4 a = peer_load4(at), b = peer_load4(at + 16);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                }
                uint32_t am = amax8(v);  // the half warps of a warp may part at the end of the loop
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffu << (threadIdx.x & 16), am, o));
                const float s = scale_of(am);
                *reinterpret_cast<uint2*>(operand_at(operand, kb, t, hl * 8)) = Coder(s)(v);
                if (hl == 0) sh[kb * kN + t] = s;
            }
        }
        fence_async_smem();
        mbar_arrive(&sm->hready);
        ok = warp_wait(&sm->hready, 0, &sm->abort, p.err, 28) && ok;
        const float* sdn = is_shared ? p.sh_s_down : p.s_down + (int64_t)expert * KBd * KBh;
        for (int t = 0; t < dt && ok; ++t) {
            const int og = o0 + 4 * t + quarter;
            const bool mine = og < o1;
            const float* sw = sdn + (int64_t)(mine ? og * 32 / kBlk : 0) * KBh;
            float2 acc[kN / 2];
#pragma unroll
            for (int c = 0; c < kN / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            float w = sw[0];
            for (int kb = 0; kb < KBh; ++kb, ++i) {
                const int b = i % kBufs;
                const float wc = w;
                if (kb + 1 < KBh) w = sw[kb + 1];
                ok = warp_wait(&sm->accf[b], (i / kBufs) & 1, &sm->abort, p.err, 29);
                if (!ok) break;
                tc5::after_sync();
                uint32_t v[kN];
                tc5::tmem_ld16(tl + b * kN, v);
                tc5::tmem_wait_ld(v);
                tc5::before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->acce[b]);
                add_scaled(acc, v, sh + kb * kN, wc);
            }
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
        if (lane == 0) mbar_arrive(&sm->pbar);
        ok = warp_wait(&sm->pbar, 0, &sm->abort, p.err, 30) && ok;
        if (ok && o1 > o0) {
            if (pt < n) sm->last[pt] = atomicAdd(&p.arrived[sm->token[pt] * 16 + rank], 1u) == (uint32_t)p.k;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->pbar);
            ok = warp_wait(&sm->pbar, 1, &sm->abort, p.err, 31);
            __threadfence();
            for (int j = 0; j < n && ok; ++j) {
                if (!sm->last[j]) continue;
                const int t = sm->token[j];
                const float* row = p.part + (int64_t)t * p.k * d;
                const float* gate = p.gate + t * p.k;
                const float* shr = p.part + ((int64_t)p.T * p.k + t) * d;
                for (int col = o0 * 32 + pt; col < o1 * 32; col += 128) {
                    float v[kMaxTopK];
#pragma unroll
                    for (int q = 0; q < kMaxTopK; ++q) v[q] = q < p.k ? __ldcg(row + (int64_t)q * d + col) : 0.0f;
                    float sum = __ldcg(shr + col);
#pragma unroll
                    for (int q = 0; q < kMaxTopK; ++q)
                        if (q < p.k) sum = fmaf(gate[q], v[q], sum);
                    if (p.y_bf16) static_cast<__nv_bfloat16*>(p.y)[(int64_t)t * d + col] = __float2bfloat16_rn(sum);
                    else static_cast<float*>(p.y)[(int64_t)t * d + col] = sum;
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

// Ring slots and offsets for a cluster of S; at least two CTAs an SM where that leaves four slots each.
Layout layout_for(const MoePlan& p, int S) {
    const int hm = std::max(p.h, p.hs), KBd = (int)blocks_of(p.d), KBh = (int)blocks_of(hm);
    Layout l = {};
    l.hidden_ld = (hm / kUnit + S - 1) / S * kUnit;
    const int operand = std::max(KBd, KBh) * kN * kBlk, hidden = kN * l.hidden_ld * 4;
    const int rest = operand + hidden + (KBd + KBh) * kN * 4;
    const int half = 113 * 1024 - 2048 - 1024, whole = 226 * 1024 - 2048 - 1024;  // less static shared memory and alignment
    const int room = (half - rest) / kSlot >= 4 ? half : whole;
    l.ring = std::min((room - rest) / kSlot, kMaxRing);
    l.operand = l.ring * kSlot;
    l.hidden = l.operand + operand;
    l.sx = l.hidden + hidden;
    l.sh = l.sx + KBd * kN * 4;
    l.bytes = l.sh + KBh * kN * 4;
    return l;
}

template <int S>
cudaError_t launch_experts(const MoePlan& p, const CUtensorMap* m, int clusters, cudaStream_t st) {
    const Layout l = layout_for(p, S);
    if (l.ring < kMinRing) return cudaErrorInvalidValue;
    auto kern = moe_experts_kernel<S>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, l.bytes + 1024);
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
    return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], p, l);
}

}  // namespace

size_t carve_moe(MoePlan& p, unsigned char* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char* q = base ? base + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return static_cast<void*>(q);
    };
    const size_t T = (size_t)p.T, k = (size_t)p.k, d = (size_t)p.d;
    p.idx = static_cast<int32_t*>(take(T * k * 4));
    p.gate = static_cast<float*>(take(T * k * 4));
    p.arrived = static_cast<uint32_t*>(take(T * 16 * 4));
    p.sx = static_cast<float*>(take(T * (size_t)blocks_of(p.d) * 4));
    p.xq = static_cast<uint8_t*>(take(T * d));
    p.part = static_cast<float*>(take(T * (k + 1) * d * 4));
    return off;
}

cudaError_t launch_moe_few(const MoePlan& p, cudaStream_t st) {
    CUtensorMap m[4];
    cudaError_t e = byte_map(&m[0], p.gate_up, (uint64_t)p.d, (uint64_t)p.E * 2 * p.h, (uint64_t)p.d, kUnit);
    if (e == cudaSuccess) e = byte_map(&m[1], p.down, (uint64_t)p.h, (uint64_t)p.E * p.d, (uint64_t)p.h, 32);
    if (e == cudaSuccess) e = byte_map(&m[2], p.sh_gate_up, (uint64_t)p.d, (uint64_t)2 * p.hs, (uint64_t)p.d, kUnit);
    if (e == cudaSuccess) e = byte_map(&m[3], p.sh_down, (uint64_t)p.hs, (uint64_t)p.d, (uint64_t)p.hs, 32);
    if (e != cudaSuccess) return e;
    const int ks = 32 * ((p.d / 32 + kRouteCluster - 1) / kRouteCluster);
    const size_t smem = (size_t)kRouteCluster * ks * 4;
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
    // clusters at most: the shared expert's chunks, an expert per slot, and a chunk more per 16 slots
    const int slots = p.T * p.k;
    const int clusters = (p.T + kN - 1) / kN + std::min(p.E, slots) + slots / kN;
    return launch_experts<8>(p, m, clusters, st);
}

}  // namespace f8
}  // namespace mmoe
