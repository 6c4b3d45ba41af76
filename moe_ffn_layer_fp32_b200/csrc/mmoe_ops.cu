// C entries of the stateless operators (declared in include/mmoe.h): the e4m3
// quantisers, products and MoE layer, and the block norm.
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "fp8.cuh"
#include "fp8_moe.cuh"
#include "mmoe_internal.cuh"
#include "norm.cuh"

using namespace mmoe;

namespace {

// What the kernels' bounded waits report to: one word of mapped host memory per device, allocated by
// the device's first call (also inside a stream capture) and kept until the process ends.
constexpr int kMaxDevices = 64;
std::mutex g_mu;
int* g_flag[kMaxDevices] = {};

std::atomic<long long> g_limit{f8::kWaitClk};  // mmoe_debug_fp8_waits
std::atomic<int> g_stall{0};

mmoe_status current_device(int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return report_cuda(e, "cudaGetDevice");
    if (*dev < 0 || *dev >= kMaxDevices) return report(MMOE_ERR_INVALID_ARG, "device %d: unsupported index", *dev);
    return MMOE_OK;
}

// Reports, once, a wait that gave up on the device (g_mu is held).
mmoe_status take_timeout(int dev) {
    const int site = g_flag[dev] ? __atomic_exchange_n(g_flag[dev], 0, __ATOMIC_ACQ_REL) : 0;
    return site ? report(MMOE_ERR_TIMEOUT, "a kernel of an earlier call gave up waiting (site %d)", site) : MMOE_OK;
}

// What the waits of the next launch on the current device are told.
mmoe_status device_waits(f8::Waits* w) {
    int dev = 0;
    const mmoe_status st = current_device(&dev);
    if (st != MMOE_OK) return st;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_flag[dev]) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        int* p = nullptr;
        cudaThreadExchangeStreamCaptureMode(&mode);
        const cudaError_t e = cudaHostAlloc(reinterpret_cast<void**>(&p), sizeof(int), cudaHostAllocMapped | cudaHostAllocPortable);
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) return report_cuda(e, "flag allocation");
        *p = 0;
        g_flag[dev] = p;  // device and host address are the same under unified addressing
    }
    const mmoe_status late = take_timeout(dev);
    if (late != MMOE_OK) return late;
    *w = f8::Waits{g_flag[dev], g_limit.load(), g_stall.exchange(0)};
    return MMOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// [a, a + n) and [b, b + m) share a byte
bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return n > 0 && m > 0 && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

mmoe_status check_type(int32_t t, const char* what) {
    if (t != MMOE_F32 && t != MMOE_BF16) return report(MMOE_ERR_INVALID_ARG, "%s=%d: must be MMOE_F32 or MMOE_BF16", what, t);
    return MMOE_OK;
}

int64_t size_of(int32_t t) { return t == MMOE_BF16 ? 2 : 4; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxDim = 1 << 20;
constexpr int64_t kMaxStride = int64_t(1) << 36;  // elements; the copy engine takes less than 2^40 bytes
constexpr int64_t kMaxSpan = int64_t(1) << 48;    // elements from the first row of a tensor to its last: more than an address space

mmoe_status check_dim(int64_t v, const char* what, int64_t step) {
    if (v < step || v > kMaxDim || v % step)
        return report(MMOE_ERR_INVALID_ARG, "%s=%lld: must be a multiple of %lld in [%lld, 2^20]", what, (long long)v,
                      (long long)step, (long long)step);
    return MMOE_OK;
}

mmoe_status check_rows(int64_t v, const char* what) {
    if (v < 0 || v > kMaxRows) return report(MMOE_ERR_INVALID_ARG, "%s=%lld: must be in [0, 2^31 - 256]", what, (long long)v);
    return MMOE_OK;
}

// So that (rows - 1) * ld, and the bytes computed from it, are far from 2^63.
mmoe_status check_span(int64_t rows, int64_t ld, const char* what) {
    if (ld > 0 && rows - 1 > kMaxSpan / ld)
        return report(MMOE_ERR_INVALID_ARG, "%lld rows %s=%lld elements apart span more than 2^48", (long long)rows, what, (long long)ld);
    return MMOE_OK;
}

#define CHECK(x)                               \
    do {                                       \
        const mmoe_status st_ = (x);           \
        if (st_ != MMOE_OK) return st_;        \
    } while (0)

// What the dense, the fused and the grouped product share.
mmoe_status check_product(int64_t M, const uint8_t* w, const float* sw, int64_t G, int64_t N, int64_t K, const void* y,
                          int32_t y_type, int64_t ldy) {
    CHECK(check_rows(M, "M"));
    CHECK(check_dim(N, "N", 1));
    CHECK(check_dim(K, "K", 16));
    CHECK(check_type(y_type, "y_type"));
    if (ldy < N || ldy > kMaxStride)
        return report(MMOE_ERR_INVALID_ARG, "ldy=%lld: must be at least N=%lld and at most 2^36", (long long)ldy, (long long)N);
    CHECK(check_span(M, ldy, "ldy"));
    if (G * N > kMaxRows || G * f8::blocks_of(N) * f8::blocks_of(K) > kMaxRows)
        return report(MMOE_ERR_INVALID_ARG, "the weights have too many rows or blocks");
    if (M == 0) return MMOE_OK;
    if (!w || !sw || !y) return report(MMOE_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned16(w)) return report(MMOE_ERR_INVALID_ARG, "the weight codes must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(y) % size_of(y_type) || reinterpret_cast<uintptr_t>(sw) % 4)
        return report(MMOE_ERR_INVALID_ARG, "y and the scales must be aligned to their elements");
    const int64_t yb = ((M - 1) * ldy + N) * size_of(y_type);
    if (overlap(y, yb, w, G * N * K) || overlap(y, yb, sw, G * f8::blocks_of(N) * f8::blocks_of(K) * 4))
        return report(MMOE_ERR_INVALID_ARG, "y overlaps the weights");
    return MMOE_OK;
}

mmoe_status check_codes(const uint8_t* a, const float* sa, int64_t M, int64_t K, const void* y, int64_t yb) {
    if (M == 0) return MMOE_OK;
    if (!a || !sa) return report(MMOE_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned16(a) || reinterpret_cast<uintptr_t>(sa) % 4)
        return report(MMOE_ERR_INVALID_ARG, "the codes must be 16-byte aligned, the scales 4-byte aligned");
    if (overlap(y, yb, a, M * K) || overlap(y, yb, sa, M * f8::blocks_of(K) * 4))
        return report(MMOE_ERR_INVALID_ARG, "y overlaps the codes or scales of a");
    return MMOE_OK;
}

// mmoe_linear_fp8's workspace: the scales, then the codes of x.
size_t scale_bytes(int64_t M, int64_t K) { return (size_t)(M * f8::blocks_of(K) * 4 + 15) / 16 * 16; }
size_t linear_workspace(int64_t M, int64_t K) { return M <= f8::kSmallRows ? 0 : scale_bytes(M, K) + (size_t)(M * K); }

mmoe_status check_fp8_config(const mmoe_config* c) {
    if (!c) return report(MMOE_ERR_INVALID_ARG, "config is NULL");
    if (c->d_model < 64 || c->d_model > 8192 || c->d_model % 32)
        return report(MMOE_ERR_INVALID_ARG, "d_model=%d: must be a multiple of 32 in [64, 8192]", c->d_model);
    if (c->n_experts < 1 || c->n_experts > kMaxExperts)
        return report(MMOE_ERR_INVALID_ARG, "n_experts=%d: must be in [1, %d]", c->n_experts, kMaxExperts);
    if (c->top_k < 1 || c->top_k > c->n_experts || c->top_k > kMaxTopK)
        return report(MMOE_ERR_INVALID_ARG, "top_k=%d: must be in [1, min(n_experts, %d)]", c->top_k, kMaxTopK);
    if (c->expert_hidden < 32 || c->expert_hidden > 4096 || c->expert_hidden % 32)
        return report(MMOE_ERR_INVALID_ARG, "expert_hidden=%d: must be a multiple of 32 in [32, 4096]", c->expert_hidden);
    if (c->shared_hidden < 32 || c->shared_hidden > 4096 || c->shared_hidden % 32)
        return report(MMOE_ERR_INVALID_ARG, "shared_hidden=%d: must be a multiple of 32 in [32, 4096]", c->shared_hidden);
    if (c->group_size != f8::kBlk) return report(MMOE_ERR_INVALID_ARG, "group_size=%d: must be 128", c->group_size);
    if (c->max_tokens < 1 || c->max_tokens > (1 << 20))
        return report(MMOE_ERR_INVALID_ARG, "max_tokens=%d: must be in [1, 2^20]", c->max_tokens);
    if (c->gating != MMOE_GATE_SOFTMAX && c->gating != MMOE_GATE_SIGMOID_TOPK_NORM &&
        c->gating != MMOE_GATE_SIGMOID_TOPK_NORM_SEL_BIAS)
        return report(MMOE_ERR_INVALID_ARG, "gating=%d: unknown", c->gating);
    if (c->has_router_bias != 0 && c->has_router_bias != 1)
        return report(MMOE_ERR_INVALID_ARG, "has_router_bias=%d: must be 0 or 1", c->has_router_bias);
    if (c->flags) return report(MMOE_ERR_INVALID_ARG, "flags=0x%x: must be 0", c->flags);
    return MMOE_OK;
}

mmoe_status check_tokens(const mmoe_config* c, int64_t T) {
    const int64_t most = c->max_tokens < f8::kFewTokens ? c->max_tokens : f8::kFewTokens;
    if (T < 0 || T > most) return report(MMOE_ERR_INVALID_ARG, "T=%lld: must be in [0, %lld]", (long long)T, (long long)most);
    return MMOE_OK;
}

f8::MoePlan moe_plan(const mmoe_config* c, int64_t T) {
    f8::MoePlan p = {};
    p.d = c->d_model;
    p.h = c->expert_hidden;
    p.hs = c->shared_hidden;
    p.E = c->n_experts;
    p.k = c->top_k;
    p.gating = c->gating;
    p.T = (int)T;
    return p;
}

}  // namespace

extern "C" {

mmoe_status mmoe_quantize_fp8_rows(const void* x, int32_t x_type, int64_t rows, int64_t K, int64_t ldx, uint8_t* q,
                                   float* s, void* stream) {
    CHECK(check_rows(rows, "rows"));
    CHECK(check_dim(K, "K", 8));
    CHECK(check_type(x_type, "x_type"));
    const int64_t es = size_of(x_type), kb = f8::blocks_of(K);
    if (ldx < K || ldx % (16 / es) || ldx > kMaxStride)
        return report(MMOE_ERR_INVALID_ARG, "ldx=%lld: must be at least K, at most 2^36 and whole 16 bytes", (long long)ldx);
    CHECK(check_span(rows, ldx, "ldx"));
    if (rows == 0) return MMOE_OK;
    if (rows * kb > (int64_t(1) << 36)) return report(MMOE_ERR_INVALID_ARG, "too many blocks");
    if (!x || !q || !s) return report(MMOE_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned16(x) || reinterpret_cast<uintptr_t>(q) % 8 || reinterpret_cast<uintptr_t>(s) % 4)
        return report(MMOE_ERR_INVALID_ARG, "x must be 16-byte, q 8-byte and s 4-byte aligned");
    const int64_t xb = ((rows - 1) * ldx + K) * es;
    if (overlap(x, xb, q, rows * K) || overlap(x, xb, s, rows * kb * 4) || overlap(q, rows * K, s, rows * kb * 4))
        return report(MMOE_ERR_INVALID_ARG, "x, q and s must not overlap");
    const cudaError_t e = f8::launch_quantize_rows(x, x_type == MMOE_BF16, rows, K, ldx, q, s, (cudaStream_t)stream);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "quantise rows launch");
}

mmoe_status mmoe_quantize_fp8_blocks(const void* w, int32_t w_type, int64_t batch, int64_t N, int64_t K, uint8_t* q,
                                     float* s, void* stream) {
    CHECK(check_rows(batch, "batch"));
    CHECK(check_dim(N, "N", 1));
    CHECK(check_dim(K, "K", 8));
    CHECK(check_type(w_type, "w_type"));
    if (batch == 0) return MMOE_OK;
    const int64_t es = size_of(w_type), nblk = batch * f8::blocks_of(N) * f8::blocks_of(K);
    if (nblk > kMaxRows) return report(MMOE_ERR_INVALID_ARG, "too many blocks");
    const int64_t n = batch * N * K;
    if (!w || !q || !s) return report(MMOE_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned16(w) || reinterpret_cast<uintptr_t>(q) % 8 || reinterpret_cast<uintptr_t>(s) % 4)
        return report(MMOE_ERR_INVALID_ARG, "w must be 16-byte, q 8-byte and s 4-byte aligned");
    if (overlap(w, n * es, q, n) || overlap(w, n * es, s, nblk * 4) || overlap(q, n, s, nblk * 4))
        return report(MMOE_ERR_INVALID_ARG, "w, q and s must not overlap");
    const cudaError_t e = f8::launch_quantize_blocks(w, w_type == MMOE_BF16, batch, N, K, q, s, (cudaStream_t)stream);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "quantise blocks launch");
}

mmoe_status mmoe_gemm_fp8(const uint8_t* a, const float* sa, int64_t M, const uint8_t* w, const float* sw, int64_t N,
                          int64_t K, void* y, int32_t y_type, int64_t ldy, void* stream) {
    CHECK(check_product(M, w, sw, 1, N, K, y, y_type, ldy));
    CHECK(check_codes(a, sa, M, K, y, ((M - 1) * ldy + N) * size_of(y_type)));
    if (M == 0) return MMOE_OK;
    f8::Product p = {a, sa, nullptr, 0, w, sw, M, (int)N, (int)K, 0, nullptr, y, y_type == MMOE_BF16, ldy, {}};
    CHECK(device_waits(&p.waits));
    const cudaError_t e = M <= f8::kSmallRows ? f8::launch_product_small(p, (cudaStream_t)stream)
                                              : f8::launch_product(p, (cudaStream_t)stream);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "product launch");
}

mmoe_status mmoe_gemm_fp8_grouped(const uint8_t* a, const float* sa, int64_t M, const int32_t* offsets, int64_t groups,
                                  const uint8_t* w, const float* sw, int64_t N, int64_t K, void* y, int32_t y_type,
                                  int64_t ldy, void* stream) {
    if (groups < 1 || groups > f8::kMaxGroups)
        return report(MMOE_ERR_INVALID_ARG, "groups=%lld: must be in [1, %d]", (long long)groups, f8::kMaxGroups);
    CHECK(check_product(M, w, sw, groups, N, K, y, y_type, ldy));
    CHECK(check_codes(a, sa, M, K, y, ((M - 1) * ldy + N) * size_of(y_type)));
    if (M == 0) return MMOE_OK;
    if (!offsets || reinterpret_cast<uintptr_t>(offsets) % 4)
        return report(MMOE_ERR_INVALID_ARG, "offsets is NULL or misaligned");
    if (overlap(y, ((M - 1) * ldy + N) * size_of(y_type), offsets, 4 * (groups + 1)))
        return report(MMOE_ERR_INVALID_ARG, "y overlaps the offsets");
    f8::Product p = {a, sa, nullptr, 0, w, sw, M, (int)N, (int)K, (int)groups, offsets, y, y_type == MMOE_BF16, ldy,
                     {}};
    CHECK(device_waits(&p.waits));
    const cudaError_t e = f8::launch_product(p, (cudaStream_t)stream);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "grouped product launch");
}

mmoe_status mmoe_linear_fp8_workspace(int64_t M, int64_t K, size_t* bytes) {
    if (!bytes) return report(MMOE_ERR_INVALID_ARG, "bytes is NULL");
    CHECK(check_rows(M, "M"));
    CHECK(check_dim(K, "K", 16));
    *bytes = linear_workspace(M, K);
    return MMOE_OK;
}

mmoe_status mmoe_linear_fp8(const uint16_t* x_bf16, int64_t M, int64_t ldx, const uint8_t* w, const float* sw, int64_t N,
                            int64_t K, void* y, int32_t y_type, int64_t ldy, void* workspace, size_t workspace_bytes,
                            void* stream) {
    CHECK(check_product(M, w, sw, 1, N, K, y, y_type, ldy));
    if (ldx < K || ldx % 8 || ldx > kMaxStride)
        return report(MMOE_ERR_INVALID_ARG, "ldx=%lld: must be at least K, at most 2^36 and a multiple of 8", (long long)ldx);
    CHECK(check_span(M, ldx, "ldx"));
    if (M == 0) return MMOE_OK;
    if (!x_bf16 || !aligned16(x_bf16)) return report(MMOE_ERR_INVALID_ARG, "x is NULL or not 16-byte aligned");
    const int64_t xb = ((M - 1) * ldx + K) * 2, yb = ((M - 1) * ldy + N) * size_of(y_type);
    if (overlap(x_bf16, xb, y, yb)) return report(MMOE_ERR_INVALID_ARG, "x and y overlap");
    f8::Product p = {nullptr, nullptr, reinterpret_cast<const __nv_bfloat16*>(x_bf16), ldx, w, sw, M, (int)N, (int)K, 0,
                     nullptr, y, y_type == MMOE_BF16, ldy, {}};
    const cudaStream_t st = (cudaStream_t)stream;
    if (M <= f8::kSmallRows) {
        CHECK(device_waits(&p.waits));
        const cudaError_t e = f8::launch_product_small(p, st);
        return e == cudaSuccess ? MMOE_OK : report_cuda(e, "linear launch");
    }
    const size_t need = linear_workspace(M, K);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need)
        return report(MMOE_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and %zu bytes long", need);
    if (overlap(workspace, (int64_t)need, y, yb) || overlap(workspace, (int64_t)need, x_bf16, xb) ||
        overlap(workspace, (int64_t)need, w, N * K) ||
        overlap(workspace, (int64_t)need, sw, f8::blocks_of(N) * f8::blocks_of(K) * 4))
        return report(MMOE_ERR_INVALID_ARG, "the workspace overlaps x, y, the weights or their scales");
    CHECK(device_waits(&p.waits));
    float* s = static_cast<float*>(workspace);
    uint8_t* q = static_cast<uint8_t*>(workspace) + scale_bytes(M, K);
    cudaError_t e = f8::launch_quantize_rows(x_bf16, true, M, K, ldx, q, s, st);
    p.a = q;
    p.sa = s;
    p.x = nullptr;
    if (e == cudaSuccess) e = f8::launch_product(p, st);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "linear launch");
}

mmoe_status mmoe_fp8_workspace(const mmoe_config* cfg, int64_t T, size_t* bytes) {
    if (!bytes) return report(MMOE_ERR_INVALID_ARG, "bytes is NULL");
    CHECK(check_fp8_config(cfg));
    CHECK(check_tokens(cfg, T));
    f8::MoePlan p = moe_plan(cfg, T);
    *bytes = T ? f8::carve_moe(p, nullptr) : 0;
    return MMOE_OK;
}

mmoe_status mmoe_forward_fp8(const mmoe_config* cfg, const mmoe_fp8_weights* w, const uint16_t* x_bf16, int64_t T, void* y,
                             int32_t y_type, int32_t* topk_idx, float* topk_gate, int32_t* expert_counts,
                             void* workspace, size_t workspace_bytes, void* stream) {
    CHECK(check_fp8_config(cfg));
    CHECK(check_tokens(cfg, T));
    CHECK(check_type(y_type, "y_type"));
    if (!w) return report(MMOE_ERR_INVALID_ARG, "weights is NULL");
    f8::MoePlan p = moe_plan(cfg, T);
    const int64_t d = p.d, h = p.h, hs = p.hs, E = p.E, k = p.k, db = f8::blocks_of(d), hb = f8::blocks_of(h), sb = f8::blocks_of(hs);
    const struct { const void* p; int64_t bytes; bool codes; } in[] = {
        {w->w_router, 4 * d * E, false}, {w->w_gate_up, E * 2 * h * d, true}, {w->s_gate_up, 4 * E * 2 * hb * db, false},
        {w->w_down, E * d * h, true}, {w->s_down, 4 * E * db * hb, false}, {w->w_shared_gate_up, 2 * hs * d, true},
        {w->s_shared_gate_up, 4 * 2 * sb * db, false}, {w->w_shared_down, d * hs, true}, {w->s_shared_down, 4 * db * sb, false}};
    for (const auto& t : in) {
        if (!t.p) return report(MMOE_ERR_INVALID_ARG, "a weight pointer is NULL");
        if (t.codes ? !aligned16(t.p) : reinterpret_cast<uintptr_t>(t.p) % 4 != 0)
            return report(MMOE_ERR_INVALID_ARG, "weight codes must be 16-byte, other weights 4-byte aligned");
    }
    if (cfg->has_router_bias && !w->router_bias)
        return report(MMOE_ERR_INVALID_ARG, "the config has a router bias but router_bias is NULL");
    if (reinterpret_cast<uintptr_t>(w->router_bias) % 4) return report(MMOE_ERR_INVALID_ARG, "router_bias must be 4-byte aligned");
    if (T == 0) return MMOE_OK;
    if (!x_bf16 || !y) return report(MMOE_ERR_INVALID_ARG, "x or y is NULL");
    if (!aligned16(x_bf16) || reinterpret_cast<uintptr_t>(y) % size_of(y_type))
        return report(MMOE_ERR_INVALID_ARG, "x must be 16-byte aligned, y aligned to its elements");
    for (const void* o : {(const void*)topk_idx, (const void*)topk_gate, (const void*)expert_counts})
        if (reinterpret_cast<uintptr_t>(o) % 4) return report(MMOE_ERR_INVALID_ARG, "optional outputs must be 4-byte aligned");
    const size_t need = f8::carve_moe(p, nullptr);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < need)
        return report(MMOE_ERR_INVALID_ARG, "the workspace must be 256-byte aligned and %zu bytes long", need);
    const struct { const void* p; int64_t bytes; } out[] = {
        {y, T * d * size_of(y_type)}, {topk_idx, topk_idx ? 4 * T * k : 0}, {topk_gate, topk_gate ? 4 * T * k : 0},
        {expert_counts, expert_counts ? 4 * (E + 1) : 0}, {workspace, (int64_t)need}};
    for (int i = 0; i < 5; ++i) {
        bool bad = overlap(out[i].p, out[i].bytes, x_bf16, T * d * 2) ||
                   (cfg->has_router_bias && overlap(out[i].p, out[i].bytes, w->router_bias, 4 * E));
        for (const auto& t : in) bad = bad || overlap(out[i].p, out[i].bytes, t.p, t.bytes);
        for (int j = 0; j < i; ++j) bad = bad || overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes);
        if (bad) return report(MMOE_ERR_INVALID_ARG, "an output or the workspace overlaps another buffer");
    }
    CHECK(device_waits(&p.waits));
    f8::carve_moe(p, static_cast<unsigned char*>(workspace));
    p.w_router = w->w_router;
    p.router_bias = cfg->has_router_bias ? w->router_bias : nullptr;
    p.gate_up = w->w_gate_up;
    p.s_gate_up = w->s_gate_up;
    p.down = w->w_down;
    p.s_down = w->s_down;
    p.sh_gate_up = w->w_shared_gate_up;
    p.sh_s_gate_up = w->s_shared_gate_up;
    p.sh_down = w->w_shared_down;
    p.sh_s_down = w->s_shared_down;
    p.x = reinterpret_cast<const __nv_bfloat16*>(x_bf16);
    p.y = y;
    p.y_bf16 = y_type == MMOE_BF16;
    p.out_idx = topk_idx;
    p.out_gate = topk_gate;
    p.out_counts = expert_counts;
    const cudaError_t e = f8::launch_moe_few(p, (cudaStream_t)stream);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "MoE layer launch");
}

mmoe_status mmoe_fp8_status(void) {
    int dev = 0;
    CHECK(current_device(&dev));
    std::lock_guard<std::mutex> lock(g_mu);
    return take_timeout(dev);
}

mmoe_status mmoe_debug_fp8_waits(int64_t clocks, int32_t stall_next) {
    if (clocks < 0) return report(MMOE_ERR_INVALID_ARG, "clocks=%lld: must be >= 0", (long long)clocks);
    if (stall_next < 0 || stall_next > 2) return report(MMOE_ERR_INVALID_ARG, "stall_next=%d: must be 0, 1 or 2", stall_next);
    g_limit.store(clocks ? clocks : f8::kWaitClk);
    g_stall.store(stall_next);
    return MMOE_OK;
}

mmoe_status mmoe_block_norm(const mmoe_norm* n, void* stream) {
    if (!n) return report(MMOE_ERR_INVALID_ARG, "arguments are NULL");
    CHECK(check_rows(n->rows, "rows"));
    if (n->d < 8 || n->d > kNormMaxDim || n->d % 8)
        return report(MMOE_ERR_INVALID_ARG, "d=%d: must be a multiple of 8 in [8, %d]", n->d, kNormMaxDim);
    CHECK(check_type(n->r_type, "r_type"));
    CHECK(check_type(n->y_type, "y_type"));
    if (!(n->eps >= 0.0f)) return report(MMOE_ERR_INVALID_ARG, "eps must not be negative or NaN");
    if (n->rows == 0) return MMOE_OK;
    const int64_t rows = n->rows, d = n->d, rs = size_of(n->r_type), ys = size_of(n->y_type), kb = f8::blocks_of(d);
    if (!n->r) return report(MMOE_ERR_INVALID_ARG, "r is NULL");
    if (!n->y && (n->w_post || n->gate)) return report(MMOE_ERR_INVALID_ARG, "w_post and gate need y");
    if ((n->x || n->xq || n->sx) && !n->w_pre) return report(MMOE_ERR_INVALID_ARG, "x, xq and sx need w_pre");
    if (n->w_pre && !n->x && !n->xq) return report(MMOE_ERR_INVALID_ARG, "w_pre needs x or xq");
    if (!n->xq != !n->sx) return report(MMOE_ERR_INVALID_ARG, "xq and sx are given together");
    if (!n->r_out && !n->w_pre) return report(MMOE_ERR_INVALID_ARG, "no output");
    const struct { const void* p; int64_t ld, size; const char* name; } strided[] = {
        {n->r, n->ldr, rs, "r"}, {n->y, n->ldy, ys, "y"}, {n->r_out, n->ldo, rs, "r_out"}};
    for (const auto& t : strided) {
        if (!t.p) continue;
        if (t.ld < d || t.ld % (16 / t.size) || t.ld > kMaxStride || !aligned16(t.p))
            return report(MMOE_ERR_INVALID_ARG, "%s must be 16-byte aligned with rows of at least d elements and whole 16 bytes apart", t.name);
        CHECK(check_span(rows, t.ld, t.name));
    }
    if (n->gate && (n->gate_col != 0 && n->gate_col != 1))
        return report(MMOE_ERR_INVALID_ARG, "gate_col=%d: must be 0 or 1", n->gate_col);
    if (n->gate && (n->gate_row < 0 || n->gate_row > kMaxStride))
        return report(MMOE_ERR_INVALID_ARG, "gate_row must be in [0, 2^36]");
    if (n->gate) CHECK(check_span(rows, n->gate_row, "gate_row"));
    if (n->gate && (n->gate_col ? (!aligned16(n->gate) || n->gate_row % 4) : reinterpret_cast<uintptr_t>(n->gate) % 4 != 0))
        return report(MMOE_ERR_INVALID_ARG, "gate: a gate per feature needs 16-byte aligned rows, one per row 4-byte ones");
    for (const void* p : {(const void*)n->w_post, (const void*)n->w_pre, (const void*)n->x, (const void*)n->xq})
        if (p && !aligned16(p)) return report(MMOE_ERR_INVALID_ARG, "w_post, w_pre, x and xq must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(n->sx) % 4) return report(MMOE_ERR_INVALID_ARG, "sx must be 4-byte aligned");
    // every output apart from every other buffer, but r_out may be r itself
    const struct { const void* p; int64_t bytes; } in[] = {
        {n->r, ((rows - 1) * n->ldr + d) * rs}, {n->y, n->y ? ((rows - 1) * n->ldy + d) * ys : 0}, {n->w_post, n->w_post ? 4 * d : 0},
        {n->w_pre, n->w_pre ? 4 * d : 0}, {n->gate, n->gate ? 4 * ((rows - 1) * n->gate_row + (n->gate_col ? d : 1)) : 0}};
    const struct { const void* p; int64_t bytes; } out[] = {
        {n->r_out, n->r_out ? ((rows - 1) * n->ldo + d) * rs : 0}, {n->x, n->x ? 2 * rows * d : 0}, {n->xq, n->xq ? rows * d : 0},
        {n->sx, n->sx ? 4 * rows * kb : 0}};
    const bool in_place = n->r_out == n->r && n->ldo == n->ldr;
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (!(i == 0 && j == 0 && in_place) && overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return report(MMOE_ERR_INVALID_ARG, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return report(MMOE_ERR_INVALID_ARG, "two outputs overlap");
    }
    const NormPlan p = {rows, n->d, n->r, n->ldr, n->r_type == MMOE_BF16, n->y, n->ldy, n->y_type == MMOE_BF16, n->w_post,
                        n->gate, n->gate_row, n->gate_col, n->residual_scale, n->eps, n->r_out, n->ldo, n->w_pre, n->x,
                        n->xq, n->sx};
    const cudaError_t e = launch_block_norm(p, (cudaStream_t)stream);
    return e == cudaSuccess ? MMOE_OK : report_cuda(e, "block norm launch");
}

}  // extern "C"
