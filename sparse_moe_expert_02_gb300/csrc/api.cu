// C ABI of libmoe: argument validation, workspace carving and the launch
// sequence of the routed-MoE layer.  Every entry point only enqueues work on
// the caller's stream; the only host synchronisation is in moe_check().
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <map>
#include <mutex>
#include <utility>

#include "common.cuh"
#include "internal.h"

namespace moe {
thread_local bool t_pdl = false;
static std::atomic<uint64_t> g_launches{0};
void count_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

namespace {
std::mutex g_setup_mu;
std::map<std::pair<const void*, int>, int> g_smem_set;  // (kernel, device) -> bytes allowed
std::map<std::pair<const void*, int>, int> g_values;    // (key, device) -> value
}  // namespace

cudaError_t ensure_smem_attr(const void* func, int bytes) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_setup_mu);
    int& cur = g_smem_set[{func, dev}];
    if (cur >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) cur = bytes;
    return e;
}

cudaError_t per_device_value(const void* key, const std::function<cudaError_t(int*)>& init, int* value) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_setup_mu);
    auto it = g_values.find({key, dev});
    if (it != g_values.end()) {
        *value = it->second;
        return cudaSuccess;
    }
    int v = 0;
    e = init(&v);
    if (e != cudaSuccess) return e;
    g_values[{key, dev}] = v;
    *value = v;
    return cudaSuccess;
}
}  // namespace moe

struct moe_plan {
    moe_config cfg;
    int device;
    int num_sms;
    int64_t spin_ns;
    // moe_forward runs the shared expert on a second stream, forked from and
    // joined back into the caller's stream with these events
    cudaStream_t side = nullptr;
    cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
    // split expert GEMMs: the permutation is done (the second stream starts
    // the single-CTA halves)
    cudaEvent_t ev_perm = nullptr;
};

namespace {

thread_local char g_detail[256];

moe_status cuda_fail(cudaError_t e, const char* where) {
    snprintf(g_detail, sizeof(g_detail), "%.160s: %s", where, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
moe_status arg_fail(moe_status s, const char* what) {
    snprintf(g_detail, sizeof(g_detail), "%s", what);
    return s;
}
#define MOE_CUDA(call)                                        \
    do {                                                      \
        cudaError_t e_ = (call);                              \
        if (e_ != cudaSuccess) return cuda_fail(e_, #call);   \
    } while (0)

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// bf16 layer: h as a bf16 hi/lo pair against the bf16 W_down (on request),
// else h as one fp16 against an fp16 copy of W_down.
bool hilo(const moe_config& c) { return c.dtype == MOE_BF16 && (c.flags & MOE_FLAG_DOWN_HILO); }
bool f16_down(const moe_config& c) { return c.dtype == MOE_BF16 && !(c.flags & MOE_FLAG_DOWN_HILO); }
// The split expert GEMMs can run for T tokens (bf16 layer at prefill sizes,
// not turned off): only then does the permutation write their tables.
bool split_sizes(const moe_config& c, int T) {
    if (c.flags & (MOE_FLAG_SPLIT_GEMM_OFF | MOE_FLAG_PAIR_CTA_ON | MOE_FLAG_FORCE_SIMT)) return false;
    return f16_down(c) && (int64_t)T * c.top_k >= 64LL * c.E;
}
// Expert outputs y: bf16 (FP8 and MXFP4 layers), fp16 (bf16 layer, fp16 down path), else fp32.
int y_elem(const moe_config& c) {
    return c.dtype == MOE_FP8_E4M3_B128 || c.dtype == MOE_MXFP4 ? moe::kBF16 : f16_down(c) ? moe::kF16 : moe::kF32;
}

// The first 256 bytes of the workspace: the error word (16 bytes), then from
// byte 64 one pair of unit-scheduling counters per GEMM launch of a forward
// (each rewound to zero by the kernel that used it).
constexpr size_t kErrBlock = 256;
constexpr int64_t kDefaultSpinNs = 2000000000LL;
constexpr size_t kFewBarrier = 128;  // uint64 barrier count of moe_forward_few
enum SchedSlot : int { kSchedRouter = 0, kSchedGateup = 1, kSchedDown = 2, kSchedSharedGateup = 3, kSchedSharedDown = 4 };

int act_bytes(int dtype) { return dtype == MOE_F32 ? 4 : (dtype == MOE_BF16 ? 2 : 1); }
int act_elem(int dtype) { return dtype == MOE_F32 ? moe::kF32 : (dtype == MOE_BF16 ? moe::kBF16 : moe::kE4M3); }
int in_elem(int dtype) { return dtype == MOE_F32 ? moe::kF32 : moe::kBF16; }  // x and router

int route_splits(const moe_config& c, int T, int num_sms) {
    return c.dtype == MOE_F32 ? 1 : moe::router_splits(T, c.E, c.D, num_sms);
}

// total never shrinks as T grows: a workspace sized for T_max is what callers
// use for every smaller T.  Parts that a larger T needs less of (hist,
// logits_part, few) therefore take what the smaller T's need of them.
void layout(const moe_config& c, int num_sms, int T, moe_ws_layout* L) {
    const int64_t TK = (int64_t)T * c.top_k, R = TK + T;
    const bool fp8 = c.dtype == MOE_FP8_E4M3_B128;
    const int ab = act_bytes(c.dtype);
    const int64_t nch = moe::perm_chunks_most(TK);
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o += up256(bytes); return at; };
    memset(L, 0, sizeof(*L));
    L->err = take(kErrBlock);
    L->logits = take((size_t)T * c.E * 4);
    L->blob = take((size_t)2 * TK * 4);
    L->counts = take((size_t)(c.E + 1) * 4);
    L->offsets = take((size_t)(c.E + 2) * 4);
    L->tiles = take((size_t)(c.E + 2) * 4);
    L->inv = take((size_t)TK * 4);
    L->src_tok = take((size_t)R * 4);
    L->hist = take((size_t)nch * c.E * 4);
    const bool mx = c.dtype == MOE_MXFP4;
    L->xq = fp8 ? take((size_t)T * c.D) : 0;
    L->xq_scale = fp8 ? take((size_t)T * (c.D / 128) * 4) : 0;
    // MXFP4: xq's rows follow xp's, so that the GEMMs see one run of R rows
    L->xp = take(mx ? (size_t)R * c.D / 2 : (size_t)TK * c.D * ab);
    L->xp_scale = fp8 ? take((size_t)TK * (c.D / 128) * 4) : mx ? take((size_t)R * c.D / 32) : 0;
    if (mx) {
        L->xq = L->xp + (size_t)TK * c.D / 2;
        L->xq_scale = L->xp_scale + (size_t)TK * c.D / 32;
    }
    // bf16 layer: h in fp16 ([R, I]), or as a bf16 hi/lo pair ([R, 2I]) under
    // MOE_FLAG_DOWN_HILO; a single bf16 rounding of h alone would cost about
    // 1e-2 of the output rms.
    L->h = take(mx ? (size_t)R * c.I / 2 : (size_t)R * c.I * (hilo(c) ? 4 : ab));
    L->h_scale = fp8 ? take((size_t)R * (c.I / 128) * 4) : mx ? take((size_t)R * c.I / 32) : 0;
    // y: fp16 for the bf16 layer, bf16 for the FP8 layer, else fp32 (a bf16 y
    // in the bf16 layer would cost about 1.3e-2 of the output rms).
    L->y = take((size_t)R * c.D * (y_elem(c) == moe::kF32 ? 4 : 2));
    const int64_t part_rows = c.dtype == MOE_F32 ? 0 : moe::router_part_rows(T, c.E, c.D, num_sms);
    const size_t part = part_rows ? take((size_t)part_rows * c.E * 4) : 0;
    L->logits_part = route_splits(c, T, num_sms) > 1 ? part : 0;
    L->tiles2 = take((size_t)(c.E + 2) * 4);
    L->pairs = take((size_t)(3 * (c.E + 2) + 2) * 4);
    L->gu = mx ? take((size_t)2 * R * c.I * 4) : 0;
    L->few = take((size_t)std::min(T, moe::kFewMax) * (c.top_k + 1) * c.I * 4);
    L->total = o;
}

struct Ws {
    moe_ws_layout L;
    char* base;
    int* sched(int slot) { return (int*)(base + L.err + 64) + 2 * slot; }
    template <typename T> T* at(size_t off) const { return (T*)(base + off); }
};

moe_status check_call(const moe_plan* p, int32_t T, void* ws, size_t ws_bytes, Ws* out) {
    if (!p) return arg_fail(MOE_ERR_INVALID_ARG, "plan is NULL");
    if (T < 1 || T > p->cfg.T_max) return arg_fail(MOE_ERR_INVALID_ARG, "T outside [1, T_max]");
    if (!ws || !aligned(ws, 256)) return arg_fail(MOE_ERR_INVALID_ARG, "workspace NULL or not 256-byte aligned");
    layout(p->cfg, p->num_sms, T, &out->L);
    if (ws_bytes < out->L.total) return arg_fail(MOE_ERR_WORKSPACE, "workspace smaller than moe_workspace_size()");
    out->base = (char*)ws;
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess || cur != p->device)
        return arg_fail(MOE_ERR_INVALID_ARG, "current CUDA device is not the plan's device");
    return MOE_OK;
}

bool ptr_ok(const void* q) { return q != nullptr && aligned(q, 16); }

moe_status check_weights(const moe_plan* p, const moe_weights* w, bool router, bool experts) {
    if (!w) return arg_fail(MOE_ERR_INVALID_ARG, "weights is NULL");
    if (router) {
        if (!ptr_ok(w->w_router)) return arg_fail(MOE_ERR_INVALID_ARG, "w_router NULL or misaligned");
        if (p->cfg.has_router_bias && !ptr_ok(w->b_router))
            return arg_fail(MOE_ERR_INVALID_ARG, "b_router NULL or misaligned");
    }
    if (experts) {
        if (!ptr_ok(w->w_gate) || !ptr_ok(w->w_up))
            return arg_fail(MOE_ERR_INVALID_ARG, "expert weight NULL or misaligned");
        // the bf16 layer's tensor-core down GEMM reads only the fp16 copy, so
        // there the bf16 w_down may be NULL (its memory freed by the caller)
        const bool f16_only = f16_down(p->cfg) && !(p->cfg.flags & MOE_FLAG_FORCE_SIMT);
        if (f16_only && !ptr_ok(w->w_down_f16))
            return arg_fail(MOE_ERR_INVALID_ARG, "w_down_f16 NULL or misaligned (see moe_convert_down_weights)");
        if (f16_only ? (w->w_down && !aligned(w->w_down, 16)) : !ptr_ok(w->w_down))
            return arg_fail(MOE_ERR_INVALID_ARG, "w_down NULL or misaligned");
        if ((p->cfg.dtype == MOE_FP8_E4M3_B128 || p->cfg.dtype == MOE_MXFP4) && (!ptr_ok(w->s_gate) || !ptr_ok(w->s_up) || !ptr_ok(w->s_down)))
            return arg_fail(MOE_ERR_INVALID_ARG, "block scales NULL or misaligned");
    }
    return MOE_OK;
}

bool use_tc(const moe_plan* p, const moe::GroupedGemm& g) {
    if (p->cfg.flags & MOE_FLAG_FORCE_SIMT) return false;
    return moe::gemm_tc_supported(g);
}

moe_status run_gemm(const moe_plan* p, const moe::GroupedGemm& g, cudaStream_t s, const char* what) {
    if (g.elem == moe::kE4M3) {
        if (!moe::gemm_fp8_supported(g)) return arg_fail(MOE_ERR_UNSUPPORTED, "FP8 GEMM shape without a kernel");
        cudaError_t e = moe::launch_gemm_fp8(g, p->num_sms, s);
        if (e != cudaSuccess) return cuda_fail(e, what);
        return MOE_OK;
    }
    if (use_tc(p, g)) {
        if (g.prefer_pairs && moe::gemm_tc2_supported(g)) MOE_CUDA(moe::launch_gemm_tc2(g, p->num_sms, s));
        else MOE_CUDA(moe::launch_gemm_tc(g, p->num_sms, s));
        return MOE_OK;
    }
    if (g.elem == moe::kE4M3) return arg_fail(MOE_ERR_UNSUPPORTED, "FP8 GEMM shape without a tensor-core kernel");
    cudaError_t e = moe::launch_gemm_simt(g, s);
    if (e != cudaSuccess) return cuda_fail(e, what);
    return MOE_OK;
}

// CTA pairs (256-row tiles) halve each CTA's operand traffic but pad every
// group to 256 rows: under skewed routing at T=8192 that is 31 % padded MMA
// rows against 18 % for 128-row tiles, and single CTAs measure faster.  So
// pairs run only on request.
int prefer_pairs(const moe_plan* p, int T) {
    (void)T;
    if (p->cfg.flags & MOE_FLAG_PAIR_CTA_OFF) return 0;
    return (p->cfg.flags & MOE_FLAG_PAIR_CTA_ON) ? 1 : 0;
}

// Tile pairs (2-CTA clusters sharing operand tiles) pay where groups hold
// several row tiles; at decode sizes the GEMMs stream weights from HBM and the
// clusters only couple the CTAs' progress.
int prefer_mcast(const moe_plan* p, int T) {
    const uint32_t f = p->cfg.flags;
    if (f & MOE_FLAG_MCAST_OFF) return 0;
    if (f & MOE_FLAG_MCAST_ON) return 1;
    return (int64_t)T * p->cfg.top_k >= 64 * (int64_t)p->cfg.E ? 1 : 0;
}

// Narrow tails save tensor time on ragged tiles; measured at T=8192 they
// take the gate/up GEMM from 1.264 to 1.247 ms, while in the down GEMM (y
// stored transposed, 2 bytes at a time) and at decode sizes they cost more
// than they save.
int prefer_narrow(const moe_plan* p, int T, bool gateup) {
    const uint32_t f = p->cfg.flags;
    if (f & MOE_FLAG_NARROW_TAILS_OFF) return 0;
    if (f & MOE_FLAG_NARROW_TAILS_ON) return 1;
    // the CTA-pair kernel stages its transposed stores: narrow tails in both GEMMs
    if (prefer_pairs(p, T)) return 1;
    return gateup && prefer_mcast(p, T) ? 1 : 0;
}

int grouped_max_tiles2(const moe_config& c, int T) {
    const int64_t R = (int64_t)T * (c.top_k + 1);
    return (int)(R / (2 * moe::kRowTile) + c.E + 2);
}

int grouped_max_tiles(const moe_config& c, int T) {
    const int64_t R = (int64_t)T * (c.top_k + 1);
    return (int)(R / moe::kRowTile + c.E + 2);
}

}  // namespace

extern "C" {

const char* moe_status_str(moe_status s) {
    switch (s) {
        case MOE_OK: return "ok";
        case MOE_ERR_INVALID_ARG: return "invalid argument";
        case MOE_ERR_UNSUPPORTED: return "unsupported shape or dtype";
        case MOE_ERR_WORKSPACE: return "workspace too small";
        case MOE_ERR_CUDA: return "CUDA error";
        case MOE_ERR_DEVICE_TIMEOUT: return "device wait timed out";
        case MOE_ERR_BOUNDS: return "device index check failed";
        case MOE_ERR_NONFINITE: return "non-finite router logit";
    }
    return "unknown status";
}

const char* moe_last_error_detail(void) { return g_detail; }

uint64_t moe_launch_count(void) { return moe::g_launches.load(std::memory_order_relaxed); }

const char* moe_build_info(void) { return "libmoe sm_103a: tcgen05+TMA grouped GEMM, SIMT grouped GEMM, route/permute/unpermute"; }

moe_status moe_plan_create(const moe_config* cfg, int device, moe_plan** out) {
    if (!out) return arg_fail(MOE_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!cfg) return arg_fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    const moe_config& c = *cfg;
    if (c.dtype < MOE_F32 || c.dtype > MOE_MXFP4) return arg_fail(MOE_ERR_UNSUPPORTED, "dtype");
    if (c.out_dtype != MOE_F32 && c.out_dtype != MOE_BF16) return arg_fail(MOE_ERR_UNSUPPORTED, "out_dtype");
    if (c.E < 1 || c.E > 1024) return arg_fail(MOE_ERR_UNSUPPORTED, "E outside [1, 1024]");
    if (c.top_k < 1 || c.top_k > std::min(c.E, 32)) return arg_fail(MOE_ERR_UNSUPPORTED, "top_k outside [1, min(E,32)]");
    if (c.T_max < 1 || c.T_max > (1 << 20)) return arg_fail(MOE_ERR_UNSUPPORTED, "T_max outside [1, 2^20]");
    if ((int64_t)c.T_max * (c.top_k + 1) >= (int64_t)1 << 31) return arg_fail(MOE_ERR_UNSUPPORTED, "T_max*(top_k+1) >= 2^31");
    const int q = (c.dtype == MOE_F32) ? 64 : 128;
    if (c.D < q || c.D % q || c.I < q || c.I % q) return arg_fail(MOE_ERR_UNSUPPORTED, "D and I must be multiples of 128 (64 for fp32)");
    if (c.D > 65536 || c.I > 65536) return arg_fail(MOE_ERR_UNSUPPORTED, "D or I above 65536");
    if (c.dtype == MOE_FP8_E4M3_B128 && c.D % 256)  // the FP8 down GEMM's units are 256 output features wide
        return arg_fail(MOE_ERR_UNSUPPORTED, "the FP8 layer needs D a multiple of 256");
    if (c.spin_limit_ns < 0) return arg_fail(MOE_ERR_INVALID_ARG, "spin_limit_ns < 0");
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev)
        return arg_fail(MOE_ERR_INVALID_ARG, "no such CUDA device");
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return arg_fail(MOE_ERR_CUDA, "device query failed");
    moe_plan* p = new moe_plan;
    p->cfg = c;
    p->device = device;
    p->num_sms = sms;
    p->spin_ns = c.spin_limit_ns ? c.spin_limit_ns : kDefaultSpinNs;
    int prev = 0;
    cudaGetDevice(&prev);
    if (cudaSetDevice(device) != cudaSuccess ||
        cudaStreamCreateWithFlags(&p->side, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->ev_fork, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->ev_join, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->ev_perm, cudaEventDisableTiming) != cudaSuccess) {
        moe_plan_destroy(p);
        cudaSetDevice(prev);
        return arg_fail(MOE_ERR_CUDA, "stream or event creation failed");
    }
    cudaSetDevice(prev);
    *out = p;
    return MOE_OK;
}

void moe_plan_destroy(moe_plan* p) {
    if (!p) return;
    if (p->ev_fork) cudaEventDestroy(p->ev_fork);
    if (p->ev_join) cudaEventDestroy(p->ev_join);
    if (p->ev_perm) cudaEventDestroy(p->ev_perm);
    if (p->side) cudaStreamDestroy(p->side);
    delete p;
}

const moe_config* moe_plan_config(const moe_plan* p) { return p ? &p->cfg : nullptr; }

moe_status moe_workspace_layout(const moe_plan* p, int32_t T, moe_ws_layout* out) {
    if (!p || !out) return arg_fail(MOE_ERR_INVALID_ARG, "NULL argument");
    if (T < 1 || T > p->cfg.T_max) return arg_fail(MOE_ERR_INVALID_ARG, "T outside [1, T_max]");
    layout(p->cfg, p->num_sms, T, out);
    return MOE_OK;
}

moe_status moe_workspace_size(const moe_plan* p, int32_t T, size_t* bytes) {
    if (!bytes) return arg_fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
    moe_ws_layout L;
    moe_status s = moe_workspace_layout(p, T, &L);
    if (s == MOE_OK) *bytes = L.total;
    return s;
}

moe_status moe_workspace_init(const moe_plan* p, void* ws, size_t ws_bytes, void* stream) {
    if (!p || !ws || !aligned(ws, 256) || ws_bytes < 256) return arg_fail(MOE_ERR_INVALID_ARG, "workspace");
    MOE_CUDA(cudaMemsetAsync(ws, 0, kErrBlock, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_quantize_weights(const moe_plan* p, const float* w, int64_t groups, int32_t rows, int32_t cols,
                                uint8_t* q, float* s, void* stream) {
    if (!p) return arg_fail(MOE_ERR_INVALID_ARG, "plan is NULL");
    if (!ptr_ok(w) || !ptr_ok(q) || !ptr_ok(s)) return arg_fail(MOE_ERR_INVALID_ARG, "NULL or misaligned pointer");
    if (groups < 1 || rows < 128 || cols < 128 || rows % 128 || cols % 128)
        return arg_fail(MOE_ERR_UNSUPPORTED, "rows and cols must be positive multiples of 128");
    MOE_CUDA(moe::launch_quant_blocks(w, groups, rows, cols, q, s, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_topk(const moe_plan* p, int32_t T, void* ws, size_t ws_bytes, void* stream) {
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    const moe_config& c = p->cfg;
    MOE_CUDA(moe::launch_topk(W.at<float>(W.L.logits), 1, nullptr, nullptr, T, c.E, c.top_k,
                              W.at<int32_t>(W.L.blob), W.at<uint32_t>(W.L.err), (cudaStream_t)stream));
    return MOE_OK;
}

namespace {
// moe_forward's route: with fused_hist the top-k kernel also counts the
// permutation's per-chunk expert histograms (zeroed here first), so that the
// permutation skips its own histogram pass.
moe_status route_impl(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, Ws& W, void* stream,
                      bool fused_hist, bool pdl = false);
}  // namespace

moe_status moe_route(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, void* ws, size_t ws_bytes,
                     void* stream) {
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if ((st = check_weights(p, w, true, false)) != MOE_OK) return st;
    if (!ptr_ok(x)) return arg_fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned");
    return route_impl(p, w, x, T, W, stream, false);
}

namespace {
bool fuse_topk_hist(const moe_plan* p, int32_t T) {
    return !(p->cfg.flags & MOE_FLAG_TOPK_HIST_OFF) && moe::permute_uses_chunks((int64_t)T * p->cfg.top_k, p->cfg.E);
}

// Zero the per-chunk histograms the fused top-k counts into.  moe_forward
// does this before it forks the shared-expert stream, so that the router
// GEMM is still the first kernel queued after the fork (a memset there let
// the shared GEMMs take the SMs first: 2.30 vs 2.25 ms at T=8192).
cudaError_t zero_topk_hist(const moe_plan* p, int32_t T, Ws& W, cudaStream_t s) {
    const int64_t TK = (int64_t)T * p->cfg.top_k;
    return cudaMemsetAsync(W.at<int32_t>(W.L.hist), 0, (size_t)moe::cdiv(TK, moe::perm_chunk(TK)) * p->cfg.E * 4, s);
}

moe_status route_impl(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, Ws& W, void* stream,
                      bool fused_hist, bool pdl) {
    moe_status st;
    const moe_config& c = p->cfg;
    moe::GroupedGemm g = {};
    g.G = 1;
    g.shared_group = -1;
    g.rows = T;
    g.max_tiles = (int)moe::cdiv(T, moe::kRowTile);
    g.N = c.E;
    g.Ka = g.Kb = c.D;
    g.ldo = c.E;
    g.a_rows = T;
    g.elem = in_elem(c.dtype);
    g.a = x;
    g.b = w->w_router;
    g.out = W.at<float>(W.L.logits);
    g.out_elem = moe::kF32;
    g.bias = c.has_router_bias ? w->b_router : nullptr;
    g.err = W.at<uint32_t>(W.L.err);
    g.sched = W.sched(kSchedRouter);
    g.spin_ns = p->spin_ns;
    // Small T: split K over several CTAs; the top-k kernel then adds the
    // slices in order (and the bias) and writes the logits.
    const int S = use_tc(p, g) ? route_splits(c, T, p->num_sms) : 1;
    if (S > 1) {
        g.ksplit = S;
        g.split_stride = (int64_t)T * c.E;
        g.out = W.at<float>(W.L.logits_part);
        g.bias = nullptr;
    }
    int32_t* hist = nullptr;
    int chunk = 1;
    if (fused_hist) {  // the caller zeroed the histograms (zero_topk_hist)
        chunk = moe::perm_chunk((int64_t)T * c.top_k);
        hist = W.at<int32_t>(W.L.hist);
    }
    if ((st = run_gemm(p, g, (cudaStream_t)stream, "router GEMM")) != MOE_OK) return st;
    moe::PdlScope scope(pdl);  // the top-k follows the router GEMM on this stream
    if (S > 1)
        MOE_CUDA(moe::launch_topk(W.at<float>(W.L.logits_part), S, c.has_router_bias ? w->b_router : nullptr,
                                  W.at<float>(W.L.logits), T, c.E, c.top_k, W.at<int32_t>(W.L.blob),
                                  W.at<uint32_t>(W.L.err), (cudaStream_t)stream, hist, chunk));
    else
        MOE_CUDA(moe::launch_topk(W.at<float>(W.L.logits), 1, nullptr, nullptr, T, c.E, c.top_k,
                                  W.at<int32_t>(W.L.blob), W.at<uint32_t>(W.L.err), (cudaStream_t)stream, hist,
                                  chunk));
    return MOE_OK;
}

// Permuted copy of x: from T >= 1024 tokens one warp per token reads its row
// once and writes its top_k copies (x leaves DRAM once); below that there
// are too few tokens to fill the GPU and one warp per output row gathers.
bool scatter_by_token(int32_t T) { return T >= 1024; }
// FP8 layer: quantise x on the way into xp (one kernel) where the scatter
// runs and a row fits the kernel's shared-memory copy
bool fused_quant_scatter(const moe_config& c, int32_t T) { return scatter_by_token(T) && c.D <= 4096; }

// quant_x: the FP8 layer quantises x into xq here (false when the caller
// already did).
// hist_ready: route_impl already counted the per-chunk histograms.
moe_status permute_impl(const moe_plan* p, const void* x, int32_t T, Ws& W, cudaStream_t s, bool quant_x,
                        bool hist_ready = false) {
    const moe_config& c = p->cfg;
    const int TK = T * c.top_k;
    MOE_CUDA(moe::launch_permute_index(W.at<int32_t>(W.L.blob), T, c.E, c.top_k, W.at<int32_t>(W.L.hist),
                                       W.at<int32_t>(W.L.counts), W.at<int32_t>(W.L.offsets),
                                       W.at<int32_t>(W.L.tiles), W.at<int32_t>(W.L.tiles2), W.at<int32_t>(W.L.inv),
                                       W.at<int32_t>(W.L.src_tok),
                                       W.at<uint32_t>(W.L.err), s, hist_ready,
                                       split_sizes(c, T) ? W.at<int32_t>(W.L.pairs) : nullptr,
                                       std::max(1, p->num_sms / 2), prefer_narrow(p, T, true)));
    if (c.dtype == MOE_MXFP4) {
        uint8_t *xq = W.at<uint8_t>(W.L.xq), *sq = W.at<uint8_t>(W.L.xq_scale);
        MOE_CUDA(moe::launch_mx_quantize(x, moe::kBF16, c.D, T, c.D, xq, sq, s));
        MOE_CUDA(moe::launch_gather_rows(xq, 1, c.D / 2, W.at<int32_t>(W.L.src_tok), TK, W.at<uint8_t>(W.L.xp), s));
        MOE_CUDA(moe::launch_gather_rows(sq, 1, c.D / 32, W.at<int32_t>(W.L.src_tok), TK, W.at<uint8_t>(W.L.xp_scale), s));
    } else if (c.dtype == MOE_FP8_E4M3_B128) {
        // xq (x quantised) is the shared expert's A operand; the routed rows
        // are quantised from x on the way into xp at scatter sizes
        if (quant_x)
            MOE_CUDA(moe::launch_quant_rows(x, moe::kBF16, T, c.D, W.at<uint8_t>(W.L.xq), W.at<float>(W.L.xq_scale), s));
        if (fused_quant_scatter(c, T)) {
            MOE_CUDA(moe::launch_scatter_quant_rows(x, moe::kBF16, T, c.D, W.at<int32_t>(W.L.inv), c.top_k,
                                                    W.at<uint8_t>(W.L.xp), W.at<float>(W.L.xp_scale), s));
        } else {
            if (scatter_by_token(T))
                MOE_CUDA(moe::launch_scatter_rows(W.at<uint8_t>(W.L.xq), c.D, W.at<int32_t>(W.L.inv), T, c.top_k,
                                                  W.at<uint8_t>(W.L.xp), s));
            else
                MOE_CUDA(moe::launch_gather_rows(W.at<uint8_t>(W.L.xq), 1, c.D, W.at<int32_t>(W.L.src_tok), TK,
                                                 W.at<uint8_t>(W.L.xp), s));
            MOE_CUDA(moe::launch_gather_rows(W.at<float>(W.L.xq_scale), 4, (int64_t)(c.D / 128) * 4,
                                             W.at<int32_t>(W.L.src_tok), TK, W.at<float>(W.L.xp_scale), s));
        }
    } else {
        const int eb = act_bytes(c.dtype);
        if (scatter_by_token(T))
            MOE_CUDA(moe::launch_scatter_rows(x, (int64_t)c.D * eb, W.at<int32_t>(W.L.inv), T, c.top_k,
                                              W.at<char>(W.L.xp), s));
        else
            MOE_CUDA(moe::launch_gather_rows(x, eb, (int64_t)c.D * eb, W.at<int32_t>(W.L.src_tok), TK,
                                             W.at<char>(W.L.xp), s));
    }
    return MOE_OK;
}
}  // namespace

moe_status moe_permute(const moe_plan* p, const void* x, int32_t T, void* ws, size_t ws_bytes, void* stream) {
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if (!ptr_ok(x)) return arg_fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned");
    return permute_impl(p, x, T, W, (cudaStream_t)stream, true);
}

namespace {

moe::GroupedGemm gateup_gemm(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, Ws& W) {
    const moe_config& c = p->cfg;
    const bool fp8 = c.dtype == MOE_FP8_E4M3_B128;
    moe::GroupedGemm g = {};
    g.G = c.E + 1;
    g.shared_group = c.E;
    g.offsets = W.at<int32_t>(W.L.offsets);
    g.tiles = W.at<int32_t>(W.L.tiles);
    g.max_tiles = grouped_max_tiles(c, T);
    g.tiles2 = W.at<int32_t>(W.L.tiles2);
    g.max_tiles2 = grouped_max_tiles2(c, T);
    g.prefer_pairs = prefer_pairs(p, T);
    g.mcast = prefer_mcast(p, T);
    g.narrow = prefer_narrow(p, T, true);
    g.N = c.I;
    g.Ka = g.Kb = c.D;
    g.out_pair = hilo(c);
    g.ldo = g.out_pair ? 2 * c.I : c.I;
    g.a_rows = T * c.top_k;
    g.a_shared_rows = T;
    g.elem = act_elem(c.dtype);
    g.a = W.at<void>(W.L.xp);
    g.a_shared = fp8 ? (const void*)W.at<uint8_t>(W.L.xq) : x;
    g.a_scale = fp8 ? W.at<float>(W.L.xp_scale) : nullptr;
    g.a_shared_scale = fp8 ? W.at<float>(W.L.xq_scale) : nullptr;
    g.b = w->w_gate;
    g.b2 = w->w_up;
    g.b_scale = w->s_gate;
    g.b2_scale = w->s_up;
    g.out = W.at<void>(W.L.h);
    g.out_elem = f16_down(c) ? moe::kF16 : act_elem(c.dtype);
    g.out_scale = fp8 ? W.at<float>(W.L.h_scale) : nullptr;
    g.err = W.at<uint32_t>(W.L.err);
    g.sched = W.sched(kSchedGateup);
    g.spin_ns = p->spin_ns;
    return g;
}

moe::GroupedGemm down_gemm(const moe_plan* p, const moe_weights* w, int32_t T, Ws& W) {
    const moe_config& c = p->cfg;
    const bool fp8 = c.dtype == MOE_FP8_E4M3_B128;
    moe::GroupedGemm g = {};
    g.G = c.E + 1;
    g.shared_group = -1;
    g.offsets = W.at<int32_t>(W.L.offsets);
    g.tiles = W.at<int32_t>(W.L.tiles);
    g.max_tiles = grouped_max_tiles(c, T);
    g.tiles2 = W.at<int32_t>(W.L.tiles2);
    g.max_tiles2 = grouped_max_tiles2(c, T);
    g.prefer_pairs = prefer_pairs(p, T);
    g.mcast = prefer_mcast(p, T);
    g.narrow = prefer_narrow(p, T, false);
    g.many_rows = (int64_t)T * c.top_k >= 64 * (int64_t)c.E;
    g.N = c.D;
    g.Kb = c.I;
    g.Ka = hilo(c) ? 2 * c.I : c.I;  // the hi/lo pair walks W_down twice
    g.ldo = c.D;
    g.a_rows = T * (c.top_k + 1);
    g.elem = act_elem(c.dtype);
    g.a = W.at<void>(W.L.h);
    g.a_scale = fp8 ? W.at<float>(W.L.h_scale) : nullptr;
    g.b = w->w_down;
    if (f16_down(c)) {
        g.elem = moe::kF16;  // fp16 h
        if (c.flags & MOE_FLAG_FORCE_SIMT) g.b_elem = moe::kBF16;  // CUDA cores read the bf16 W_down
        else g.b = w->w_down_f16;                                   // tensor cores: one type for A and B
    }
    g.b_scale = w->s_down;
    g.out = W.at<void>(W.L.y);
    g.out_elem = y_elem(c);
    g.err = W.at<uint32_t>(W.L.err);
    // dynamic unit order measured slower for the bf16 down GEMM (0.80 vs
    // 0.78 ms at T=8192), faster for the FP8 one (1.42 vs 1.43 ms) and for
    // every gate/up GEMM
    g.sched = W.sched(kSchedDown);  // (tile pairs at prefill take the static order)
    g.spin_ns = p->spin_ns;
    return g;
}

// MXFP4: an expert GEMM over all E+1 groups (the shared expert's rows follow
// the routed ones), gate, up (fp32) or down.
moe::MxGemm mx_gemm(const moe_plan* p, int32_t T, Ws& W, const uint8_t* a, const uint8_t* as, const void* b, const void* bs,
                    int N, int K, void* out, int out_elem) {
    const moe_config& c = p->cfg;
    moe::MxGemm g = {};
    g.a = a;
    g.a_scale = as;
    g.b = (const uint8_t*)b;
    g.b_scale = (const uint8_t*)bs;
    g.offsets = W.at<int32_t>(W.L.offsets);
    g.rows = T * (c.top_k + 1);
    g.G = c.E + 1;
    g.N = N;
    g.K = K;
    g.out = out;
    g.out_elem = out_elem;
    g.ldo = N;
    g.err = W.at<uint32_t>(W.L.err);
    g.spin_ns = p->spin_ns;
    return g;
}

// h = silu(gate) * up quantised: two GEMMs, then one pass over their outputs
// (h's scales need 32 finished columns of both).
moe_status mx_gateup(const moe_plan* p, const moe_weights* w, int32_t T, Ws& W, cudaStream_t s) {
    const moe_config& c = p->cfg;
    const int64_t R = (int64_t)T * (c.top_k + 1);
    float* gu = W.at<float>(W.L.gu);
    const uint8_t *a = W.at<uint8_t>(W.L.xp), *as = W.at<uint8_t>(W.L.xp_scale);
    MOE_CUDA(moe::launch_gemm_mx(mx_gemm(p, T, W, a, as, w->w_gate, w->s_gate, c.I, c.D, gu, moe::kF32), p->num_sms, s));
    MOE_CUDA(moe::launch_gemm_mx(mx_gemm(p, T, W, a, as, w->w_up, w->s_up, c.I, c.D, gu + R * c.I, moe::kF32), p->num_sms, s));
    MOE_CUDA(moe::launch_mx_swiglu(gu, gu + R * c.I, R * c.I, W.at<uint8_t>(W.L.h), W.at<uint8_t>(W.L.h_scale), s));
    return MOE_OK;
}
moe_status mx_down(const moe_plan* p, const moe_weights* w, int32_t T, Ws& W, cudaStream_t s) {
    const moe_config& c = p->cfg;
    MOE_CUDA(moe::launch_gemm_mx(mx_gemm(p, T, W, W.at<uint8_t>(W.L.h), W.at<uint8_t>(W.L.h_scale), w->w_down, w->s_down, c.D, c.I,
                                         W.at<void>(W.L.y), moe::kBF16),
                                 p->num_sms, s));
    return MOE_OK;
}

int elem_bytes(int e) { return e == moe::kF32 ? 4 : e == moe::kE4M3 ? 1 : 2; }

// The shared expert alone, as a dense GEMM over its T rows (which sit after
// the T*k routed rows of the grouped layout).  Its A comes from x (gate/up)
// or from the shared rows of h (down); its B is group E of the weights.
moe::GroupedGemm shared_only(const moe::GroupedGemm& full, const moe_config& c, int32_t T, bool gateup,
                             const void* x, const float* x_scale) {
    moe::GroupedGemm g = full;
    const int64_t TK = (int64_t)T * c.top_k;
    g.G = 1;
    g.shared_group = -1;
    g.offsets = g.tiles = g.tiles2 = nullptr;
    g.prefer_pairs = 0;
    g.rows = T;
    g.max_tiles = (int)moe::cdiv(T, moe::kRowTile);
    g.a_rows = T;
    g.a_shared = nullptr;
    g.a_shared_rows = 0;
    const int eb = elem_bytes(g.elem);
    const int bb = elem_bytes(g.b_elem > 0 ? g.b_elem : g.elem);
    if (gateup) {
        g.a = x;
        g.a_scale = x_scale;
    } else {
        g.a = (const char*)full.a + TK * g.Ka * eb;
        if (full.a_scale) g.a_scale = full.a_scale + TK * (g.Ka / 128);
    }
    g.a_shared_scale = nullptr;
    const int64_t group = (int64_t)g.N * g.Kb * bb;
    g.b = (const char*)full.b + c.E * group;
    if (g.b2) g.b2 = (const char*)full.b2 + c.E * group;
    const int64_t sgroup = (int64_t)(g.N / 128) * (g.Kb / 128);  // FP8 block scales of one group
    if (full.b_scale) g.b_scale = full.b_scale + c.E * sgroup;
    if (full.b2_scale) g.b2_scale = full.b2_scale + c.E * sgroup;
    g.out = (char*)full.out + TK * g.ldo * elem_bytes(g.out_elem);
    if (full.out_scale) g.out_scale = full.out_scale + TK * (g.N / 128);
    return g;
}

// Split expert GEMMs (see moe_forward): the bf16 layer at prefill sizes,
// unless the caller asked for the plain CTA-pair kernel or turned the split
// off.  Fills the two launches of each GEMM: gp on CTA pairs over the whole
// 256-row pairs (pairs[0..E+1]), as many pairs as the permutation counted
// (pairs[2(E+2) + i]); gr on single CTAs over the rest of each group
// (pairs[E+2..], in the group order at pairs[2(E+2)+2..] that keeps it near
// the pair launch's progress), drawing units from the shared expert's
// counters (its GEMMs are done by then on the same stream).
bool split_wanted(const moe_plan* p, int T, Ws& W, const moe::GroupedGemm& gu, const moe::GroupedGemm& dn,
                  moe::GroupedGemm* gp, moe::GroupedGemm* gr) {
    const moe_config& c = p->cfg;
    if (!split_sizes(c, T)) return false;
    int32_t* pairs = W.at<int32_t>(W.L.pairs);
    for (int i = 0; i < 2; ++i) {
        const moe::GroupedGemm& base = i == 0 ? gu : dn;
        gp[i] = base;
        gp[i].prefer_pairs = 1;
        gp[i].tiles2 = pairs;
        gp[i].narrow = 0;
        gp[i].pair_active = pairs + 2 * (c.E + 2) + i;
        gr[i] = base;
        gr[i].tiles = pairs + (c.E + 2);
        gr[i].rem_only = 1;
        gr[i].rem_order = pairs + 2 * (c.E + 2) + 2;
        gr[i].mcast = 0;
        gr[i].prefer_pairs = 0;
        gr[i].sched = W.sched(i == 0 ? kSchedSharedGateup : kSchedSharedDown);
        if (!moe::gemm_tc2_supported(gp[i]) || !moe::gemm_tc_supported(gr[i])) return false;
    }
    return true;
}

// A stage entry point's expert GEMM (all groups, the shared one included),
// split as in moe_forward where that applies: the whole 256-row pairs on the
// caller's stream, the rest on the plan's second stream, joined back before
// returning.  which: 0 gate/up, 1 down.
moe_status run_stage_gemm(const moe_plan* p, const moe::GroupedGemm& g, int which, int32_t T, Ws& W, cudaStream_t s,
                          const char* what) {
    moe::GroupedGemm gp[2], gr[2];
    if (!split_wanted(p, T, W, g, g, gp, gr)) return run_gemm(p, g, s, what);
    MOE_CUDA(cudaEventRecord(p->ev_fork, s));
    MOE_CUDA(cudaStreamWaitEvent(p->side, p->ev_fork, 0));
    const moe_status st = run_gemm(p, gp[which], s, what);
    const moe_status st2 = run_gemm(p, gr[which], p->side, what);
    MOE_CUDA(cudaEventRecord(p->ev_join, p->side));
    MOE_CUDA(cudaStreamWaitEvent(s, p->ev_join, 0));  // joined even after an error (stream capture)
    return st != MOE_OK ? st : st2;
}

}  // namespace

moe_status moe_gemm_gateup(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, void* ws,
                           size_t ws_bytes, void* stream) {
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if ((st = check_weights(p, w, false, true)) != MOE_OK) return st;
    if (!ptr_ok(x)) return arg_fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned");
    if (p->cfg.dtype == MOE_MXFP4) return mx_gateup(p, w, T, W, (cudaStream_t)stream);
    return run_stage_gemm(p, gateup_gemm(p, w, x, T, W), 0, T, W, (cudaStream_t)stream, "gate/up GEMM");
}

moe_status moe_gemm_down(const moe_plan* p, const moe_weights* w, int32_t T, void* ws, size_t ws_bytes,
                         void* stream) {
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if ((st = check_weights(p, w, false, true)) != MOE_OK) return st;
    if (p->cfg.dtype == MOE_MXFP4) return mx_down(p, w, T, W, (cudaStream_t)stream);
    return run_stage_gemm(p, down_gemm(p, w, T, W), 1, T, W, (cudaStream_t)stream, "down GEMM");
}

moe_status moe_unpermute(const moe_plan* p, int32_t T, void* out, void* ws, size_t ws_bytes, void* stream) {
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if (!ptr_ok(out)) return arg_fail(MOE_ERR_INVALID_ARG, "out NULL or misaligned");
    const moe_config& c = p->cfg;
    MOE_CUDA(moe::launch_unpermute(W.at<void>(W.L.y), y_elem(c),
                                   W.at<int32_t>(W.L.blob), W.at<int32_t>(W.L.inv), T, c.D, c.top_k, out,
                                   c.out_dtype == MOE_F32 ? moe::kF32 : moe::kBF16, W.at<uint32_t>(W.L.err),
                                   (cudaStream_t)stream));
    return MOE_OK;
}

namespace {
// moe_forward's optional copies of the routing blob and the logits.
moe_status copy_routing_out(const moe_plan* p, Ws& W, int32_t T, int32_t* blob_out, float* logits_out,
                            cudaStream_t s) {
    const moe_config& c = p->cfg;
    if (blob_out)
        MOE_CUDA(cudaMemcpyAsync(blob_out, W.at<int32_t>(W.L.blob), (size_t)2 * T * c.top_k * 4,
                                 cudaMemcpyDeviceToDevice, s));
    if (logits_out)
        MOE_CUDA(cudaMemcpyAsync(logits_out, W.at<float>(W.L.logits), (size_t)T * c.E * 4, cudaMemcpyDeviceToDevice, s));
    return MOE_OK;
}
}  // namespace

moe_status moe_forward(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, void* out,
                       int32_t* blob_out, float* logits_out, void* ws, size_t ws_bytes, void* stream) {
    if (p && T == 0) return MOE_OK;  // an empty batch: nothing to read, write or launch
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if ((st = check_weights(p, w, true, true)) != MOE_OK) return st;
    if (!ptr_ok(x) || !ptr_ok(out)) return arg_fail(MOE_ERR_INVALID_ARG, "x or out NULL or misaligned");
    if ((blob_out && !aligned(blob_out, 16)) || (logits_out && !aligned(logits_out, 16)))
        return arg_fail(MOE_ERR_INVALID_ARG, "blob_out or logits_out misaligned");
    cudaStream_t s = (cudaStream_t)stream;
    const moe_config& cf = p->cfg;
    MOE_CUDA(cudaMemsetAsync(ws, 0, kErrBlock, s));
    const bool fh = fuse_topk_hist(p, T);
    if (fh) MOE_CUDA(zero_topk_hist(p, T, W, s));
    if (cf.dtype == MOE_MXFP4) {
        if ((st = route_impl(p, w, x, T, W, stream, fh)) != MOE_OK) return st;
        if ((st = permute_impl(p, x, T, W, s, true, fh)) != MOE_OK) return st;
        if ((st = mx_gateup(p, w, T, W, s)) != MOE_OK) return st;
        if ((st = mx_down(p, w, T, W, s)) != MOE_OK) return st;
        if ((st = moe_unpermute(p, T, out, ws, ws_bytes, stream)) != MOE_OK) return st;
        return copy_routing_out(p, W, T, blob_out, logits_out, s);
    }
    moe::GroupedGemm gu = gateup_gemm(p, w, x, T, W), dn = down_gemm(p, w, T, W);
    const bool fp8 = cf.dtype == MOE_FP8_E4M3_B128;
    moe::GroupedGemm sgu = shared_only(gu, cf, T, true, fp8 ? (const void*)W.at<uint8_t>(W.L.xq) : x,
                                       fp8 ? W.at<float>(W.L.xq_scale) : nullptr);
    moe::GroupedGemm sdn = shared_only(dn, cf, T, false, nullptr, nullptr);
    // The shared expert needs no routing: on the tensor-core path its two
    // GEMMs run on the plan's second stream while the router, top-k and
    // permutation run here; the routed GEMMs then skip the shared group.
    // (FP8: the shared GEMM reads xq, x quantised per row; see below.)
    const bool overlap =
        !(cf.flags & MOE_FLAG_FORCE_SIMT) &&
        (fp8 ? (moe::gemm_fp8_supported(gu) && moe::gemm_fp8_supported(dn) && moe::gemm_fp8_supported(sgu) &&
                moe::gemm_fp8_supported(sdn))
             : (cf.dtype == MOE_BF16 && moe::gemm_tc_supported(gu) && moe::gemm_tc_supported(dn) &&
                moe::gemm_tc_supported(sgu) && moe::gemm_tc_supported(sdn)));
    // Fused unpermutation (MOE_FLAG_FUSED_COMBINE, fp16 / bf16 y): the
    // shared expert's down GEMM runs last, on this stream, and its epilogue
    // writes out; the unpermute kernel is not launched.
    const bool fused_comb = overlap && (cf.flags & MOE_FLAG_FUSED_COMBINE) && (fp8 || f16_down(cf));
    if (fused_comb) {
        sdn.cmb_out = out;
        sdn.cmb_out_f32 = cf.out_dtype == MOE_F32;
        sdn.cmb_blob = W.at<int32_t>(W.L.blob);
        sdn.cmb_inv = W.at<int32_t>(W.L.inv);
        sdn.cmb_y = W.at<void>(W.L.y);
        sdn.cmb_k = cf.top_k;
        const bool ok = fp8 ? moe::gemm_fp8_supported(sdn) : moe::gemm_tc_supported(sdn);
        if (!ok) return arg_fail(MOE_ERR_UNSUPPORTED, "fused unpermutation: shape without a kernel");
    }
    // Programmatic dependent launch along the main-stream chain (top-k,
    // permutation, expert GEMMs) below prefill sizes: batched decode bf16,
    // T=1024, 0.880 ms per layer against 0.898 without.  At T*k >= 64E
    // (prefill) it cost 15-25 us, also with only the routing and permutation
    // kernels dependent: early-launched CTAs waiting on their predecessor
    // hold SMs that the shared expert's GEMMs would otherwise take.
    const bool pdl = (int64_t)T * cf.top_k < 64LL * cf.E;
    if (overlap) {
        gu.g_end = dn.g_end = cf.E;
        // The FP8 kernel's CTA holds all of an SM's registers, so nothing
        // else runs beside it: the shared GEMMs then take five eighths of the
        // SMs and leave the rest to the top-k and permutation kernels (FP8
        // prefill, T=16384: 2.880 ms per layer against 2.894 with half, 2.896
        // with 3/4, 2.930 with all; decode sizes unchanged).  The bf16
        // shared GEMMs take three quarters (prefill bf16, T=8192: 2.223 ms
        // per layer against 2.252 with all SMs, 2.233 with 5/8, 2.251 with
        // 7/8; decode sizes unchanged).
        if (fp8) sgu.max_ctas = sdn.max_ctas = std::max(1, p->num_sms * 5 / 8);
        else sgu.max_ctas = sdn.max_ctas = std::max(1, p->num_sms * 3 / 4);
        if (fused_comb) sdn.max_ctas = 0;  // it runs alone at the end
        sgu.sched = W.sched(kSchedSharedGateup);
        sdn.sched = W.sched(kSchedSharedDown);
        // FP8: xq (the shared expert's A) is made on the side stream at
        // scatter sizes, where the permutation quantises the routed rows
        // itself; below them the gather reads xq, so it is made here
        const bool side_quant = fp8 && fused_quant_scatter(cf, T);
        if (fp8 && !side_quant)
            MOE_CUDA(moe::launch_quant_rows(x, moe::kBF16, T, cf.D, W.at<uint8_t>(W.L.xq), W.at<float>(W.L.xq_scale), s));
        MOE_CUDA(cudaEventRecord(p->ev_fork, s));
        // the router GEMM is enqueued first so that it gets the SMs; the
        // shared GEMMs fill them as its CTAs retire and run beside the
        // top-k and permutation kernels
        st = route_impl(p, w, x, T, W, stream, fh, pdl);
        MOE_CUDA(cudaStreamWaitEvent(p->side, p->ev_fork, 0));
        if (side_quant)
            MOE_CUDA(moe::launch_quant_rows(x, moe::kBF16, T, cf.D, W.at<uint8_t>(W.L.xq), W.at<float>(W.L.xq_scale),
                                            p->side));
        moe_status side_st = run_gemm(p, sgu, p->side, "shared gate/up GEMM");
        if (side_st == MOE_OK && !fused_comb) side_st = run_gemm(p, sdn, p->side, "shared down GEMM");
        // Split expert GEMMs (MOE_FLAG_SPLIT_GEMM_OFF): each routed GEMM as the
        // whole 256-row pairs on CTA pairs here and the rest of every group on
        // single CTAs on the second stream, at the same time.  The two halves
        // write disjoint rows, and each down half reads only the h rows its
        // own gate/up half wrote.  Prefill bf16, T=8192: see the design notes.
        moe::GroupedGemm gp[2], gr[2];
        const bool split = !fp8 && !fused_comb && split_wanted(p, T, W, gu, dn, gp, gr);
        if (!split) MOE_CUDA(cudaEventRecord(p->ev_join, p->side));
        {
            // the main-stream chain after the top-k: each kernel a programmatic
            // dependent of the one before it
            moe::PdlScope scope(pdl);
            if (st == MOE_OK) st = permute_impl(p, x, T, W, s, !fp8, fh);
            if (split) {
                MOE_CUDA(cudaEventRecord(p->ev_perm, s));
                MOE_CUDA(cudaStreamWaitEvent(p->side, p->ev_perm, 0));
                for (int i = 0; i < 2; ++i) {
                    if (st == MOE_OK) st = run_gemm(p, gp[i], s, i == 0 ? "gate/up GEMM, 256-row pairs" : "down GEMM, 256-row pairs");
                    if (side_st == MOE_OK)
                        side_st = run_gemm(p, gr[i], p->side, i == 0 ? "gate/up GEMM, remaining rows" : "down GEMM, remaining rows");
                }
                MOE_CUDA(cudaEventRecord(p->ev_join, p->side));
            } else {
                if (st == MOE_OK) st = run_gemm(p, gu, s, "gate/up GEMM");
                if (st == MOE_OK) st = run_gemm(p, dn, s, "down GEMM");
            }
        }
        MOE_CUDA(cudaStreamWaitEvent(s, p->ev_join, 0));  // joined even after an error (stream capture)
        if (side_st != MOE_OK) return side_st;
        if (st != MOE_OK) return st;
        if (fused_comb) {
            if ((st = run_gemm(p, sdn, s, "shared down GEMM with the unpermutation")) != MOE_OK) return st;
            return copy_routing_out(p, W, T, blob_out, logits_out, s);
        }
    } else {
        if ((st = route_impl(p, w, x, T, W, stream, fh, pdl)) != MOE_OK) return st;
        moe::PdlScope scope(pdl);
        if ((st = permute_impl(p, x, T, W, s, true, fh)) != MOE_OK) return st;
        if ((st = run_gemm(p, gu, s, "gate/up GEMM")) != MOE_OK) return st;
        if ((st = run_gemm(p, dn, s, "down GEMM")) != MOE_OK) return st;
    }
    if ((st = moe_unpermute(p, T, out, ws, ws_bytes, stream)) != MOE_OK) return st;
    return copy_routing_out(p, W, T, blob_out, logits_out, s);
}

// ------------------------------------------------- operators of the block
// Each is launched as a programmatic dependent of what is before it on the
// stream: its launch overlaps that kernel's end, some 2 us a call (7 x 4096 x
// 4096 product 8.2 -> 6.0 us back to back, 301 x 1023 post-norm 10.3 -> 8.3).

moe_status moe_forward_few(const moe_plan* p, const moe_weights* w, const void* x, int32_t T, void* out,
                           int32_t* blob_out, float* logits_out, void* ws, size_t ws_bytes, void* stream) {
    if (p && T == 0) return MOE_OK;
    Ws W;
    moe_status st = check_call(p, T, ws, ws_bytes, &W);
    if (st != MOE_OK) return st;
    if (T > moe::kFewMax) return arg_fail(MOE_ERR_UNSUPPORTED, "T above MOE_FEW_MAX (use moe_forward)");
    if ((st = check_weights(p, w, true, true)) != MOE_OK) return st;
    if (!ptr_ok(x) || !ptr_ok(out)) return arg_fail(MOE_ERR_INVALID_ARG, "x or out NULL or misaligned");
    if ((blob_out && !aligned(blob_out, 16)) || (logits_out && !aligned(logits_out, 16)))
        return arg_fail(MOE_ERR_INVALID_ARG, "blob_out or logits_out misaligned");
    const moe_config& c = p->cfg;
    const int down_f16 = f16_down(c) && w->w_down_f16;
    if (!moe::few_fits(c.dtype, down_f16, c.D, c.I, c.top_k)) return moe_forward(p, w, x, T, out, blob_out, logits_out, ws, ws_bytes, stream);
    moe::FewParams f = {};
    f.T = T;
    f.D = c.D;
    f.E = c.E;
    f.I = c.I;
    f.k = c.top_k;
    f.dtype = c.dtype;
    f.out_elem = c.out_dtype == MOE_F32 ? moe::kF32 : moe::kBF16;
    f.x = x;
    f.w_router = w->w_router;
    f.b_router = c.has_router_bias ? w->b_router : nullptr;
    f.w_gate = w->w_gate;
    f.w_up = w->w_up;
    f.down_f16 = down_f16;
    f.w_down = f.down_f16 ? w->w_down_f16 : w->w_down;
    f.s_gate = w->s_gate;
    f.s_up = w->s_up;
    f.s_down = w->s_down;
    f.logits = W.at<float>(W.L.logits);
    f.blob = W.at<int32_t>(W.L.blob);
    f.h = W.at<float>(W.L.few);
    f.out = out;
    f.err = W.at<uint32_t>(W.L.err);
    f.bar = (unsigned long long*)W.at<char>(W.L.err + kFewBarrier);
    f.spin_ns = p->spin_ns;
    cudaStream_t s = (cudaStream_t)stream;
    MOE_CUDA(moe::launch_few(f, p->num_sms, s));
    return copy_routing_out(p, W, T, blob_out, logits_out, s);
}

namespace {

bool float_type(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
int float_elem(int dtype) { return dtype == MOE_F32 ? moe::kF32 : moe::kBF16; }
// A tensor of rows with any element-aligned base and a row stride that holds a row.
bool rows_ok(const void* q, int dtype, int64_t ld, int64_t cols) {
    return q && aligned(q, dtype == MOE_F32 ? 4 : 2) && ld >= cols;
}

moe_status check_norm(const moe_norm& n, moe::NormParams* out) {
    if (n.kind < MOE_NORM_NONE || n.kind > MOE_NORM_LAYER) return arg_fail(MOE_ERR_INVALID_ARG, "norm kind");
    out->kind = n.kind;
    if (n.kind == MOE_NORM_NONE) return MOE_OK;
    if (!(n.eps >= 0.0f)) return arg_fail(MOE_ERR_INVALID_ARG, "norm eps negative or NaN");
    if ((n.w || n.b) && !float_type(n.p_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "norm parameters neither fp32 nor bf16");
    const size_t a = n.p_dtype == MOE_F32 ? 4 : 2;
    if (!aligned(n.w, a) || !aligned(n.b, a)) return arg_fail(MOE_ERR_INVALID_ARG, "norm parameters misaligned");
    out->eps = n.eps;
    out->w_offset = n.w_offset;
    out->p_bf16 = n.p_dtype == MOE_BF16;
    out->w = n.w;
    out->b = n.b;
    return MOE_OK;
}

moe_status check_rows(int32_t T, int32_t D) {
    if (T < 0 || D < 1) return arg_fail(MOE_ERR_INVALID_ARG, "T < 0 or D < 1");
    if (!moe::norm_supported(D)) return arg_fail(MOE_ERR_UNSUPPORTED, "rows above 16384 elements");
    return MOE_OK;
}

}  // namespace

moe_status moe_norm_pre(const moe_norm* n, const void* x, int32_t dtype, int64_t ld_x, int32_t T, int32_t D, void* out,
                        int32_t out_dtype, int64_t ld_out, void* stream) {
    if (!n) return arg_fail(MOE_ERR_INVALID_ARG, "norm is NULL");
    moe::NormParams np = {};
    moe_status st = check_norm(*n, &np);
    if (st != MOE_OK || (st = check_rows(T, D)) != MOE_OK) return st;
    if (!float_type(dtype) || !float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "x and out must be fp32 or bf16");
    if (T == 0) return MOE_OK;
    if (!rows_ok(x, dtype, ld_x, D) || !rows_ok(out, out_dtype, ld_out, D))
        return arg_fail(MOE_ERR_INVALID_ARG, "x or out NULL or misaligned, or a row stride below D");
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_norm_pre(np, x, float_elem(dtype), ld_x, T, D, out, float_elem(out_dtype), ld_out,
                                  (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_norm_post(const moe_post* post, const void* y, int32_t dtype, int64_t ld_y, const void* res,
                         int32_t res_dtype, int64_t ld_res, int32_t T, int32_t D, void* out, int64_t ld_out,
                         void* next_out, int32_t next_dtype, int64_t ld_next, void* stream) {
    if (!post) return arg_fail(MOE_ERR_INVALID_ARG, "post is NULL");
    moe::PostParams p = {};
    moe_status st = check_norm(post->norm, &p.norm);
    if (st != MOE_OK || (st = check_norm(post->next, &p.next)) != MOE_OK || (st = check_rows(T, D)) != MOE_OK) return st;
    const bool has_next = p.next.kind != MOE_NORM_NONE;
    if (!float_type(dtype) || !float_type(res_dtype) || (has_next && !float_type(next_dtype)))
        return arg_fail(MOE_ERR_UNSUPPORTED, "y, res and next_out must be fp32 or bf16");
    if (post->gate_by < MOE_GATE_NONE || post->gate_by > MOE_GATE_FULL) return arg_fail(MOE_ERR_INVALID_ARG, "gate_by");
    if (post->gate_by != MOE_GATE_NONE && !float_type(post->gate_dtype))
        return arg_fail(MOE_ERR_UNSUPPORTED, "the gate must be fp32 or bf16");
    if (T == 0) return MOE_OK;
    if (!rows_ok(y, dtype, ld_y, D) || !rows_ok(res, res_dtype, ld_res, D) || !rows_ok(out, res_dtype, ld_out, D) ||
        (has_next && !rows_ok(next_out, next_dtype, ld_next, D)))
        return arg_fail(MOE_ERR_INVALID_ARG, "y, res, out or next_out NULL or misaligned, or a row stride below D");
    if (out == res && ld_out != ld_res) return arg_fail(MOE_ERR_INVALID_ARG, "out = res needs the same row stride");
    if (post->gate_by != MOE_GATE_NONE &&
        !rows_ok(post->gate, post->gate_dtype, post->gate_by == MOE_GATE_FULL ? post->ld_gate : D, D))
        return arg_fail(MOE_ERR_INVALID_ARG, "gate NULL or misaligned, or a row stride below D");
    p.T = T;
    p.D = D;
    p.res_scale = post->res_scale;
    p.branch_scale = post->branch_scale;
    p.gate_by = post->gate_by;
    p.gate_bf16 = post->gate_dtype == MOE_BF16;
    p.gate_sigmoid = post->gate_sigmoid != 0;
    p.gate = post->gate;
    p.ld_gate = post->ld_gate;
    p.y = y;
    p.y_elem = float_elem(dtype);
    p.ld_y = ld_y;
    p.res = res;
    p.out = out;
    p.r_elem = float_elem(res_dtype);
    p.ld_res = ld_res;
    p.ld_out = ld_out;
    p.next_out = next_out;
    p.n_elem = has_next ? float_elem(next_dtype) : moe::kBF16;
    p.ld_next = ld_next;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_norm_post(p, (cudaStream_t)stream));
    return MOE_OK;
}

namespace {
moe_status check_mx(const void* x, int32_t dtype, int64_t ld, int64_t rows, int32_t cols, const void* q, const void* s) {
    if (rows < 0 || cols < 1) return arg_fail(MOE_ERR_INVALID_ARG, "rows < 0 or cols < 1");
    if (cols > (1 << 30)) return arg_fail(MOE_ERR_UNSUPPORTED, "cols above 2^30");
    if (!float_type(dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "values must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(x, dtype, ld, cols)) return arg_fail(MOE_ERR_INVALID_ARG, "values NULL or misaligned, or a row stride below cols");
    if (!ptr_ok(q) || !s) return arg_fail(MOE_ERR_INVALID_ARG, "codes NULL or misaligned, or scales NULL");
    return MOE_OK;
}
}  // namespace

moe_status moe_mx_quantize(const void* x, int32_t dtype, int64_t ld_x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* s,
                           void* stream) {
    const moe_status st = check_mx(x, dtype, ld_x, rows, cols, q, s);
    if (st != MOE_OK || rows == 0) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_mx_quantize(x, float_elem(dtype), ld_x, rows, cols, q, s, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int32_t cols, void* out, int32_t out_dtype,
                             int64_t ld_out, void* stream) {
    const moe_status st = check_mx(out, out_dtype, ld_out, rows, cols, q, s);
    if (st != MOE_OK || rows == 0) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_mx_dequantize(q, s, rows, cols, out, float_elem(out_dtype), ld_out, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_mx_gemm(const uint8_t* a, const uint8_t* a_scale, const uint8_t* b, const uint8_t* b_scale,
                       const int32_t* offsets, int32_t rows, int32_t G, int32_t N, int32_t K, void* out, int32_t out_dtype,
                       int64_t ld_out, uint32_t* err, void* stream) {
    if (rows < 0 || G < 1 || N < 1 || K < 1) return arg_fail(MOE_ERR_INVALID_ARG, "rows < 0, or G, N or K < 1");
    if (!offsets && G != 1) return arg_fail(MOE_ERR_INVALID_ARG, "offsets NULL with several groups");
    if (K % 32 || G > 1025 || N > (1 << 20) || K > (1 << 20) || (int64_t)G * N >= ((int64_t)1 << 31) || rows > (1 << 30))
        return arg_fail(MOE_ERR_UNSUPPORTED, "K not a multiple of 32, G above 1025, N or K above 2^20, G*N above 2^31 or rows above 2^30");
    if (!float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "out must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!ptr_ok(a) || !ptr_ok(b) || !a_scale || !b_scale) return arg_fail(MOE_ERR_INVALID_ARG, "operand NULL or misaligned");
    if (!rows_ok(out, out_dtype, ld_out, N) || !aligned(offsets, 4) || !aligned(err, 4))
        return arg_fail(MOE_ERR_INVALID_ARG, "out NULL or misaligned or its row stride below N, or offsets or err misaligned");
    int dev = 0;
    MOE_CUDA(cudaGetDevice(&dev));
    static const char key = 0;
    int sms = 0;
    MOE_CUDA(moe::per_device_value(&key, [dev](int* v) { return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev); }, &sms));
    moe::MxGemm g = {};
    g.a = a;
    g.a_scale = a_scale;
    g.b = b;
    g.b_scale = b_scale;
    g.offsets = offsets;
    g.rows = rows;
    g.G = G;
    g.N = N;
    g.K = K;
    g.out = out;
    g.out_elem = float_elem(out_dtype);
    g.ldo = ld_out;
    g.err = err;
    g.spin_ns = kDefaultSpinNs;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_gemm_mx(g, sms, (cudaStream_t)stream));
    return MOE_OK;
}

// ------------------------------------------------- experts' products

namespace {
moe_status current_sms(int* sms) {
    int dev = 0;
    MOE_CUDA(cudaGetDevice(&dev));
    static const char key = 0;
    MOE_CUDA(moe::per_device_value(&key, [dev](int* v) { return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev); }, sms));
    return MOE_OK;
}

moe_status check_groups(const int32_t* offsets, int32_t rows, int32_t G, int32_t N, int32_t K, const uint32_t* err) {
    if (rows < 0 || G < 1 || N < 1 || K < 1) return arg_fail(MOE_ERR_INVALID_ARG, "rows < 0, or G, N or K < 1");
    if (!offsets && G != 1) return arg_fail(MOE_ERR_INVALID_ARG, "offsets NULL with several groups");
    if (G > moe::kProductMaxG || N > (1 << 20) || K > (1 << 20) || rows > (1 << 30))
        return arg_fail(MOE_ERR_UNSUPPORTED, "G above 1025, N or K above 2^20 or rows above 2^30");
    if (!aligned(offsets, 4) || !aligned(err, 4)) return arg_fail(MOE_ERR_INVALID_ARG, "offsets or err misaligned");
    return MOE_OK;
}

// Few rows a group, so that the weights' bytes bound: the kernels that take
// eight rows at a time against the tensor-memory ones, us.  bf16 1024 x 4096:
// 64 groups of 8 rows 79 against 89, of 12 rows 103 against 89; one matrix, 16
// rows 5.6 against 6.7, 32 rows 6.2 against 6.9.  4 bits: 64 groups of 8 rows
// 55 against 87, of 16 rows 103 against 87; one matrix, 32 rows 6.5 against 9.7.
bool few_rows(int64_t rows, int64_t G) { return rows <= 8 * G || rows <= 32; }

moe_status run_product(moe::GroupProduct& g, int32_t dtype, int32_t out_dtype, void* stream) {
    g.elem = float_elem(dtype);
    g.out_elem = float_elem(out_dtype);
    g.spin_ns = kDefaultSpinNs;
    int sms = 0;
    const moe_status st = current_sms(&sms);
    if (st != MOE_OK) return st;
    moe::PdlScope scope(true);
    cudaError_t e = cudaErrorNotSupported;
    if (few_rows(g.rows, g.G)) e = moe::launch_product_few(g, sms, (cudaStream_t)stream);
    if (e == cudaErrorNotSupported)
        e = g.elem == moe::kBF16 ? moe::launch_product_tc(g, sms, (cudaStream_t)stream) : moe::launch_product_f32(g, sms, (cudaStream_t)stream);
    MOE_CUDA(e);
    return MOE_OK;
}

// out = rows of `in` columns times the groups' weights, in `op`'s direction.
moe_status rows_product(int op, const void* a, int64_t ld_a, int32_t in, const void* w, int32_t dtype, const int32_t* offsets, int32_t rows,
                        int32_t G, int32_t N, int32_t K, void* out, int32_t out_dtype, int64_t ld_out, uint32_t* err, void* stream) {
    const moe_status st = check_groups(offsets, rows, G, N, K, err);
    if (st != MOE_OK) return st;
    if (!float_type(dtype) || !float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "operands and out must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(a, dtype, ld_a, in) || !rows_ok(w, dtype, K, K))
        return arg_fail(MOE_ERR_INVALID_ARG, "operand NULL or misaligned, or a row stride below its columns");
    if (!rows_ok(out, out_dtype, ld_out, N + K - in)) return arg_fail(MOE_ERR_INVALID_ARG, "out NULL or misaligned, or its row stride too small");
    moe::GroupProduct g = {};
    g.op = op;
    g.a = a;
    g.lda = ld_a;
    g.b = w;
    g.ldb = K;
    g.offsets = offsets;
    g.rows = rows;
    g.G = G;
    g.N = N;
    g.K = K;
    g.out = out;
    g.ldo = ld_out;
    g.err = err;
    return run_product(g, dtype, out_dtype, stream);
}
}  // namespace

moe_status moe_grouped_gemm(const void* x, int64_t ld_x, const void* w, int32_t dtype, const int32_t* offsets, int32_t rows, int32_t G,
                            int32_t N, int32_t K, void* out, int32_t out_dtype, int64_t ld_out, uint32_t* err, void* stream) {
    return rows_product(moe::kProductFwd, x, ld_x, K, w, dtype, offsets, rows, G, N, K, out, out_dtype, ld_out, err, stream);
}

moe_status moe_grouped_gemm_dx(const void* dy, int64_t ld_dy, const void* w, int32_t dtype, const int32_t* offsets, int32_t rows, int32_t G,
                               int32_t N, int32_t K, void* dx, int32_t out_dtype, int64_t ld_dx, uint32_t* err, void* stream) {
    return rows_product(moe::kProductDx, dy, ld_dy, N, w, dtype, offsets, rows, G, N, K, dx, out_dtype, ld_dx, err, stream);
}

moe_status moe_grouped_gemm_dw(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int32_t dtype, const int32_t* offsets,
                               int32_t rows, int32_t G, int32_t N, int32_t K, void* dw, int32_t out_dtype, int32_t accumulate, uint32_t* err,
                               void* stream) {
    const moe_status st = check_groups(offsets, rows, G, N, K, err);
    if (st != MOE_OK) return st;
    if (!float_type(dtype) || !float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "operands and dw must be fp32 or bf16");
    if (rows > 0 && (!rows_ok(dy, dtype, ld_dy, N) || !rows_ok(x, dtype, ld_x, K)))
        return arg_fail(MOE_ERR_INVALID_ARG, "dy or x NULL or misaligned, or a row stride below its columns");
    if (!rows_ok(dw, out_dtype, K, K)) return arg_fail(MOE_ERR_INVALID_ARG, "dw NULL or misaligned");
    moe::GroupProduct g = {};
    g.op = moe::kProductDw;
    g.a = dy;
    g.lda = ld_dy;
    g.b = x;
    g.ldb = ld_x;
    g.offsets = offsets;
    g.rows = rows;
    g.G = G;
    g.N = N;
    g.K = K;
    g.out = dw;
    g.ldo = K;
    g.accumulate = accumulate != 0;
    g.err = err;
    return run_product(g, dtype, out_dtype, stream);
}

namespace {
moe_status check_act(int32_t dtype, int32_t rows, int32_t I, const void* gate, int64_t ld_gate, const void* up, int64_t ld_up,
                     const float* weight) {
    if (rows < 0 || I < 1) return arg_fail(MOE_ERR_INVALID_ARG, "rows < 0 or I < 1");
    if (I > (1 << 20)) return arg_fail(MOE_ERR_UNSUPPORTED, "I above 2^20");
    if (!float_type(dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "gate and up must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(gate, dtype, ld_gate, I) || !rows_ok(up, dtype, ld_up, I) || !aligned(weight, 4))
        return arg_fail(MOE_ERR_INVALID_ARG, "gate or up NULL or misaligned, a row stride below I, or weight misaligned");
    return MOE_OK;
}
}  // namespace

moe_status moe_swiglu(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int32_t dtype, const float* weight, int32_t rows,
                      int32_t I, void* out, int32_t out_dtype, int64_t ld_out, void* stream) {
    moe_status st = check_act(dtype, rows, I, gate, ld_gate, up, ld_up, weight);
    if (st != MOE_OK) return st;
    if (!float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "out must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(out, out_dtype, ld_out, I)) return arg_fail(MOE_ERR_INVALID_ARG, "out NULL or misaligned, or its row stride below I");
    moe::ActParams p = {};
    p.rows = rows;
    p.I = I;
    p.elem = float_elem(dtype);
    p.out_elem = float_elem(out_dtype);
    p.gate = gate;
    p.up = up;
    p.ld_gate = ld_gate;
    p.ld_up = ld_up;
    p.weight = weight;
    p.out = out;
    p.ld_out = ld_out;
    int sms = 0;
    if ((st = current_sms(&sms)) != MOE_OK) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_swiglu(p, sms, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_swiglu_grad(const void* dh, int64_t ld_dh, const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int32_t dtype,
                           const float* weight, int32_t rows, int32_t I, void* dgate, int64_t ld_dgate, void* dup, int64_t ld_dup,
                           float* dweight, void* stream) {
    moe_status st = check_act(dtype, rows, I, gate, ld_gate, up, ld_up, weight);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!rows_ok(dh, dtype, ld_dh, I) || !rows_ok(dgate, dtype, ld_dgate, I) || !rows_ok(dup, dtype, ld_dup, I) || !aligned(dweight, 4))
        return arg_fail(MOE_ERR_INVALID_ARG, "dh, dgate or dup NULL or misaligned, a row stride below I, or dweight misaligned");
    moe::ActParams p = {};
    p.rows = rows;
    p.I = I;
    p.elem = p.out_elem = float_elem(dtype);
    p.gate = gate;
    p.up = up;
    p.dh = dh;
    p.ld_gate = ld_gate;
    p.ld_up = ld_up;
    p.ld_dh = ld_dh;
    p.weight = weight;
    p.dgate = dgate;
    p.dup = dup;
    p.ld_dgate = ld_dgate;
    p.ld_dup = ld_dup;
    p.dweight = dweight;
    int sms = 0;
    if ((st = current_sms(&sms)) != MOE_OK) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_swiglu_grad(p, sms, (cudaStream_t)stream));
    return MOE_OK;
}

namespace {
// Codes of rows of cols columns (at least one row).
moe_status check_int4(const uint8_t* codes, const void* scales, int32_t scale_dtype, int32_t group, int32_t cols, bool used) {
    if (cols < 1) return arg_fail(MOE_ERR_INVALID_ARG, "columns < 1");
    if (cols % 32 || cols > (1 << 20)) return arg_fail(MOE_ERR_UNSUPPORTED, "columns no multiple of 32, or above 2^20");
    if (group != 32 && group != 64 && group != 128) return arg_fail(MOE_ERR_UNSUPPORTED, "groups of 32, 64 or 128 columns");
    if (!float_type(scale_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "scales must be fp32 or bf16");
    if (used && (!ptr_ok(codes) || !rows_ok(scales, scale_dtype, 1, 1)))
        return arg_fail(MOE_ERR_INVALID_ARG, "codes or scales NULL or misaligned");
    return MOE_OK;
}
moe::Int4 int4_of(const uint8_t* codes, const void* scales, int32_t scale_dtype, const uint8_t* zeros, int32_t group) {
    moe::Int4 q = {};
    q.codes = codes;
    q.scales = scales;
    q.scale_elem = float_elem(scale_dtype);
    q.zeros = zeros;
    q.group = group;
    return q;
}
}  // namespace

moe_status moe_int4_quantize(const void* x, int32_t dtype, int64_t ld_x, int64_t rows, int32_t cols, int32_t group, uint8_t* codes,
                             void* scales, int32_t scale_dtype, uint8_t* zeros, void* stream) {
    if (rows < 0) return arg_fail(MOE_ERR_INVALID_ARG, "rows < 0");
    moe_status st = check_int4(codes, scales, scale_dtype, group, cols, rows > 0);
    if (st != MOE_OK) return st;
    if (!float_type(dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "values must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(x, dtype, ld_x, cols)) return arg_fail(MOE_ERR_INVALID_ARG, "values NULL or misaligned, or a row stride below cols");
    int sms = 0;
    if ((st = current_sms(&sms)) != MOE_OK) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_int4_quantize(x, float_elem(dtype), ld_x, rows, cols, int4_of(codes, scales, scale_dtype, zeros, group), sms,
                                       (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_int4_dequantize(const uint8_t* codes, const void* scales, int32_t scale_dtype, const uint8_t* zeros, int32_t group,
                               int64_t rows, int32_t cols, void* out, int32_t out_dtype, int64_t ld_out, void* stream) {
    if (rows < 0) return arg_fail(MOE_ERR_INVALID_ARG, "rows < 0");
    moe_status st = check_int4(codes, scales, scale_dtype, group, cols, rows > 0);
    if (st != MOE_OK) return st;
    if (!float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "out must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(out, out_dtype, ld_out, cols)) return arg_fail(MOE_ERR_INVALID_ARG, "out NULL or misaligned, or its row stride below cols");
    int sms = 0;
    if ((st = current_sms(&sms)) != MOE_OK) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(moe::launch_int4_dequantize(int4_of(codes, scales, scale_dtype, zeros, group), rows, cols, out, float_elem(out_dtype), ld_out, sms,
                                         (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_int4_gemm(const void* x, int32_t dtype, int64_t ld_x, const uint8_t* codes, const void* scales, int32_t scale_dtype,
                         const uint8_t* zeros, int32_t group, const int32_t* offsets, int32_t rows, int32_t G, int32_t N, int32_t K,
                         void* out, int32_t out_dtype, int64_t ld_out, uint32_t* err, void* stream) {
    moe_status st = check_groups(offsets, rows, G, N, K, err);
    if (st != MOE_OK || (st = check_int4(codes, scales, scale_dtype, group, K, rows > 0)) != MOE_OK) return st;
    if (!float_type(dtype) || !float_type(out_dtype)) return arg_fail(MOE_ERR_UNSUPPORTED, "x and out must be fp32 or bf16");
    if (rows == 0) return MOE_OK;
    if (!rows_ok(x, dtype, ld_x, K)) return arg_fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned, or its row stride below K");
    if (!rows_ok(out, out_dtype, ld_out, N)) return arg_fail(MOE_ERR_INVALID_ARG, "out NULL or misaligned, or its row stride below N");
    moe::Int4Product g = {};
    g.x = x;
    g.elem = float_elem(dtype);
    g.ldx = ld_x;
    g.w = int4_of(codes, scales, scale_dtype, zeros, group);
    g.offsets = offsets;
    g.rows = rows;
    g.G = G;
    g.N = N;
    g.K = K;
    g.out = out;
    g.out_elem = float_elem(out_dtype);
    g.ldo = ld_out;
    g.err = err;
    g.spin_ns = kDefaultSpinNs;
    int sms = 0;
    if ((st = current_sms(&sms)) != MOE_OK) return st;
    moe::PdlScope scope(true);
    MOE_CUDA(g.elem == moe::kBF16 && !few_rows(rows, G) ? moe::launch_int4_tc(g, sms, (cudaStream_t)stream)
                                                       : moe::launch_int4_few(g, sms, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_pointer_kind(const void* ptr, int32_t* kind) {
    if (!kind) return arg_fail(MOE_ERR_INVALID_ARG, "kind is NULL");
    *kind = 0;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
        cudaGetLastError();  // unregistered host memory on older drivers
        return MOE_OK;
    }
    switch (a.type) {
        case cudaMemoryTypeDevice: *kind = 2; break;
        case cudaMemoryTypeManaged: *kind = 3; break;
        case cudaMemoryTypeHost: *kind = (a.devicePointer == ptr) ? 1 : 0; break;
        default: *kind = 0; break;
    }
    return MOE_OK;
}

moe_status moe_convert_down_weights(const moe_plan* p, const void* w_down, void* w_down_f16, void* ws,
                                   size_t ws_bytes, void* stream) {
    if (!p) return arg_fail(MOE_ERR_INVALID_ARG, "plan is NULL");
    if (p->cfg.dtype != MOE_BF16) return arg_fail(MOE_ERR_UNSUPPORTED, "only the bf16 layer has an fp16 W_down copy");
    if (!ptr_ok(w_down) || !ptr_ok(w_down_f16)) return arg_fail(MOE_ERR_INVALID_ARG, "NULL or misaligned pointer");
    if (!ws || !aligned(ws, 256) || ws_bytes < 256) return arg_fail(MOE_ERR_INVALID_ARG, "workspace");
    const int64_t n = (int64_t)(p->cfg.E + 1) * p->cfg.D * p->cfg.I;
    MOE_CUDA(moe::launch_bf16_to_f16(w_down, w_down_f16, n, (uint32_t*)ws, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_pack_routing_words(const moe_plan* p, int32_t T, const void* ws, size_t ws_bytes, int32_t* words,
                                  void* stream) {
    Ws W;
    moe_status st = check_call(p, T, const_cast<void*>(ws), ws_bytes, &W);
    if (st != MOE_OK) return st;
    if (!ptr_ok(words)) return arg_fail(MOE_ERR_INVALID_ARG, "words NULL or misaligned");
    MOE_CUDA(moe::launch_pack_words(W.at<int32_t>(W.L.blob), (int64_t)T * p->cfg.top_k, words, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_check(const moe_plan* p, const void* ws, void* stream) {
    if (!p || !ws) return arg_fail(MOE_ERR_INVALID_ARG, "NULL argument");
    uint32_t word[4] = {0, 0, 0, 0};
    MOE_CUDA(cudaStreamSynchronize((cudaStream_t)stream));
    MOE_CUDA(cudaMemcpy(word, ws, sizeof(word), cudaMemcpyDeviceToHost));
    if (word[0] != 0) {
        snprintf(g_detail, sizeof(g_detail), "device error %u (%s), info %u %u %u", word[0],
                 moe_status_str((moe_status)word[0]), word[1], word[2], word[3]);
        return (moe_status)word[0];
    }
    return MOE_OK;
}

moe_status moe_selftest_wait_timeout(const moe_plan* p, void* ws, size_t ws_bytes, int64_t limit_ns, void* stream) {
    if (!p || !ws || !aligned(ws, 256) || ws_bytes < 256) return arg_fail(MOE_ERR_INVALID_ARG, "workspace");
    if (limit_ns < 0 || limit_ns > 10000000000LL) return arg_fail(MOE_ERR_INVALID_ARG, "limit_ns outside [0, 10 s]");
    MOE_CUDA(moe::launch_selftest_timeout((uint32_t*)ws, limit_ns, (cudaStream_t)stream));
    return MOE_OK;
}

}  // extern "C"
