// api.cu: the extern "C" boundary of the selector library (declared in include/dflash.h).
//
// This file validates arguments on the host, finds the device facts the launchers need,
// owns the device status word, and runs the fused selector and its stage tracing. All
// arithmetic of the method lives in topk.cu, projection.cu and edges.cu.
#include "dflash.h"
#include "common.cuh"
#include "ptx.cuh"

#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>
#include <vector>

namespace {

// In the fused selector, a projection of more than this many FLOPs is launched before the
// top-k, a smaller one after it (see dflash_selector). The measured cases on either side:
// 3.8 GFLOP (gemma_softcap) and 21.1 GFLOP (gemma_large).
constexpr double kProjectionFirstFlops = 8e9;

thread_local std::string g_last_error;

dflash_status fail(dflash_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

dflash_status ok() {
    g_last_error.clear();
    return DFLASH_OK;
}

dflash_status cuda_fail(cudaError_t e, const char* what) {
    return fail(DFLASH_CUDA_ERROR, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bits the kernels set on problems they detect; read through dflash_device_status.
__device__ uint32_t g_device_status;

// Zeroed scratch of dflash_selftest_wait_timeout's queue check (1 KB).
__device__ __align__(16) uint32_t g_selftest_buffer[256];

constexpr int kMaxDevices = 64;
struct DeviceSlot {
    dflash::DeviceInfo info;
    uint32_t* status_word = nullptr;
    bool ready = false;
};

std::mutex g_dev_mu;
DeviceSlot g_dev[kMaxDevices];

// Facts about the current device, looked up once per device.
dflash_status current_device(dflash::DeviceInfo* info, uint32_t** status_word) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DFLASH_NO_DEVICE, "no CUDA device: %s", cudaGetErrorString(e));
    }
    if (dev < 0 || dev >= kMaxDevices) return fail(DFLASH_NO_DEVICE, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_dev_mu);
    DeviceSlot& s = g_dev[dev];
    if (!s.ready) {
        cudaDeviceProp prop;
        e = cudaGetDeviceProperties(&prop, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDeviceProperties");
        if (prop.major != 10 || prop.minor != 3)
            return fail(DFLASH_NO_DEVICE,
                        "device %d is sm_%d%d; this library is built for sm_103a (GB300)", dev,
                        prop.major, prop.minor);
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_device_status);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status word)");
        s.info.device = dev;
        s.info.sm_count = prop.multiProcessorCount;
        s.info.cc_major = prop.major;
        s.info.cc_minor = prop.minor;
        s.info.smem_optin = prop.sharedMemPerBlockOptin;
        s.status_word = static_cast<uint32_t*>(p);
        s.ready = true;
    }
    if (info) *info = s.info;
    if (status_word) *status_word = s.status_word;
    return DFLASH_OK;
}

// ---------------------------------------------------------------- argument checks

dflash_status check_dims_topk(int R, int S, int V, int K) {
    if (R < 1 || S < 1 || V < 1 || K < 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R, S, V and K must be >= 1 (got R=%d S=%d V=%d K=%d)",
                    R, S, V, K);
    if (K > V) return fail(DFLASH_INVALID_ARGUMENT, "K=%d exceeds V=%d", K, V);
    if (K > 32) return fail(DFLASH_UNSUPPORTED, "K=%d: top-k supports K <= 32", K);
    if ((long long)R * S > (1LL << 31) - 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R*S=%lld rows exceeds 2^31-1", (long long)R * S);
    return DFLASH_OK;
}

dflash_status check_rank(int rank) {
    if (rank < 1) return fail(DFLASH_INVALID_ARGUMENT, "rank=%d must be >= 1", rank);
    if (rank % 8 != 0 || rank > 256)
        return fail(DFLASH_UNSUPPORTED, "rank=%d: supported ranks are multiples of 8 up to 256", rank);
    return DFLASH_OK;
}

dflash_status check_dims_projection(int R, int S, int H, int rank) {
    if (R < 1 || S < 1 || H < 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R, S and H must be >= 1 (got R=%d S=%d H=%d)", R, S, H);
    if (H % 8 != 0) return fail(DFLASH_UNSUPPORTED, "H=%d: must be a multiple of 8", H);
    if ((long long)R * S > (1LL << 31) - 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R*S=%lld rows exceeds 2^31-1", (long long)R * S);
    return check_rank(rank);
}

dflash_status check_dims_edges(int R, int S, int K, int V, int rank) {
    if (R < 1 || S < 1 || V < 1 || K < 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R, S, V and K must be >= 1 (got R=%d S=%d V=%d K=%d)",
                    R, S, V, K);
    if (K > V) return fail(DFLASH_INVALID_ARGUMENT, "K=%d exceeds V=%d", K, V);
    if (K > 32) return fail(DFLASH_UNSUPPORTED, "K=%d: edges support K <= 32", K);
    if ((long long)R * S > (1LL << 31) - 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R*S=%lld rows exceeds 2^31-1", (long long)R * S);
    return check_rank(rank);
}

dflash_status check_processor(float softcap, float scale) {
    if (!(softcap >= 0.f) || isinf(softcap))
        return fail(DFLASH_INVALID_ARGUMENT, "softcap=%g must be finite and >= 0 (0 = no cap)",
                    (double)softcap);
    if (!(scale > 0.f) || isinf(scale))
        return fail(DFLASH_INVALID_ARGUMENT, "scale=%g must be finite and > 0", (double)scale);
    return DFLASH_OK;
}

dflash_status check_ptr(const void* p, const char* name) {
    if (!p) return fail(DFLASH_INVALID_ARGUMENT, "%s is NULL", name);
    if (!aligned16(p)) return fail(DFLASH_INVALID_ARGUMENT, "%s is not 16-byte aligned", name);
    return DFLASH_OK;
}

// For the arrays that need only their natural 4-byte alignment: the anchors, candidate ids,
// unary values, edge scores and best-path outputs (read and written one element at a time,
// or staged with copies as wide as their alignment allows) and the logits (the top-k finds
// the 16-byte boundaries itself), so a slice of requests out of larger arrays stays valid.
dflash_status check_ptr4(const void* p, const char* name) {
    if (!p) return fail(DFLASH_INVALID_ARGUMENT, "%s is NULL", name);
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0)
        return fail(DFLASH_INVALID_ARGUMENT, "%s is not 4-byte aligned", name);
    return DFLASH_OK;
}

// For 8-byte elements.
dflash_status check_ptr8(const void* p, const char* name) {
    if (!p) return fail(DFLASH_INVALID_ARGUMENT, "%s is NULL", name);
    if ((reinterpret_cast<uintptr_t>(p) & 7u) != 0)
        return fail(DFLASH_INVALID_ARGUMENT, "%s is not 8-byte aligned", name);
    return DFLASH_OK;
}

#define DFLASH_TRY(expr)                     \
    do {                                     \
        dflash_status _s = (expr);           \
        if (_s != DFLASH_OK) return _s;      \
    } while (0)

// A stride in elements that keeps rows aligned for loads of 8 elements. A dimension of one element
// is never stepped along, whatever its stride.
dflash_status check_stride(long long stride, int dim, int multiple, const char* name) {
    if (dim == 1) return DFLASH_OK;
    if (stride < 0) return fail(DFLASH_INVALID_ARGUMENT, "%s=%lld must be >= 0", name, stride);
    if (stride % multiple != 0)
        return fail(DFLASH_UNSUPPORTED, "%s=%lld: must be a multiple of %d elements", name, stride,
                    multiple);
    return DFLASH_OK;
}

// Checks a dflash_kv_cache whose users have queries, or new keys and values, of type dtype.
dflash_status check_cache(const dflash_kv_cache* c, int dtype, dflash::KvCache* out) {
    if (!c) return fail(DFLASH_INVALID_ARGUMENT, "cache is NULL");
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP16)
        return fail(DFLASH_INVALID_ARGUMENT, "dtype=%d: must be DFLASH_BF16 or DFLASH_FP16", dtype);
    if (c->dtype != dtype && c->dtype != DFLASH_E4M3)
        return fail(DFLASH_INVALID_ARGUMENT, "cache dtype=%d: must be dtype=%d or DFLASH_E4M3",
                    c->dtype, dtype);
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1)
        return fail(DFLASH_INVALID_ARGUMENT,
                    "num_pages, page_size, kv_heads and head_dim must be >= 1 (got %d, %d, %d, %d)",
                    c->num_pages, c->page_size, c->kv_heads, c->head_dim);
    const int mult = c->dtype == DFLASH_E4M3 ? 16 : 8;
    if (c->head_dim % mult != 0 || c->head_dim > 256)
        return fail(DFLASH_UNSUPPORTED, "head_dim=%d: must be a multiple of %d up to 256",
                    c->head_dim, mult);
    DFLASH_TRY(check_stride(c->page_stride, c->num_pages, mult, "page_stride"));
    DFLASH_TRY(check_stride(c->token_stride, c->page_size, mult, "token_stride"));
    DFLASH_TRY(check_stride(c->head_stride, c->kv_heads, mult, "head_stride"));
    if (!(c->k_scale > 0.f) || isinf(c->k_scale) || !(c->v_scale > 0.f) || isinf(c->v_scale))
        return fail(DFLASH_INVALID_ARGUMENT, "k_scale=%g and v_scale=%g must be finite and > 0",
                    (double)c->k_scale, (double)c->v_scale);
    if (c->dtype != DFLASH_E4M3 && (c->k_scale != 1.f || c->v_scale != 1.f))
        return fail(DFLASH_INVALID_ARGUMENT, "k_scale and v_scale must be 1 without DFLASH_E4M3");
    DFLASH_TRY(check_ptr(c->key, "cache key"));
    DFLASH_TRY(check_ptr(c->value, "cache value"));
    *out = dflash::KvCache{c->key, c->value, c->page_stride, c->token_stride, c->head_stride,
                           c->num_pages, c->page_size, c->kv_heads, c->head_dim, c->dtype,
                           c->k_scale, c->v_scale};
    return DFLASH_OK;
}

// The strides of queries, keys or values, or of their outputs.
dflash_status check_row_strides(long long token, int T, long long head, int heads, const char* token_name,
                                const char* head_name) {
    DFLASH_TRY(check_stride(token, T, 8, token_name));
    DFLASH_TRY(check_stride(head, heads, 8, head_name));
    if ((T != 1 && token > INT_MAX) || (heads != 1 && head > INT_MAX))
        return fail(DFLASH_UNSUPPORTED, "%s=%lld and %s=%lld must be below 2^31", token_name, token, head_name,
                    head);
    return DFLASH_OK;
}

// Checks a dflash_norm_rope and the sizes and strides of the calls that take one; fills in what it says.
dflash_status check_norm_rope(const dflash_norm_rope* how, dflash::NormRopeArgs* a) {
    if (!how) return fail(DFLASH_INVALID_ARGUMENT, "how is NULL");
    if (a->dtype != DFLASH_BF16 && a->dtype != DFLASH_FP16)
        return fail(DFLASH_INVALID_ARGUMENT, "dtype=%d: must be DFLASH_BF16 or DFLASH_FP16", a->dtype);
    if (a->T < 0) return fail(DFLASH_INVALID_ARGUMENT, "T=%d must be >= 0", a->T);
    if (a->head_dim < 1) return fail(DFLASH_INVALID_ARGUMENT, "head_dim=%d must be >= 1", a->head_dim);
    if (a->head_dim % 8 != 0 || a->head_dim > 256)
        return fail(DFLASH_UNSUPPORTED, "head_dim=%d: must be a multiple of 8 up to 256", a->head_dim);
    if (a->q_heads + 2LL * a->kv_heads > (1 << 24) ||
        a->T * (a->q_heads + 2LL * a->kv_heads) > (1LL << 31) - 1)
        return fail(DFLASH_INVALID_ARGUMENT, "T=%d tokens of %d and %d heads are more than 2^31-1 rows",
                    a->T, a->q_heads, a->kv_heads);
    if (how->rotary_dim < 0 || how->rotary_dim % 2 != 0 || how->rotary_dim > a->head_dim)
        return fail(DFLASH_INVALID_ARGUMENT, "rotary_dim=%d must be even, from 0 to head_dim=%d",
                    how->rotary_dim, a->head_dim);
    if (!(how->eps >= 0.f) || isinf(how->eps))
        return fail(DFLASH_INVALID_ARGUMENT, "eps=%g must be finite and >= 0", (double)how->eps);
    if (!isfinite(how->rope_scale))
        return fail(DFLASH_INVALID_ARGUMENT, "rope_scale=%g must be finite", (double)how->rope_scale);
    if ((how->q_weight || how->k_weight) && how->weight_dtype != a->dtype &&
        how->weight_dtype != DFLASH_FP32)
        return fail(DFLASH_INVALID_ARGUMENT, "weight_dtype=%d: must be dtype=%d or DFLASH_FP32",
                    how->weight_dtype, a->dtype);
    if (a->q_heads > 0) {
        DFLASH_TRY(check_row_strides(a->qt, a->T, a->qh, a->q_heads, "q_token_stride", "q_head_stride"));
        DFLASH_TRY(check_row_strides(a->qot, a->T, a->qoh, a->q_heads, "q_out_token_stride",
                                     "q_out_head_stride"));
    }
    if (a->kv_heads > 0)
        DFLASH_TRY(check_row_strides(a->kt, a->T, a->kh, a->kv_heads, "k_token_stride", "k_head_stride"));
    a->q_weight = how->q_weight;
    a->k_weight = how->k_weight;
    a->weight_dtype = how->weight_dtype;
    a->eps = how->eps;
    a->frequencies = how->frequencies;
    a->rotary_dim = how->rotary_dim;
    a->interleaved = how->interleaved != 0;
    a->rope_scale = how->rope_scale;
    return DFLASH_OK;
}

// The pointers of such a call with any tokens.
dflash_status check_norm_rope_pointers(const dflash::NormRopeArgs& a) {
    if (a.q_heads > 0) {
        DFLASH_TRY(check_ptr(a.query, "query"));
        DFLASH_TRY(check_ptr(a.query_out, "query_out"));
    }
    if (a.kv_heads > 0) DFLASH_TRY(check_ptr(a.key, "key"));
    if (a.q_weight) DFLASH_TRY(check_ptr(a.q_weight, "q_weight"));
    if (a.k_weight) DFLASH_TRY(check_ptr(a.k_weight, "k_weight"));
    if (a.rotary_dim > 0) {
        DFLASH_TRY(check_ptr4(a.positions, "positions"));
        DFLASH_TRY(check_ptr8(a.frequencies, "frequencies"));
    }
    return DFLASH_OK;
}

// One temperature for all requests; with one for each it is not looked at.
dflash_status check_temperature(const float* temperatures, float temperature) {
    if (temperatures) return check_ptr4(temperatures, "temperatures");
    if (!(temperature >= 0.f) || isinf(temperature))
        return fail(DFLASH_INVALID_ARGUMENT, "temperature=%g must be finite and >= 0",
                    (double)temperature);
    return DFLASH_OK;
}

// A named NVTX range around one library call (host side: it brackets the argument checks and
// the enqueue, and profilers attach the call's CUDA launches to it). Free when no tool is
// attached.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// ---------------------------------------------------------------- stage tracing

struct Trace {
    std::mutex mu;
    int device = -1;
    int capacity = 0;   // calls
    int used = 0;
    std::vector<cudaEvent_t> events;   // 4 per call
};
Trace g_trace;

// Event slots for the next traced call, or nullptr when tracing is off or full.
cudaEvent_t* trace_slot(int device) {
    std::lock_guard<std::mutex> lock(g_trace.mu);
    if (g_trace.capacity == 0 || g_trace.used >= g_trace.capacity || g_trace.device != device)
        return nullptr;
    return &g_trace.events[4 * (g_trace.used++)];
}

}  // namespace

extern "C" {

const char* dflash_version(void) { return "0.1.0"; }

const char* dflash_status_string(int status) {
    switch (status) {
        case DFLASH_OK: return "DFLASH_OK";
        case DFLASH_INVALID_ARGUMENT: return "DFLASH_INVALID_ARGUMENT";
        case DFLASH_UNSUPPORTED: return "DFLASH_UNSUPPORTED";
        case DFLASH_WORKSPACE_TOO_SMALL: return "DFLASH_WORKSPACE_TOO_SMALL";
        case DFLASH_CUDA_ERROR: return "DFLASH_CUDA_ERROR";
        case DFLASH_NO_DEVICE: return "DFLASH_NO_DEVICE";
        default: return "DFLASH_UNKNOWN_STATUS";
    }
}

const char* dflash_last_error(void) { return g_last_error.c_str(); }

size_t dflash_topk_workspace_bytes(int R, int S, int V, int K) {
    if (check_dims_topk(R, S, V, K) != DFLASH_OK) return 0;
    dflash::DeviceInfo dev;
    if (current_device(&dev, nullptr) != DFLASH_OK) return 0;
    return dflash::topk_plan(dev, (long long)R * S, V).workspace_bytes();
}

size_t dflash_selector_workspace_bytes(int R, int S, int V, int K) {
    if (check_dims_topk(R, S, V, K) != DFLASH_OK) return 0;
    dflash::DeviceInfo dev;
    if (current_device(&dev, nullptr) != DFLASH_OK) return 0;
    const long long rows = (long long)R * S;
    // The top-k's workspace with the edge tiles' ready queue between its counters and its
    // partial lists (zeroed together).
    return dflash::topk_plan(dev, rows, V).workspace_bytes() + dflash::edge_queue_bytes(rows);
}

dflash_status dflash_topk_candidates(const float* logits, int R, int S, int V, int K,
                                     float softcap, float scale, int32_t* cand_ids,
                                     float* unary, void* workspace, size_t workspace_bytes,
                                     dflash_stream_t stream) {
    NvtxRange range("dflash_topk_candidates");
    DFLASH_TRY(check_dims_topk(R, S, V, K));
    DFLASH_TRY(check_processor(softcap, scale));
    DFLASH_TRY(check_ptr4(logits, "logits"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    DFLASH_TRY(check_ptr(workspace, "workspace"));
    dflash::DeviceInfo dev;
    DFLASH_TRY(current_device(&dev, nullptr));
    const dflash::TopkPlan plan = dflash::topk_plan(dev, (long long)R * S, V);
    if (workspace_bytes < plan.workspace_bytes())
        return fail(DFLASH_WORKSPACE_TOO_SMALL, "workspace of %zu bytes; %zu needed",
                    workspace_bytes, plan.workspace_bytes());
    cudaError_t e = dflash::launch_topk(plan, logits, V, K, cand_ids, unary, workspace,
                                        reinterpret_cast<cudaStream_t>(stream), softcap, scale);
    if (e != cudaSuccess) return cuda_fail(e, "top-k launch");
    return ok();
}

dflash_status dflash_topk_candidates_noalloc(const float* logits, int R, int S, int V, int K,
                                             int32_t* cand_ids, float* unary,
                                             dflash_stream_t stream) {
    NvtxRange range("dflash_topk_candidates_noalloc");
    DFLASH_TRY(check_dims_topk(R, S, V, K));
    DFLASH_TRY(check_ptr4(logits, "logits"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    dflash::DeviceInfo dev;
    DFLASH_TRY(current_device(&dev, nullptr));
    const dflash::TopkPlan plan = dflash::topk_plan(dev, (long long)R * S, V);
    if (plan.workspace_bytes() > dflash::kStaticScratchBytes)
        return fail(DFLASH_UNSUPPORTED,
                    "R*S=%lld rows need %zu bytes of scratch; the built-in scratch holds %zu. "
                    "Use dflash_topk_candidates with a caller-owned workspace",
                    (long long)R * S, plan.workspace_bytes(), dflash::kStaticScratchBytes);
    void* scratch = nullptr;
    cudaError_t e = dflash::topk_static_scratch(dev.device, &scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(top-k scratch)");
    // launch_topk clears the arrival counters on the stream before the kernel runs.
    e = dflash::launch_topk(plan, logits, V, K, cand_ids, unary, scratch,
                            reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "top-k launch");
    return ok();
}

size_t dflash_lmhead_topk_workspace_bytes(int R, int S, int V, int K) {
    if (check_dims_topk(R, S, V, K) != DFLASH_OK) return 0;
    dflash::DeviceInfo dev;
    if (current_device(&dev, nullptr) != DFLASH_OK) return 0;
    return dflash::lmhead_plan(dev, (long long)R * S, V).workspace_bytes();
}

dflash_status dflash_lmhead_topk(const uint16_t* hidden, const uint16_t* lm_head, int R, int S,
                                 int H, int V, int K, float softcap, float scale,
                                 int32_t* cand_ids, float* unary, void* workspace,
                                 size_t workspace_bytes, dflash_stream_t stream) {
    NvtxRange range("dflash_lmhead_topk");
    DFLASH_TRY(check_dims_topk(R, S, V, K));
    DFLASH_TRY(check_processor(softcap, scale));
    if (H < 1) return fail(DFLASH_INVALID_ARGUMENT, "H=%d must be >= 1", H);
    if (H % 8 != 0) return fail(DFLASH_UNSUPPORTED, "H=%d: must be a multiple of 8", H);
    DFLASH_TRY(check_ptr(hidden, "hidden"));
    DFLASH_TRY(check_ptr(lm_head, "lm_head"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    DFLASH_TRY(check_ptr(workspace, "workspace"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    const dflash::LmheadPlan plan = dflash::lmhead_plan(dev, (long long)R * S, V);
    if (workspace_bytes < plan.workspace_bytes())
        return fail(DFLASH_WORKSPACE_TOO_SMALL, "workspace of %zu bytes; %zu needed",
                    workspace_bytes, plan.workspace_bytes());
    cudaError_t e = dflash::launch_lmhead_topk(dev, plan, hidden, lm_head, R * S, H, V, K, softcap,
                                               scale, cand_ids, unary, workspace, status,
                                               reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "LM-head top-k launch");
    return ok();
}

dflash_status dflash_hidden_projection(const uint16_t* hidden, const uint16_t* w_proj, int R,
                                       int S, int H, int rank, uint16_t* h_out,
                                       dflash_stream_t stream) {
    NvtxRange range("dflash_hidden_projection");
    DFLASH_TRY(check_dims_projection(R, S, H, rank));
    DFLASH_TRY(check_ptr(hidden, "hidden"));
    DFLASH_TRY(check_ptr(w_proj, "w_proj"));
    DFLASH_TRY(check_ptr(h_out, "h_out"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    cudaError_t e = dflash::launch_projection(dev, hidden, w_proj, R * S, H, rank, h_out, status,
                                              reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "projection launch");
    return ok();
}

dflash_status dflash_candidate_edges(const uint16_t* pred_cb, const uint16_t* succ_cb,
                                     const int32_t* cand_ids, const float* unary,
                                     const uint16_t* h, const int32_t* anchors, int R, int S,
                                     int K, int V, int rank, float* edges,
                                     dflash_stream_t stream) {
    NvtxRange range("dflash_candidate_edges");
    DFLASH_TRY(check_dims_edges(R, S, K, V, rank));
    DFLASH_TRY(check_ptr(pred_cb, "pred_cb"));
    DFLASH_TRY(check_ptr(succ_cb, "succ_cb"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    DFLASH_TRY(check_ptr(h, "h"));
    DFLASH_TRY(check_ptr4(anchors, "anchors"));
    DFLASH_TRY(check_ptr4(edges, "edges"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    cudaError_t e = dflash::launch_edges(dev, pred_cb, succ_cb, cand_ids, unary, h, anchors, R, S,
                                         K, V, rank, edges, status,
                                         reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "edges launch");
    return ok();
}

dflash_status dflash_selector(const float* logits, const uint16_t* hidden, const uint16_t* w_proj,
                              const uint16_t* pred_cb, const uint16_t* succ_cb,
                              const int32_t* anchors, int R, int S, int K, int V, int H, int rank,
                              float softcap, float scale, int32_t* cand_ids, float* unary,
                              uint16_t* h_out, float* edges, void* workspace,
                              size_t workspace_bytes, dflash_stream_t stream) {
    NvtxRange range("dflash_selector");
    DFLASH_TRY(check_dims_topk(R, S, V, K));
    DFLASH_TRY(check_processor(softcap, scale));
    DFLASH_TRY(check_dims_projection(R, S, H, rank));
    DFLASH_TRY(check_ptr4(logits, "logits"));
    DFLASH_TRY(check_ptr(hidden, "hidden"));
    DFLASH_TRY(check_ptr(w_proj, "w_proj"));
    DFLASH_TRY(check_ptr(pred_cb, "pred_cb"));
    DFLASH_TRY(check_ptr(succ_cb, "succ_cb"));
    DFLASH_TRY(check_ptr4(anchors, "anchors"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    DFLASH_TRY(check_ptr(h_out, "h_out"));
    DFLASH_TRY(check_ptr4(edges, "edges"));
    DFLASH_TRY(check_ptr(workspace, "workspace"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    const long long rows = (long long)R * S;
    const dflash::TopkPlan plan = dflash::topk_plan(dev, rows, V);
    const size_t qbytes = dflash::edge_queue_bytes(rows);
    if (workspace_bytes < plan.workspace_bytes() + qbytes)
        return fail(DFLASH_WORKSPACE_TOO_SMALL, "workspace of %zu bytes; %zu needed",
                    workspace_bytes, plan.workspace_bytes() + qbytes);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaEvent_t* ev = trace_slot(dev.device);
    // Workspace: the top-k's arrival counters, the edge tiles' ready queue, the top-k's partial
    // lists. The counters and the queue are zeroed first.
    dflash::EdgeQueue queue =
        dflash::edge_queue_at(static_cast<char*>(workspace) + plan.counter_bytes, rows, S);
    queue.proj_ctas = dflash::projection_ctas(dev, R * S, H, rank);
    // Schedule, one stream. Each kernel is the next one's programmatic dependent: it may start
    // once every CTA of the kernel before it has started, and takes only the resources that
    // kernel leaves. The edges come last and take the SMs that top-k CTAs leave as they
    // finish, each scoring a tile once the ready queue hands it over (its rows are written)
    // and the projection's count of finished CTAs is complete: most edges run in the top-k's
    // tail. The projection comes first when it is large (more than kProjectionFirstFlops):
    // it then runs beside the top-k (an SM holding a projection CTA takes one top-k CTA at
    // once and two more when the projection CTA ends: its shared-memory configuration leaves
    // room for only one more CTA) and h is ready long before the edges need it. A smaller
    // projection comes after the top-k instead and runs on the SMs the top-k's first finished
    // CTAs leave, so every top-k CTA starts at once. Measured on GB300 (same bits either way):
    // gemma_large (21.1 GFLOP of projection) 1174-1176 us projection first against 1205 us
    // after; gemma_softcap (3.8 GFLOP) 589-590 -> 585.5-585.7 us, qwen_zipf 122.7-123.0 ->
    // 119.1-119.4 us, small_ties 28.7-28.9 -> 27.2-27.5 us, tiny 17.4-18.7 -> 17.2 us with the
    // projection after the top-k. Either way every producer a wait depends on has all its CTAs
    // resident before any edge CTA exists, so nothing can stall. A traced call
    // (dflash_trace_begin) records events between the kernels, which then run one after
    // another in the first order, so that each can be timed.
    const bool chain = ev == nullptr;
    const double proj_flops = 2.0 * (double)rows * (double)H * (double)rank;
    const bool topk_first = chain && proj_flops <= kProjectionFirstFlops;
    cudaError_t e;
    if (ev && (e = cudaEventRecord(ev[0], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    if ((e = cudaMemsetAsync(workspace, 0, plan.counter_bytes + qbytes, st)) != cudaSuccess)
        return cuda_fail(e, "clearing the workspace");
    if (topk_first) {
        e = dflash::launch_topk(plan, logits, V, K, cand_ids, unary, workspace, st, softcap, scale,
                                qbytes, /*clear_counters=*/false, queue, /*programmatic=*/false);
        if (e != cudaSuccess) return cuda_fail(e, "top-k launch");
        e = dflash::launch_projection(dev, hidden, w_proj, R * S, H, rank, h_out, status, st,
                                      /*beside_topk=*/true, queue.proj_done,
                                      /*programmatic=*/true);
        if (e != cudaSuccess) return cuda_fail(e, "projection launch");
    } else {
        e = dflash::launch_projection(dev, hidden, w_proj, R * S, H, rank, h_out, status, st,
                                      /*beside_topk=*/true, queue.proj_done);
        if (e != cudaSuccess) return cuda_fail(e, "projection launch");
        if (ev && (e = cudaEventRecord(ev[1], st)) != cudaSuccess)
            return cuda_fail(e, "trace event");
        e = dflash::launch_topk(plan, logits, V, K, cand_ids, unary, workspace, st, softcap,
                                scale, qbytes, /*clear_counters=*/false, queue,
                                /*programmatic=*/chain);
        if (e != cudaSuccess) return cuda_fail(e, "top-k launch");
    }
    if (ev && (e = cudaEventRecord(ev[2], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    e = dflash::launch_edges(dev, pred_cb, succ_cb, cand_ids, unary, h_out, anchors, R, S, K, V,
                             rank, edges, status, st, /*after_h_producer=*/false, queue,
                             /*programmatic=*/chain);
    if (e != cudaSuccess) return cuda_fail(e, "edges launch");
    if (ev && (e = cudaEventRecord(ev[3], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    return ok();
}

dflash_status dflash_selector_forward(const int32_t* cand_ids, const float* unary,
                                      const uint16_t* hidden, const int32_t* anchors,
                                      const uint16_t* w_proj, const uint16_t* pred_cb,
                                      const uint16_t* succ_cb, int R, int S, int K, int V, int H,
                                      int rank, uint16_t* h_out, float* edges,
                                      dflash_stream_t stream) {
    NvtxRange range("dflash_selector_forward");
    DFLASH_TRY(check_dims_edges(R, S, K, V, rank));
    DFLASH_TRY(check_dims_projection(R, S, H, rank));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    DFLASH_TRY(check_ptr(hidden, "hidden"));
    DFLASH_TRY(check_ptr4(anchors, "anchors"));
    DFLASH_TRY(check_ptr(w_proj, "w_proj"));
    DFLASH_TRY(check_ptr(pred_cb, "pred_cb"));
    DFLASH_TRY(check_ptr(succ_cb, "succ_cb"));
    DFLASH_TRY(check_ptr(h_out, "h_out"));
    DFLASH_TRY(check_ptr4(edges, "edges"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dflash::launch_projection(dev, hidden, w_proj, R * S, H, rank, h_out, status, st);
    if (e != cudaSuccess) return cuda_fail(e, "projection launch");
    // The edges start their gathers while the projection finishes and wait for it only to
    // read h (programmatic dependent launch).
    e = dflash::launch_edges(dev, pred_cb, succ_cb, cand_ids, unary, h_out, anchors, R, S, K, V,
                             rank, edges, status, st, /*after_h_producer=*/true);
    if (e != cudaSuccess) return cuda_fail(e, "edges launch");
    return ok();
}

dflash_status dflash_best_path(const float* edges, const int32_t* cand_ids, int R, int S, int K,
                               int32_t* path, int32_t* tokens, float* score,
                               dflash_stream_t stream) {
    NvtxRange range("dflash_best_path");
    if (R < 1 || S < 1 || K < 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R, S and K must be >= 1 (got R=%d S=%d K=%d)", R, S,
                    K);
    if (K > 32) return fail(DFLASH_UNSUPPORTED, "K=%d: the best path supports K <= 32", K);
    if (S > dflash::kMaxPathSteps)
        return fail(DFLASH_UNSUPPORTED, "S=%d: the best path supports S <= %d", S,
                    dflash::kMaxPathSteps);
    DFLASH_TRY(check_ptr4(edges, "edges"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(path, "path"));
    DFLASH_TRY(check_ptr4(tokens, "tokens"));
    DFLASH_TRY(check_ptr4(score, "score"));
    DFLASH_TRY(current_device(nullptr, nullptr));
    cudaError_t e = dflash::launch_best_path(edges, cand_ids, R, S, K, path, tokens, score,
                                             reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "best path launch");
    return ok();
}

size_t dflash_selector_lmhead_workspace_bytes(int R, int S, int V, int K) {
    return dflash_lmhead_topk_workspace_bytes(R, S, V, K);
}

dflash_status dflash_selector_lmhead(const uint16_t* hidden, const uint16_t* lm_head,
                                     const uint16_t* w_proj, const uint16_t* pred_cb,
                                     const uint16_t* succ_cb, const int32_t* anchors, int R,
                                     int S, int K, int V, int H, int rank, float softcap,
                                     float scale, int32_t* cand_ids, float* unary,
                                     uint16_t* h_out, float* edges, void* workspace,
                                     size_t workspace_bytes, dflash_stream_t stream) {
    NvtxRange range("dflash_selector_lmhead");
    DFLASH_TRY(check_dims_topk(R, S, V, K));
    DFLASH_TRY(check_processor(softcap, scale));
    DFLASH_TRY(check_dims_projection(R, S, H, rank));
    DFLASH_TRY(check_ptr(hidden, "hidden"));
    DFLASH_TRY(check_ptr(lm_head, "lm_head"));
    DFLASH_TRY(check_ptr(w_proj, "w_proj"));
    DFLASH_TRY(check_ptr(pred_cb, "pred_cb"));
    DFLASH_TRY(check_ptr(succ_cb, "succ_cb"));
    DFLASH_TRY(check_ptr4(anchors, "anchors"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(unary, "unary"));
    DFLASH_TRY(check_ptr(h_out, "h_out"));
    DFLASH_TRY(check_ptr4(edges, "edges"));
    DFLASH_TRY(check_ptr(workspace, "workspace"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    const dflash::LmheadPlan plan = dflash::lmhead_plan(dev, (long long)R * S, V);
    if (workspace_bytes < plan.workspace_bytes())
        return fail(DFLASH_WORKSPACE_TOO_SMALL, "workspace of %zu bytes; %zu needed",
                    workspace_bytes, plan.workspace_bytes());
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaEvent_t* ev = trace_slot(dev.device);
    // One stream: the LM-head top-k sizes its grid to one CTA per SM, and a projection CTA
    // beside it would push one of them into a second wave.
    cudaError_t e;
    if (ev && (e = cudaEventRecord(ev[0], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    e = dflash::launch_projection(dev, hidden, w_proj, R * S, H, rank, h_out, status, st);
    if (e != cudaSuccess) return cuda_fail(e, "projection launch");
    if (ev && (e = cudaEventRecord(ev[1], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    e = dflash::launch_lmhead_topk(dev, plan, hidden, lm_head, R * S, H, V, K, softcap, scale,
                                   cand_ids, unary, workspace, status, st);
    if (e != cudaSuccess) return cuda_fail(e, "LM-head top-k launch");
    if (ev && (e = cudaEventRecord(ev[2], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    e = dflash::launch_edges(dev, pred_cb, succ_cb, cand_ids, unary, h_out, anchors, R, S, K, V,
                             rank, edges, status, st);
    if (e != cudaSuccess) return cuda_fail(e, "edges launch");
    if (ev && (e = cudaEventRecord(ev[3], st)) != cudaSuccess) return cuda_fail(e, "trace event");
    return ok();
}

dflash_status dflash_block_tables(const int32_t* context_lens, const int32_t* new_lens,
                                  const int32_t* held_pages, const int32_t* free_pages, int R,
                                  int n_free, int page_size, int max_pages, int T,
                                  int32_t* block_table, int32_t* query_start, int32_t* kv_lens,
                                  int32_t* held_out, int32_t* positions, int64_t* slots,
                                  int32_t* pages_needed, dflash_stream_t stream) {
    NvtxRange range("dflash_block_tables");
    if (R < 1 || page_size < 1 || max_pages < 1 || T < 0 || n_free < 0)
        return fail(DFLASH_INVALID_ARGUMENT,
                    "R, page_size and max_pages must be >= 1, T and n_free >= 0 (got %d, %d, %d, "
                    "%d, %d)", R, page_size, max_pages, T, n_free);
    if (R > dflash::kMaxTableRequests)
        return fail(DFLASH_UNSUPPORTED, "R=%d: block tables support R <= %d", R,
                    dflash::kMaxTableRequests);
    DFLASH_TRY(check_ptr4(context_lens, "context_lens"));
    DFLASH_TRY(check_ptr4(new_lens, "new_lens"));
    DFLASH_TRY(check_ptr4(held_pages, "held_pages"));
    if (n_free > 0) DFLASH_TRY(check_ptr4(free_pages, "free_pages"));
    DFLASH_TRY(check_ptr4(block_table, "block_table"));
    DFLASH_TRY(check_ptr4(query_start, "query_start"));
    DFLASH_TRY(check_ptr4(kv_lens, "kv_lens"));
    DFLASH_TRY(check_ptr4(held_out, "held_out"));
    if (T > 0) {
        DFLASH_TRY(check_ptr4(positions, "positions"));
        DFLASH_TRY(check_ptr8(slots, "slots"));
    }
    DFLASH_TRY(check_ptr4(pages_needed, "pages_needed"));
    if (held_out == held_pages || kv_lens == context_lens)
        return fail(DFLASH_INVALID_ARGUMENT,
                    "held_out must not be held_pages, nor kv_lens context_lens");
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    const dflash::BlockTableArgs a{context_lens, new_lens, held_pages, free_pages, R, n_free,
                                   page_size, max_pages, T, block_table, query_start, kv_lens,
                                   held_out, positions, slots, pages_needed};
    cudaError_t e = dflash::launch_block_tables(dev, a, status,
                                                reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "block tables launch");
    return ok();
}

dflash_status dflash_store_kv(const void* key, const void* value, int dtype, const int64_t* slots,
                              int T, long long key_token_stride, long long key_head_stride,
                              long long value_token_stride, long long value_head_stride,
                              const dflash_kv_cache* cache, dflash_stream_t stream) {
    NvtxRange range("dflash_store_kv");
    if (T < 0) return fail(DFLASH_INVALID_ARGUMENT, "T=%d must be >= 0", T);
    dflash::KvCache c;
    DFLASH_TRY(check_cache(cache, dtype, &c));
    DFLASH_TRY(check_stride(key_token_stride, T, 8, "key_token_stride"));
    DFLASH_TRY(check_stride(key_head_stride, c.kv_heads, 8, "key_head_stride"));
    DFLASH_TRY(check_stride(value_token_stride, T, 8, "value_token_stride"));
    DFLASH_TRY(check_stride(value_head_stride, c.kv_heads, 8, "value_head_stride"));
    if (T == 0) return ok();
    DFLASH_TRY(check_ptr(key, "key"));
    DFLASH_TRY(check_ptr(value, "value"));
    DFLASH_TRY(check_ptr8(slots, "slots"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    cudaError_t e = dflash::launch_store_kv(dev, key, value, dtype, slots, T, key_token_stride,
                                            key_head_stride, value_token_stride, value_head_stride,
                                            c, status, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "key-value store launch");
    return ok();
}

size_t dflash_paged_attention_workspace_bytes(int R, int T, int q_heads, int kv_heads,
                                              int head_dim) {
    if (R < 1 || T < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1) {
        fail(DFLASH_INVALID_ARGUMENT, "R, q_heads, kv_heads and head_dim must be >= 1, T >= 0");
        return 0;
    }
    dflash::DeviceInfo dev;
    if (current_device(&dev, nullptr) != DFLASH_OK) return 0;
    // The kernel for other head sizes and groups writes its outputs at once.
    if (!dflash::attention_may_use_tensor_cores(head_dim, q_heads / kv_heads, R)) return 256;
    return dflash::attention_workspace_bytes(dev, head_dim);
}

dflash_status dflash_paged_attention(const void* query, int dtype, int T, int q_heads,
                                     long long q_token_stride, long long q_head_stride,
                                     const dflash_kv_cache* cache, const int32_t* block_table,
                                     int R, int max_pages, const int32_t* query_start,
                                     const int32_t* kv_lens, float scale, int window_left,
                                     int window_right, float softcap, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes,
                                     dflash_stream_t stream) {
    NvtxRange range("dflash_paged_attention");
    if (T < 0 || R < 1 || max_pages < 1 || q_heads < 1)
        return fail(DFLASH_INVALID_ARGUMENT,
                    "R, max_pages and q_heads must be >= 1, T >= 0 (got %d, %d, %d, %d)", R,
                    max_pages, q_heads, T);
    dflash::KvCache c;
    DFLASH_TRY(check_cache(cache, dtype, &c));
    if (q_heads % c.kv_heads != 0)
        return fail(DFLASH_INVALID_ARGUMENT, "q_heads=%d must be a multiple of kv_heads=%d", q_heads,
                    c.kv_heads);
    if ((long long)T * q_heads > (1LL << 31) - 1)
        return fail(DFLASH_INVALID_ARGUMENT, "T*q_heads=%lld rows exceeds 2^31-1",
                    (long long)T * q_heads);
    if (!(scale > 0.f) || isinf(scale))
        return fail(DFLASH_INVALID_ARGUMENT, "scale=%g must be finite and > 0", (double)scale);
    if (window_left < -1 || window_right < -1)
        return fail(DFLASH_INVALID_ARGUMENT, "window_left=%d and window_right=%d must be >= -1",
                    window_left, window_right);
    if (!(softcap >= 0.f) || isinf(softcap))
        return fail(DFLASH_INVALID_ARGUMENT, "softcap=%g must be finite and >= 0 (0 = no cap)",
                    (double)softcap);
    DFLASH_TRY(check_stride(q_token_stride, T, 8, "q_token_stride"));
    DFLASH_TRY(check_stride(q_head_stride, q_heads, 8, "q_head_stride"));
    if (T == 0) return ok();
    DFLASH_TRY(check_ptr(query, "query"));
    DFLASH_TRY(check_ptr4(block_table, "block_table"));
    DFLASH_TRY(check_ptr4(query_start, "query_start"));
    DFLASH_TRY(check_ptr4(kv_lens, "kv_lens"));
    DFLASH_TRY(check_ptr(out, "out"));
    if (lse) DFLASH_TRY(check_ptr4(lse, "lse"));
    DFLASH_TRY(check_ptr(workspace, "workspace"));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    const dflash::AttentionArgs a{query, dtype, T, q_heads, q_token_stride, q_head_stride, c,
                                  block_table, R, max_pages, query_start, kv_lens, scale,
                                  window_left, window_right, softcap, out, lse};
    const size_t need = dflash_paged_attention_workspace_bytes(R, T, q_heads, c.kv_heads, c.head_dim);
    if (workspace_bytes < need)
        return fail(DFLASH_WORKSPACE_TOO_SMALL, "workspace of %zu bytes; %zu needed",
                    workspace_bytes, need);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dflash::attention_on_tensor_cores(a)
                        ? dflash::launch_attention(dev, a, workspace, status, st)
                        : dflash::launch_attention_rows(dev, a, status, st);
    if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
    return ok();
}

dflash_status dflash_rope_frequencies(int rotary_dim, double base, double factor,
                                      double original_len, double turns_slow, double turns_fast,
                                      const double* inv_freq, int64_t* frequencies) {
    if (rotary_dim < 0 || rotary_dim % 2 != 0)
        return fail(DFLASH_INVALID_ARGUMENT, "rotary_dim=%d must be even and >= 0", rotary_dim);
    if (rotary_dim > 0 && !frequencies) return fail(DFLASH_INVALID_ARGUMENT, "frequencies is NULL");
    if (!inv_freq) {
        if (!(base > 0) || std::isinf(base))
            return fail(DFLASH_INVALID_ARGUMENT, "base=%g must be finite and > 0", base);
        if (!(factor > 0) || std::isinf(factor))
            return fail(DFLASH_INVALID_ARGUMENT, "factor=%g must be finite and > 0", factor);
        if (!(original_len >= 0) || std::isinf(original_len))
            return fail(DFLASH_INVALID_ARGUMENT, "original_len=%g must be finite and >= 0",
                        original_len);
        if (original_len > 0 && !(turns_slow < turns_fast && std::isfinite(turns_slow) &&
                                  std::isfinite(turns_fast)))
            return fail(DFLASH_INVALID_ARGUMENT,
                        "turns_slow=%g and turns_fast=%g must be finite, the first below the second",
                        turns_slow, turns_fast);
    }
    const double two_pi = 6.283185307179586476925;
    for (int j = 0; j < rotary_dim / 2; ++j) {
        double f;
        if (inv_freq) {
            f = inv_freq[j];
            if (!std::isfinite(f))
                return fail(DFLASH_INVALID_ARGUMENT, "inv_freq[%d]=%g must be finite", j, f);
        } else {
            f = std::pow(base, -2.0 * j / rotary_dim);
            double keep = 0.0;
            if (original_len > 0)
                keep = std::min(1.0, std::max(0.0, (original_len * f / two_pi - turns_slow) /
                                                       (turns_fast - turns_slow)));
            if (factor != 1.0) f = f / factor * (1.0 - keep) + f * keep;
            if (!std::isfinite(f))
                return fail(DFLASH_INVALID_ARGUMENT, "the frequency of pair %d is not finite: base=%g, factor=%g", j,
                            base, factor);
        }
        double turns = std::fabs(f) / two_pi;
        turns -= std::floor(turns);                          // whole turns do not show
        // Two halves of 32 bits, each exact. (Backward turns are those forward, negated: the rest of a small one to 1
        // would be rounded to 2^-53.)
        const double high = std::floor(turns * 4294967296.0);
        const double low = std::floor((turns * 4294967296.0 - high) * 4294967296.0 + 0.5);
        const uint64_t whole = ((uint64_t)high << 32) + (uint64_t)low;
        frequencies[j] = (int64_t)(f < 0 ? 0 - whole : whole);
    }
    return ok();
}

dflash_status dflash_qk_norm_rope(const void* query, const void* key, int dtype,
                                  const int32_t* positions, int T, int q_heads, int kv_heads,
                                  int head_dim, long long q_token_stride, long long q_head_stride,
                                  long long k_token_stride, long long k_head_stride,
                                  const dflash_norm_rope* how, void* query_out, void* key_out,
                                  long long q_out_token_stride, long long q_out_head_stride,
                                  long long k_out_token_stride, long long k_out_head_stride,
                                  dflash_stream_t stream) {
    NvtxRange range("dflash_qk_norm_rope");
    dflash::NormRopeArgs a{};
    a.query = query; a.key = key; a.dtype = dtype; a.T = T; a.q_heads = q_heads;
    a.kv_heads = kv_heads; a.head_dim = head_dim; a.positions = positions;
    a.qt = q_token_stride; a.qh = q_head_stride; a.kt = k_token_stride; a.kh = k_head_stride;
    a.query_out = query_out; a.key_out = key_out;
    a.qot = q_out_token_stride; a.qoh = q_out_head_stride;
    a.kot = k_out_token_stride; a.koh = k_out_head_stride;
    a.cache.k_scale = a.cache.v_scale = 1.f;
    if (q_heads < 0 || kv_heads < 0 || q_heads + (long long)kv_heads < 1)
        return fail(DFLASH_INVALID_ARGUMENT,
                    "q_heads=%d and kv_heads=%d must be >= 0, and one of them >= 1", q_heads, kv_heads);
    DFLASH_TRY(check_norm_rope(how, &a));
    if (kv_heads > 0)
        DFLASH_TRY(check_row_strides(k_out_token_stride, T, k_out_head_stride, kv_heads,
                                     "k_out_token_stride", "k_out_head_stride"));
    if (T == 0) return ok();
    if (kv_heads > 0) DFLASH_TRY(check_ptr(key_out, "key_out"));
    DFLASH_TRY(check_norm_rope_pointers(a));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    cudaError_t e = dflash::launch_norm_rope(dev, a, status, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "norm and rotation launch");
    return ok();
}

dflash_status dflash_qk_norm_rope_store(
    const void* query, const void* key, const void* value, int dtype, const int32_t* positions,
    const int64_t* slots, int T, int q_heads, long long q_token_stride, long long q_head_stride,
    long long k_token_stride, long long k_head_stride, long long v_token_stride,
    long long v_head_stride, const dflash_norm_rope* how, const dflash_kv_cache* cache,
    void* query_out, long long q_out_token_stride, long long q_out_head_stride,
    dflash_stream_t stream) {
    NvtxRange range("dflash_qk_norm_rope_store");
    dflash::NormRopeArgs a{};
    DFLASH_TRY(check_cache(cache, dtype, &a.cache));
    a.query = query; a.key = key; a.value = value; a.dtype = dtype; a.T = T; a.q_heads = q_heads;
    a.kv_heads = a.cache.kv_heads; a.head_dim = a.cache.head_dim; a.positions = positions;
    a.qt = q_token_stride; a.qh = q_head_stride; a.kt = k_token_stride; a.kh = k_head_stride;
    a.vt = v_token_stride; a.vh = v_head_stride;
    a.query_out = query_out; a.qot = q_out_token_stride; a.qoh = q_out_head_stride;
    a.slots = slots;
    if (q_heads < 0) return fail(DFLASH_INVALID_ARGUMENT, "q_heads=%d must be >= 0", q_heads);
    DFLASH_TRY(check_norm_rope(how, &a));
    DFLASH_TRY(check_row_strides(v_token_stride, T, v_head_stride, a.kv_heads, "v_token_stride",
                                 "v_head_stride"));
    if (T == 0) return ok();
    DFLASH_TRY(check_ptr(value, "value"));
    DFLASH_TRY(check_ptr8(slots, "slots"));
    DFLASH_TRY(check_norm_rope_pointers(a));
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    cudaError_t e = dflash::launch_norm_rope(dev, a, status, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "norm, rotation and store launch");
    return ok();
}

dflash_status dflash_sample_path(const float* edges, const int32_t* cand_ids, const float* uniforms,
                                 const float* temperatures, float temperature, int R, int S, int K,
                                 int32_t* path, int32_t* tokens, float* probs,
                                 dflash_stream_t stream) {
    NvtxRange range("dflash_sample_path");
    if (R < 1 || S < 1 || K < 1)
        return fail(DFLASH_INVALID_ARGUMENT, "R, S and K must be >= 1 (got R=%d S=%d K=%d)", R, S, K);
    if (K > 32) return fail(DFLASH_UNSUPPORTED, "K=%d: a path supports K <= 32", K);
    if (S > dflash::kMaxPathSteps)
        return fail(DFLASH_UNSUPPORTED, "S=%d: a path supports S <= %d", S, dflash::kMaxPathSteps);
    DFLASH_TRY(check_temperature(temperatures, temperature));
    DFLASH_TRY(check_ptr4(edges, "edges"));
    DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
    DFLASH_TRY(check_ptr4(uniforms, "uniforms"));
    DFLASH_TRY(check_ptr4(path, "path"));
    DFLASH_TRY(check_ptr4(tokens, "tokens"));
    DFLASH_TRY(check_ptr4(probs, "probs"));
    DFLASH_TRY(current_device(nullptr, nullptr));
    const dflash::SamplePathArgs a{edges, cand_ids, uniforms, temperatures, temperature, R, S, K,
                                   path, tokens, probs};
    cudaError_t e = dflash::launch_sample_path(a, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "sampled path launch");
    return ok();
}

size_t dflash_verify_drafts_workspace_bytes(int R, int T, int V) {
    if (R < 1 || T < 0 || V < 1) {
        fail(DFLASH_INVALID_ARGUMENT, "R and V must be >= 1, T >= 0 (got R=%d T=%d V=%d)", R, T, V);
        return 0;
    }
    return dflash::verify_workspace_bytes(R, T, V);
}

dflash_status dflash_verify_drafts(const void* logits, int dtype, int T, int V, long long row_stride,
                                   const int32_t* query_start, const int32_t* draft_tokens, int R,
                                   int S, const int32_t* cand_ids, const float* draft_probs, int K,
                                   const float* accept_uniforms, const float* sample_uniforms,
                                   const float* temperatures, float temperature, int32_t* tokens,
                                   int32_t* counts, float* logprobs, void* workspace,
                                   size_t workspace_bytes, dflash_stream_t stream) {
    NvtxRange range("dflash_verify_drafts");
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP16 && dtype != DFLASH_FP32)
        return fail(DFLASH_INVALID_ARGUMENT, "dtype=%d: must be DFLASH_BF16, DFLASH_FP16 or DFLASH_FP32",
                    dtype);
    if (T < 0 || V < 1 || R < 1 || S < 0)
        return fail(DFLASH_INVALID_ARGUMENT, "V and R must be >= 1, T and S >= 0 (got V=%d R=%d T=%d S=%d)",
                    V, R, T, S);
    if (S > dflash::kMaxDrafts)
        return fail(DFLASH_UNSUPPORTED, "S=%d: the verification supports S <= %d", S, dflash::kMaxDrafts);
    if (V > dflash::kMaxVerifyVocab)
        return fail(DFLASH_UNSUPPORTED, "V=%d: the verification supports V <= %d", V,
                    dflash::kMaxVerifyVocab);
    if (T > 1 && row_stride < V)
        return fail(DFLASH_INVALID_ARGUMENT, "row_stride=%lld must be >= V=%d", row_stride, V);
    if ((cand_ids == nullptr) != (draft_probs == nullptr) && S > 0)
        return fail(DFLASH_INVALID_ARGUMENT, "cand_ids and draft_probs must be given together");
    if (cand_ids && K < 1) return fail(DFLASH_INVALID_ARGUMENT, "K=%d must be >= 1", K);
    if (cand_ids && K > 32) return fail(DFLASH_UNSUPPORTED, "K=%d: the verification supports K <= 32", K);
    DFLASH_TRY(check_temperature(temperatures, temperature));
    DFLASH_TRY(check_ptr4(query_start, "query_start"));
    DFLASH_TRY(check_ptr4(sample_uniforms, "sample_uniforms"));
    if (S > 0) {
        DFLASH_TRY(check_ptr4(draft_tokens, "draft_tokens"));
        DFLASH_TRY(check_ptr4(accept_uniforms, "accept_uniforms"));
        if (cand_ids) {
            DFLASH_TRY(check_ptr4(cand_ids, "cand_ids"));
            DFLASH_TRY(check_ptr4(draft_probs, "draft_probs"));
        }
    }
    DFLASH_TRY(check_ptr4(tokens, "tokens"));
    DFLASH_TRY(check_ptr4(counts, "counts"));
    if (logprobs) DFLASH_TRY(check_ptr4(logprobs, "logprobs"));
    DFLASH_TRY(check_ptr(workspace, "workspace"));
    if (T > 0) {
        if (!logits) return fail(DFLASH_INVALID_ARGUMENT, "logits is NULL");
        const unsigned size = dtype == DFLASH_FP32 ? 4 : 2;
        if (reinterpret_cast<uintptr_t>(logits) % size != 0)
            return fail(DFLASH_INVALID_ARGUMENT, "logits is not %u-byte aligned", size);
    }
    const size_t need = dflash::verify_workspace_bytes(R, T, V);
    if (workspace_bytes < need)
        return fail(DFLASH_WORKSPACE_TOO_SMALL, "workspace of %zu bytes; %zu needed",
                    workspace_bytes, need);
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    const dflash::VerifyArgs a{logits, dtype, T, V, row_stride, query_start, draft_tokens, R, S,
                               cand_ids, draft_probs, K, accept_uniforms, sample_uniforms,
                               temperatures, temperature, tokens, counts, logprobs};
    cudaError_t e = dflash::launch_verify(dev, a, workspace, status,
                                          reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "verification launch");
    return ok();
}

namespace {

// One thread waits on an mbarrier that nothing arrives on; the bounded wait gives up.
__global__ void wait_timeout_kernel(uint32_t* status) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        const uint32_t b = dflash::ptx::smem_u32(&bar);
        dflash::ptx::mbar_init(b, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (!dflash::ptx::mbar_wait(b, 0)) atomicOr(status, dflash::kStatusTimeout);
    }
}

}  // namespace

dflash_status dflash_selftest_wait_timeout(void) {
    dflash::DeviceInfo dev;
    uint32_t* status = nullptr;
    DFLASH_TRY(current_device(&dev, &status));
    wait_timeout_kernel<<<1, 32>>>(status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "wait self-check launch");
    e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "wait self-check");
    // The edge tiles' ready queue: one edge CTA waits for a tile that is never pushed. Its
    // queue and every array it is given live in a zeroed static buffer; it gives up before it
    // reads any of them and writes nothing.
    void* buf = nullptr;
    e = cudaGetSymbolAddress(&buf, g_selftest_buffer);
    if (e == cudaSuccess) e = cudaMemset(buf, 0, sizeof(g_selftest_buffer));
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_fail(e, "queue self-check buffer");
    }
    uint32_t* w = static_cast<uint32_t*>(buf);
    dflash::EdgeQueue q = dflash::edge_queue_at(w, 1, 1);
    q.proj_ctas = 1;
    const uint16_t* b16 = reinterpret_cast<const uint16_t*>(w + 64);
    e = dflash::launch_edges(dev, b16, b16, reinterpret_cast<const int32_t*>(w + 64),
                             reinterpret_cast<const float*>(w + 64), b16,
                             reinterpret_cast<const int32_t*>(w + 64), 1, 1, 1, 1, 8,
                             reinterpret_cast<float*>(w + 128), status, nullptr, false, q);
    if (e != cudaSuccess) return cuda_fail(e, "queue self-check launch");
    e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "queue self-check");
    return ok();
}

dflash_status dflash_device_status(uint32_t* flags, int clear) {
    if (!flags) return fail(DFLASH_INVALID_ARGUMENT, "flags is NULL");
    DFLASH_TRY(current_device(nullptr, nullptr));
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
    e = cudaMemcpyFromSymbol(flags, g_device_status, sizeof(uint32_t));
    if (e != cudaSuccess) return cuda_fail(e, "read status word");
    if (clear) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(uint32_t));
        if (e != cudaSuccess) return cuda_fail(e, "clear status word");
    }
    return ok();
}

dflash_status dflash_trace_begin(int n_calls) {
    if (n_calls < 1 || n_calls > (1 << 20))
        return fail(DFLASH_INVALID_ARGUMENT, "n_calls=%d must be in [1, 2^20]", n_calls);
    dflash::DeviceInfo dev;
    DFLASH_TRY(current_device(&dev, nullptr));
    std::lock_guard<std::mutex> lock(g_trace.mu);
    if (g_trace.capacity != 0) return fail(DFLASH_INVALID_ARGUMENT, "a trace is already active");
    g_trace.events.assign(4 * (size_t)n_calls, nullptr);
    for (auto& ev : g_trace.events) {
        cudaError_t e = cudaEventCreate(&ev);
        if (e != cudaSuccess) {
            for (auto& x : g_trace.events)
                if (x) cudaEventDestroy(x);
            g_trace.events.clear();
            return cuda_fail(e, "cudaEventCreate");
        }
    }
    g_trace.device = dev.device;
    g_trace.capacity = n_calls;
    g_trace.used = 0;
    return ok();
}

dflash_status dflash_trace_end(float* stage_ms, int max_calls, int* n_calls) {
    std::lock_guard<std::mutex> lock(g_trace.mu);
    if (g_trace.capacity == 0) return fail(DFLASH_INVALID_ARGUMENT, "no trace is active");
    dflash_status st = DFLASH_OK;
    const int n = g_trace.used < max_calls ? g_trace.used : (max_calls > 0 ? max_calls : 0);
    for (int i = 0; i < n && st == DFLASH_OK; ++i) {
        cudaEvent_t* ev = &g_trace.events[4 * (size_t)i];
        cudaError_t e = cudaEventSynchronize(ev[3]);
        // Events: [0] start, [1] projection done, [2] top-k done, [3] edges done; a traced
        // call runs its kernels one after another, so each stage is the time between two.
        const int from[3] = {0, 1, 2}, to[3] = {1, 2, 3};
        for (int k = 0; k < 3 && e == cudaSuccess; ++k) {
            float ms = 0.f;
            e = cudaEventElapsedTime(&ms, ev[from[k]], ev[to[k]]);
            if (stage_ms) stage_ms[3 * i + k] = ms;
        }
        if (e != cudaSuccess) st = cuda_fail(e, "reading trace events");
    }
    for (auto& ev : g_trace.events) cudaEventDestroy(ev);
    g_trace.events.clear();
    g_trace.capacity = 0;
    g_trace.used = 0;
    g_trace.device = -1;
    if (n_calls) *n_calls = n;
    return st == DFLASH_OK ? ok() : st;
}

}  // extern "C"
