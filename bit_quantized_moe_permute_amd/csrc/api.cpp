// C-ABI entry points of libmoe2bit: argument checking on the host, then kernel
// dispatch on the caller's stream.  Nothing here allocates device memory or
// synchronizes (unless MOE_SYNC_DEBUG asks for it); no C++ exception crosses
// the interface.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "../../include/moe2bit.h"
#include "internal.h"

namespace {

thread_local char g_err[512] = "";

moe_status fail(moe_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

moe_status ok() {
    g_err[0] = '\0';
    return MOE_OK;
}

// MOE_SYNC_DEBUG, read once per process: any value but "" or "0" turns it on.
bool sync_debug() {
    static const bool on = [] {
        const char *v = std::getenv("MOE_SYNC_DEBUG");
        return v && *v && std::strcmp(v, "0") != 0;
    }();
    return on;
}

// Result of a group of launches on stream s.  With the debug switch on, the call first waits for s (unless s is
// being captured into a graph, where waiting is not allowed) so that a fault in those kernels is reported by the
// entry point that launched them.
moe_status from_hip(hipError_t e, const char *what, hipStream_t s) {
    if (e == hipSuccess && sync_debug()) {
        hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
        e = hipStreamIsCapturing(s, &cs);
        if (e == hipSuccess && cs == hipStreamCaptureStatusNone) {
            e = hipStreamSynchronize(s);
            if (e == hipSuccess) e = hipGetLastError();
        }
    }
    if (e == hipSuccess) return ok();
    return fail(MOE_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

int block_bytes(int fmt) {
    switch (fmt) {
        case MOE_FMT_IQ2X: return 66;
        case MOE_FMT_Q2K: return 84;
        case MOE_FMT_Q4K: return 144;
        default: return 0;
    }
}

// Sub-blocks may not straddle rows.
int sub_len(int fmt) { return fmt == MOE_FMT_Q2K ? 16 : 32; }

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

moe_status check_matrix(int fmt, int64_t n_mats, int64_t rows, int64_t cols, const char *what) {
    if (!block_bytes(fmt)) return fail(MOE_ERR_INVALID_ARG, "%s: unknown format %d", what, fmt);
    if (n_mats < 1 || rows < 1 || cols < 1) return fail(MOE_ERR_INVALID_ARG, "%s: empty shape", what);
    if ((rows * cols) % 256) return fail(MOE_ERR_INVALID_ARG, "%s: rows*cols not a multiple of 256", what);
    if (cols % sub_len(fmt))
        return fail(MOE_ERR_INVALID_ARG, "%s: cols %% %d != 0 (sub-blocks would straddle rows)", what, sub_len(fmt));
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_ABI_VERSION; }

int moe_sync_debug(void) { return sync_debug() ? 1 : 0; }

const char *moe_last_error(void) { return g_err; }

size_t moe_weight_bytes(int32_t fmt, int64_t n_mats, int64_t rows, int64_t cols) {
    const int bb = block_bytes(fmt);
    if (!bb || n_mats < 1 || rows < 1 || cols < 1 || (rows * cols) % 256) return 0;
    return (size_t)(n_mats * rows * cols / 256) * (size_t)bb;
}

moe_status moe_prepare_weights(int32_t fmt, int64_t n_mats, int64_t rows, int64_t cols, const void *canonical,
                               void *prepared, void *stream) {
    moe_status st = check_matrix(fmt, n_mats, rows, cols, "moe_prepare_weights");
    if (st != MOE_OK) return st;
    if (!canonical || !prepared) return fail(MOE_ERR_INVALID_ARG, "moe_prepare_weights: null pointer");
    if (!aligned(prepared, 16)) return fail(MOE_ERR_INVALID_ARG, "moe_prepare_weights: prepared not 16-byte aligned");
    const size_t bytes = moe_weight_bytes(fmt, n_mats, rows, cols);
    const char *c = static_cast<const char *>(canonical), *p = static_cast<const char *>(prepared);
    if (c < p + bytes && p < c + bytes) return fail(MOE_ERR_INVALID_ARG, "moe_prepare_weights: buffers overlap");
    const int64_t NB = n_mats * rows * cols / 256;
    return from_hip(moe::launch_prepare(fmt, NB, canonical, prepared, (hipStream_t)stream), "moe_prepare_weights",
                    (hipStream_t)stream);
}

moe_status moe_dequantize(int32_t fmt, const void *prepared, int64_t n_mats, int64_t rows, int64_t cols,
                          int64_t mat_begin, int64_t mat_count, const uint8_t *codebook, float *out, void *stream) {
    moe_status st = check_matrix(fmt, n_mats, rows, cols, "moe_dequantize");
    if (st != MOE_OK) return st;
    if (!prepared || !out || (fmt == MOE_FMT_IQ2X && !codebook))
        return fail(MOE_ERR_INVALID_ARG, "moe_dequantize: null pointer");
    if (!aligned(prepared, 16) || !aligned(out, 4)) return fail(MOE_ERR_INVALID_ARG, "moe_dequantize: misaligned");
    if (mat_begin < 0 || mat_count < 1 || mat_begin + mat_count > n_mats)
        return fail(MOE_ERR_INVALID_ARG, "moe_dequantize: matrix range [%lld, +%lld) outside [0, %lld)",
                    (long long)mat_begin, (long long)mat_count, (long long)n_mats);
    if ((rows * cols) % 256) return fail(MOE_ERR_INVALID_ARG, "moe_dequantize: matrix not whole blocks");
    const int64_t per = rows * cols / 256;
    return from_hip(moe::launch_dequant(fmt, n_mats * per, mat_begin * per, mat_count * per, prepared, codebook, out,
                                        (hipStream_t)stream),
                    "moe_dequantize", (hipStream_t)stream);
}

// logits [T][E] fp32 | bounds of the matrix-core router: lo, hi [T][E] fp32, expert flags [E] int32
static size_t route_logits_bytes(int32_t T, int32_t E) { return ((size_t)T * E * sizeof(float) + 255) / 256 * 256; }

size_t moe_route_workspace(int32_t n_tokens, int32_t n_experts, int32_t top_k) {
    (void)top_k;
    if (n_tokens < 1 || n_experts < 1) return 0;
    return route_logits_bytes(n_tokens, n_experts) +
           ((2 * (size_t)n_tokens * n_experts + n_experts) * sizeof(float) + 255) / 256 * 256;
}

// Host checks of the routing arguments; fills `a` (logits scratch at ws).
static moe_status route_args(const char *fn, const void *x, int32_t x_dt, int32_t n_tokens, int32_t hidden,
                             const void *w_router, int32_t w_dt, int32_t n_experts, const float *bias, int32_t top_k,
                             int32_t *topk_idx, float *topk_w, float *logits, int32_t *expert_offsets, int32_t *perm,
                             int32_t *active, void *ws, size_t ws_bytes, moe::RouteArgs &a) {
    if (!x || !w_router || !topk_idx || !topk_w || !expert_offsets || !perm || !active || !ws)
        return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((x_dt != MOE_DT_F32 && x_dt != MOE_DT_BF16) || (w_dt != MOE_DT_F32 && w_dt != MOE_DT_BF16))
        return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (n_tokens < 1) return fail(MOE_ERR_INVALID_ARG, "%s: n_tokens < 1", fn);
    if (hidden < 64 || hidden % 64) return fail(MOE_ERR_INVALID_ARG, "%s: hidden %% 64 != 0", fn);
    if (n_experts < 1 || n_experts > 256) return fail(MOE_ERR_INVALID_ARG, "%s: n_experts outside [1, 256]", fn);
    if (top_k < 1 || top_k > n_experts) return fail(MOE_ERR_INVALID_ARG, "%s: top_k outside [1, n_experts]", fn);
    if ((int64_t)n_tokens * top_k > (int64_t)1 << 30) return fail(MOE_ERR_INVALID_ARG, "%s: too many slots", fn);
    if (ws_bytes < moe_route_workspace(n_tokens, n_experts, top_k))
        return fail(MOE_ERR_INVALID_ARG, "%s: workspace too small (%zu < %zu)", fn, ws_bytes,
                    moe_route_workspace(n_tokens, n_experts, top_k));
    if (!aligned(ws, 16) || !aligned(x, 4) || !aligned(w_router, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    a.x = x; a.x_bf16 = x_dt == MOE_DT_BF16; a.T = n_tokens; a.H = hidden;
    a.w = w_router; a.w_bf16 = w_dt == MOE_DT_BF16; a.E = n_experts; a.bias = bias; a.k = top_k;
    a.topk_idx = topk_idx; a.topk_w = topk_w; a.logits_out = logits;
    a.offsets = expert_offsets; a.perm = perm; a.active = active;
    a.logits_ws = static_cast<float *>(ws);
    a.bounds_ws = reinterpret_cast<float *>(static_cast<char *>(ws) + route_logits_bytes(n_tokens, n_experts));
    return MOE_OK;
}

moe_status moe_route(const void *x, int32_t x_dt, int32_t n_tokens, int32_t hidden, const void *w_router,
                     int32_t w_dt, int32_t n_experts, const float *bias, int32_t top_k, int32_t *topk_idx,
                     float *topk_w, float *logits, int32_t *expert_offsets, int32_t *perm, int32_t *active, void *ws,
                     size_t ws_bytes, void *stream) {
    moe::RouteArgs a;
    moe_status st = route_args("moe_route", x, x_dt, n_tokens, hidden, w_router, w_dt, n_experts, bias, top_k,
                               topk_idx, topk_w, logits, expert_offsets, perm, active, ws, ws_bytes, a);
    if (st != MOE_OK) return st;
    return from_hip(moe::launch_route(a, (hipStream_t)stream), "moe_route", (hipStream_t)stream);
}

static moe_status check_layer(const moe_layer_desc *L, const char *fn) {
    if (!L) return fail(MOE_ERR_INVALID_ARG, "%s: null layer", fn);
    if (L->hidden < 1 || L->inter < 1) return fail(MOE_ERR_INVALID_ARG, "%s: bad shape", fn);
    if (L->n_experts < 1 || L->n_experts > 256) return fail(MOE_ERR_INVALID_ARG, "%s: n_experts outside [1, 256]", fn);
    if (L->top_k < 1 || L->top_k > L->n_experts) return fail(MOE_ERR_INVALID_ARG, "%s: top_k outside [1, E]", fn);
    if (L->gate_up_fmt != MOE_FMT_IQ2X && L->gate_up_fmt != MOE_FMT_Q4K)
        return fail(MOE_ERR_INVALID_ARG, "%s: gate/up format must be iq2x or q4k", fn);
    if (L->down_fmt != MOE_FMT_Q2K && L->down_fmt != MOE_FMT_Q4K)
        return fail(MOE_ERR_INVALID_ARG, "%s: down format must be q2k or q4k", fn);
    moe_status st = check_matrix(L->gate_up_fmt, L->n_experts, L->inter, L->hidden, fn);
    if (st != MOE_OK) return st;
    if ((st = check_matrix(L->down_fmt, L->n_experts, L->hidden, L->inter, fn)) != MOE_OK) return st;
    if (!L->gate || !L->up || !L->down) return fail(MOE_ERR_INVALID_ARG, "%s: null expert weights", fn);
    if (!aligned(L->gate, 16) || !aligned(L->up, 16) || !aligned(L->down, 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: expert weights not 16-byte aligned", fn);
    if (L->gate_up_fmt == MOE_FMT_IQ2X && !L->codebook) return fail(MOE_ERR_INVALID_ARG, "%s: null codebook", fn);
    if (L->gate_up_fmt == MOE_FMT_IQ2X && !aligned(L->codebook, 8))
        return fail(MOE_ERR_INVALID_ARG, "%s: codebook not 8-byte aligned", fn);
    if (L->shared_inter < 0) return fail(MOE_ERR_INVALID_ARG, "%s: shared_inter < 0", fn);
    if (L->shared_inter > 0) {
        if (!L->shared_gate || !L->shared_up || !L->shared_down)
            return fail(MOE_ERR_INVALID_ARG, "%s: null shared expert weights", fn);
        if (!aligned(L->shared_gate, 16) || !aligned(L->shared_up, 16) || !aligned(L->shared_down, 16))
            return fail(MOE_ERR_INVALID_ARG, "%s: shared expert weights not 16-byte aligned", fn);
        if (L->hidden % 8 || L->shared_inter % 8)
            return fail(MOE_ERR_INVALID_ARG, "%s: shared expert dims must be multiples of 8", fn);
    }
    if (L->path < MOE_PATH_AUTO || L->path > MOE_PATH_GEMM) return fail(MOE_ERR_INVALID_ARG, "%s: unknown path", fn);
    if (L->precision != MOE_PRECISION_EXACT && L->precision != MOE_PRECISION_FAST)
        return fail(MOE_ERR_INVALID_ARG, "%s: unknown precision", fn);
    return MOE_OK;
}

static moe::FfnArgs make_args(const moe_layer_desc *L, const void *x, int x_dt, int T) {
    moe::FfnArgs a;
    memset(&a, 0, sizeof a);
    a.H = L->hidden; a.I = L->inter; a.E = L->n_experts; a.k = L->top_k; a.T = T;
    a.fmt_gu = L->gate_up_fmt; a.fmt_d = L->down_fmt;
    a.gate = static_cast<const uint8_t *>(L->gate);
    a.up = static_cast<const uint8_t *>(L->up);
    a.down = static_cast<const uint8_t *>(L->down);
    a.codebook = L->codebook;
    a.Is = L->shared_inter;
    a.sg = static_cast<const uint16_t *>(L->shared_gate);
    a.su = static_cast<const uint16_t *>(L->shared_up);
    a.sd = static_cast<const uint16_t *>(L->shared_down);
    a.x = x; a.x_bf16 = x_dt == MOE_DT_BF16;
    a.fast = L->precision == MOE_PRECISION_FAST;
    return a;
}

// Kernel family for this call: 1 generic, 2 gemv, 3 gemm.
static int choose_path(const moe_layer_desc *L, const moe::FfnArgs &a) {
    if (L->path != MOE_PATH_AUTO) return L->path;
    if (moe::ffn_gemv_supported(a)) return MOE_PATH_GEMV;
    if (a.T > 4 && moe::ffn_gemm_supported(a)) return MOE_PATH_GEMM;
    return MOE_PATH_GENERIC;
}

static size_t workspace_for(int path, const moe_layer_desc *L, int32_t T) {
    const int Is = L->shared_inter;
    switch (path) {
        case MOE_PATH_GEMV: return moe::ffn_workspace_gemv(L->hidden, L->inter, L->n_experts, L->top_k, Is, T);
        case MOE_PATH_GEMM: return moe::ffn_workspace_gemm(L->hidden, L->inter, L->n_experts, L->top_k, Is, T);
        default: return moe::ffn_workspace_generic(L->hidden, L->inter, L->n_experts, L->top_k, Is, T);
    }
}

size_t moe_expert_ffn_workspace(const moe_layer_desc *L, int32_t n_tokens) {
    if (n_tokens < 1 || check_layer(L, "moe_expert_ffn_workspace") != MOE_OK) return 0;
    size_t m = 0;
    for (int p = MOE_PATH_GENERIC; p <= MOE_PATH_GEMM; ++p) {
        size_t b = workspace_for(p, L, n_tokens);
        if (b > m) m = b;
    }
    return m;
}

// ---------------------------------------------------------------------------
// Static device scratch of moe_expert_ffn_noalloc: one copy per GPU, held until
// the process ends.  In host code `scratch` only names the symbol; its device
// address is looked up per device with hipGetSymbolAddress and used instead.
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

// Device address of the current device's `scratch`, looked up on the first call on that device (with the device
// current).  The caller's stream must belong to the current device.
moe_status scratch_for(void *stream, const char *fn, void **out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(MOE_ERR_DEVICE, "%s: hipGetDevice: %s", fn, hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices)
        return fail(MOE_ERR_UNSUPPORTED, "%s: device %d beyond the %d the library tracks", fn, dev, kMaxDevices);
    if (stream) {
        int sdev = -1;
        e = hipStreamGetDevice((hipStream_t)stream, &sdev);
        if (e != hipSuccess) return fail(MOE_ERR_DEVICE, "%s: hipStreamGetDevice: %s", fn, hipGetErrorString(e));
        if (sdev != dev)
            return fail(MOE_ERR_INVALID_ARG, "%s: the stream belongs to device %d, the current device is %d", fn,
                        sdev, dev);
    }
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p)
            return fail(MOE_ERR_DEVICE, "%s: hipGetSymbolAddress of the static scratch: %s", fn,
                        hipGetErrorString(e));
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return MOE_OK;
}

}  // namespace

// Routing done inside the gate/up launch of a one-token call (moe_layer): the logits to select from and the
// routing outputs to write.
struct InKernelRoute {
    const float *logits;
    int32_t *idx;
    float *w;
    int32_t *offsets, *perm, *active;
};

// ws == nullptr with static_ws: the kernels' scratch is this device's static `scratch`.
static moe_status expert_call(const char *fn, int stages, const moe_layer_desc *L, const void *x, int32_t x_dt,
                              int32_t n_tokens, const int32_t *topk_idx, const int32_t *expert_offsets,
                              const int32_t *perm, const int32_t *active, float *slot_out, float *shared_out,
                              void *ws, size_t ws_bytes, void *stream, bool static_ws = false,
                              const InKernelRoute *route = nullptr) {
    moe_status st = check_layer(L, fn);
    if (st != MOE_OK) return st;
    if (!x || !topk_idx || !expert_offsets || !perm || !active || (!ws && !static_ws))
        return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((stages & moe::STAGE_DOWN) && !slot_out) return fail(MOE_ERR_INVALID_ARG, "%s: null slot_out", fn);
    if (x_dt != MOE_DT_F32 && x_dt != MOE_DT_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (n_tokens < 1) return fail(MOE_ERR_INVALID_ARG, "%s: n_tokens < 1", fn);
    if ((stages & moe::STAGE_DOWN) && (L->shared_inter > 0) != (shared_out != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "%s: shared_out must be given iff the layer has a shared expert", fn);
    if (!aligned(x, 16) || (slot_out && !aligned(slot_out, 16)) || (ws && !aligned(ws, 256)) ||
        (shared_out && !aligned(shared_out, 16)))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer (x/outputs 16 B, ws 256 B)", fn);
    moe::FfnArgs a = make_args(L, x, x_dt, n_tokens);
    a.topk_idx = topk_idx; a.offsets = expert_offsets; a.perm = perm; a.active = active;
    a.slot_out = slot_out; a.shared_out = shared_out; a.ws = ws; a.stages = stages;
    const int path = choose_path(L, a);
    if (path == MOE_PATH_GEMV && !(moe::ffn_gemv_supported(a)))
        return fail(MOE_ERR_UNSUPPORTED, "%s: decode kernels need bf16 x, T <= 4 (T <= 8 with iq2x gate/up, "
                                         "q2k down and T*k <= 64), hidden in {512..4096}, supported inter/shared "
                                         "sizes", fn);
    if (path == MOE_PATH_GEMM && !(moe::ffn_gemm_supported(a)))
        return fail(MOE_ERR_UNSUPPORTED, "%s: grouped-GEMM kernels need bf16 x and hidden, inter, "
                                         "shared_inter multiples of 256", fn);
    const size_t need = workspace_for(path, L, n_tokens);
    if (static_ws) {
        if (need > MOE_NOALLOC_SCRATCH_BYTES)
            return fail(MOE_ERR_INVALID_ARG, "%s: %d tokens need %zu bytes of scratch, the static scratch holds %zu; "
                                             "use moe_expert_ffn with a workspace", fn, n_tokens, need,
                        (size_t)MOE_NOALLOC_SCRATCH_BYTES);
        if ((st = scratch_for(stream, fn, &a.ws)) != MOE_OK) return st;
    } else if (ws_bytes < need) {
        return fail(MOE_ERR_INVALID_ARG, "%s: workspace too small (%zu < %zu)", fn, ws_bytes, need);
    }
    if (route) {
        a.sel_logits = route->logits;
        a.sel_idx = route->idx; a.sel_w = route->w;
        a.sel_offsets = route->offsets; a.sel_perm = route->perm; a.sel_active = route->active;
    }
    hipError_t e;
    if (path == MOE_PATH_GEMV) e = moe::launch_ffn_gemv(a, (hipStream_t)stream);
    else if (path == MOE_PATH_GEMM) e = moe::launch_ffn_gemm(a, (hipStream_t)stream);
    else e = moe::launch_ffn_generic(a, (hipStream_t)stream);
    return from_hip(e, fn, (hipStream_t)stream);
}

moe_status moe_expert_ffn(const moe_layer_desc *L, const void *x, int32_t x_dt, int32_t n_tokens,
                          const int32_t *topk_idx, const int32_t *expert_offsets, const int32_t *perm,
                          const int32_t *active, float *slot_out, float *shared_out, void *ws, size_t ws_bytes,
                          void *stream) {
    return expert_call("moe_expert_ffn", moe::STAGE_GATE_UP | moe::STAGE_DOWN, L, x, x_dt, n_tokens, topk_idx,
                       expert_offsets, perm, active, slot_out, shared_out, ws, ws_bytes, stream);
}

moe_status moe_expert_ffn_noalloc(const moe_layer_desc *L, const void *x, int32_t x_dt, int32_t n_tokens,
                                  const int32_t *topk_idx, const int32_t *expert_offsets, const int32_t *perm,
                                  const int32_t *active, float *slot_out, float *shared_out, void *stream) {
    return expert_call("moe_expert_ffn_noalloc", moe::STAGE_GATE_UP | moe::STAGE_DOWN, L, x, x_dt, n_tokens,
                       topk_idx, expert_offsets, perm, active, slot_out, shared_out, nullptr, 0, stream, true);
}

moe_status moe_expert_gate_up(const moe_layer_desc *L, const void *x, int32_t x_dt, int32_t n_tokens,
                              const int32_t *topk_idx, const int32_t *expert_offsets, const int32_t *perm,
                              const int32_t *active, void *ws, size_t ws_bytes, void *stream) {
    return expert_call("moe_expert_gate_up", moe::STAGE_GATE_UP, L, x, x_dt, n_tokens, topk_idx, expert_offsets,
                       perm, active, nullptr, nullptr, ws, ws_bytes, stream);
}

moe_status moe_expert_down(const moe_layer_desc *L, const void *x, int32_t x_dt, int32_t n_tokens,
                           const int32_t *topk_idx, const int32_t *expert_offsets, const int32_t *perm,
                           const int32_t *active, float *slot_out, float *shared_out, void *ws, size_t ws_bytes,
                           void *stream) {
    return expert_call("moe_expert_down", moe::STAGE_DOWN, L, x, x_dt, n_tokens, topk_idx, expert_offsets, perm,
                       active, slot_out, shared_out, ws, ws_bytes, stream);
}

moe_status moe_combine(const float *slot_out, const float *topk_w, const float *shared_out, int32_t n_tokens,
                       int32_t top_k, int32_t hidden, float *y, void *stream) {
    if (!slot_out || !topk_w || !y) return fail(MOE_ERR_INVALID_ARG, "moe_combine: null pointer");
    if (n_tokens < 1 || top_k < 1 || hidden < 1) return fail(MOE_ERR_INVALID_ARG, "moe_combine: bad shape");
    if (!aligned(slot_out, 4) || !aligned(y, 4) || !aligned(topk_w, 4) || (shared_out && !aligned(shared_out, 4)))
        return fail(MOE_ERR_INVALID_ARG, "moe_combine: misaligned pointer");
    return from_hip(moe::launch_combine(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, y, (hipStream_t)stream),
                    "moe_combine", (hipStream_t)stream);
}

moe_status moe_combine_steer(const float *slot_out, const float *topk_w, const float *shared_out, int32_t n_tokens,
                             int32_t top_k, int32_t hidden, const float *steer_v, float steer_f, float *y,
                             void *stream) {
    if (!slot_out || !topk_w || !y || !steer_v) return fail(MOE_ERR_INVALID_ARG, "moe_combine_steer: null pointer");
    if (n_tokens < 1 || top_k < 1 || hidden < 1) return fail(MOE_ERR_INVALID_ARG, "moe_combine_steer: bad shape");
    if (!aligned(slot_out, 4) || !aligned(y, 4) || !aligned(topk_w, 4) || !aligned(steer_v, 4) ||
        (shared_out && !aligned(shared_out, 4)))
        return fail(MOE_ERR_INVALID_ARG, "moe_combine_steer: misaligned pointer");
    if (!std::isfinite(steer_f)) return fail(MOE_ERR_INVALID_ARG, "moe_combine_steer: steering strength not finite");
    return from_hip(moe::launch_combine_steer(slot_out, topk_w, shared_out, n_tokens, top_k, hidden, steer_v, steer_f,
                                              y, (hipStream_t)stream),
                    "moe_combine_steer", (hipStream_t)stream);
}

static size_t align256(size_t b) { return (b + 255) / 256 * 256; }

size_t moe_layer_workspace(const moe_layer_desc *L, int32_t n_tokens) {
    if (n_tokens < 1 || check_layer(L, "moe_layer_workspace") != MOE_OK) return 0;
    return align256(moe_route_workspace(n_tokens, L->n_experts, L->top_k)) + moe_expert_ffn_workspace(L, n_tokens);
}

moe_status moe_layer(const moe_layer_desc *L, const void *x, int32_t x_dt, int32_t n_tokens, const void *w_router,
                     int32_t w_dt, const float *bias, int32_t *topk_idx, float *topk_w, float *logits,
                     int32_t *expert_offsets, int32_t *perm, int32_t *active, float *slot_out, float *shared_out,
                     const float *steer_v, float steer_f, float *y, void *ws, size_t ws_bytes, void *stream) {
    const char *fn = "moe_layer";
    moe_status st = check_layer(L, fn);
    if (st != MOE_OK) return st;
    if (!y || !slot_out) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(y, 4) || (steer_v && !aligned(steer_v, 4)))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (steer_v && !std::isfinite(steer_f)) return fail(MOE_ERR_INVALID_ARG, "%s: steering strength not finite", fn);
    const size_t rws = align256(moe_route_workspace(n_tokens, L->n_experts, L->top_k));
    if (!ws || ws_bytes < rws) return fail(MOE_ERR_INVALID_ARG, "%s: workspace too small", fn);
    moe::RouteArgs ra;
    st = route_args(fn, x, x_dt, n_tokens, L->hidden, w_router, w_dt, L->n_experts, bias, L->top_k, topk_idx, topk_w,
                    logits, expert_offsets, perm, active, ws, rws, ra);
    if (st != MOE_OK) return st;
    void *fws = static_cast<char *>(ws) + rws;
    const size_t fbytes = ws_bytes - rws;
    // one token on the decode kernels: the routed gate/up workgroups select the token's experts from the logits
    // themselves, so routing takes one launch (the logits) instead of two
    moe::FfnArgs probe = make_args(L, x, x_dt, n_tokens);
    const bool in_kernel = n_tokens == 1 && L->top_k <= moe::SEL_MAXK && x_dt == MOE_DT_BF16 &&
                           choose_path(L, probe) == MOE_PATH_GEMV && moe::ffn_gemv_supported(probe);
    const hipStream_t hs = (hipStream_t)stream;
    if (in_kernel) {
        if ((st = from_hip(moe::launch_route_logits(ra, hs), fn, hs)) != MOE_OK) return st;
        const InKernelRoute r{ra.logits_ws, topk_idx, topk_w, expert_offsets, perm, active};
        st = expert_call(fn, moe::STAGE_GATE_UP, L, x, x_dt, n_tokens, topk_idx, expert_offsets, perm, active,
                         nullptr, nullptr, fws, fbytes, stream, false, &r);
        if (st != MOE_OK) return st;
        st = expert_call(fn, moe::STAGE_DOWN, L, x, x_dt, n_tokens, topk_idx, expert_offsets, perm, active, slot_out,
                         shared_out, fws, fbytes, stream);
    } else {
        if ((st = from_hip(moe::launch_route(ra, hs), fn, hs)) != MOE_OK) return st;
        st = expert_call(fn, moe::STAGE_GATE_UP | moe::STAGE_DOWN, L, x, x_dt, n_tokens, topk_idx, expert_offsets,
                         perm, active, slot_out, shared_out, fws, fbytes, stream);
    }
    if (st != MOE_OK) return st;
    const int T = n_tokens, k = L->top_k, H = L->hidden;
    if (steer_v)
        return from_hip(moe::launch_combine_steer(slot_out, topk_w, shared_out, T, k, H, steer_v, steer_f, y, hs), fn,
                        hs);
    return from_hip(moe::launch_combine(slot_out, topk_w, shared_out, T, k, H, y, hs), fn, hs);
}

// ---------------------------------------------------------------------------
// residual addition + RMS norm
// ---------------------------------------------------------------------------
static bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
    const char *a = static_cast<const char *>(p), *b = static_cast<const char *>(q);
    return a && b && a < b + qn && b < a + pn;
}

static size_t dt_bytes(int32_t dt) { return dt == MOE_DT_F32 ? 4 : dt == MOE_DT_BF16 ? 2 : 1; }

// Host checks of what the two norm calls share; fills `a` apart from the source row.
static moe_status norm_args(const char *fn, int32_t n_tokens, int32_t hidden, const void *residual,
                            void *residual_out, int32_t res_dt, const void *weight, int32_t w_dt, float eps, void *y,
                            int32_t y_dt, void *y_scale, moe::NormArgs &a) {
    memset(&a, 0, sizeof a);
    if (n_tokens < 1) return fail(MOE_ERR_INVALID_ARG, "%s: n_tokens < 1", fn);
    if (hidden < 1) return fail(MOE_ERR_INVALID_ARG, "%s: hidden < 1", fn);
    if (!weight || !y) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((residual == nullptr) != (residual_out == nullptr))
        return fail(MOE_ERR_INVALID_ARG, "%s: residual_out must be given iff residual is", fn);
    if ((residual && res_dt != MOE_DT_F32 && res_dt != MOE_DT_BF16) || (w_dt != MOE_DT_F32 && w_dt != MOE_DT_BF16))
        return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (y_dt < MOE_DT_F32 || y_dt > MOE_DT_E4M3_ROW) return fail(MOE_ERR_INVALID_ARG, "%s: unknown output dtype", fn);
    const bool scaled = y_dt == MOE_DT_E4M3_BLOCK || y_dt == MOE_DT_E4M3_ROW;
    if (scaled != (y_scale != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "%s: y_scale must be given iff y is e4m3", fn);
    if (!std::isfinite(eps) || eps < 0.f) return fail(MOE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
    if ((residual && (!aligned(residual, dt_bytes(res_dt)) || !aligned(residual_out, dt_bytes(res_dt)))) ||
        !aligned(weight, dt_bytes(w_dt)) || !aligned(y, dt_bytes(y_dt)) ||
        (y_dt == MOE_DT_E4M3_ROW && !aligned(y_scale, 4)))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t n = (size_t)n_tokens * hidden, rb = residual ? n * dt_bytes(res_dt) : 0, yb = n * dt_bytes(y_dt);
    const size_t sb = y_dt == MOE_DT_E4M3_ROW ? 4 * (size_t)n_tokens
                                              : (size_t)n_tokens * (((size_t)hidden + 31) / 32);
    const size_t wb = (size_t)hidden * dt_bytes(w_dt);
    if (overlap(y, yb, residual, rb) || overlap(y, yb, residual_out, rb) || overlap(y, yb, weight, wb) ||
        overlap(y, yb, y_scale, sb) || overlap(residual_out, rb, weight, wb) || overlap(residual_out, rb, y_scale, sb) ||
        overlap(y_scale, sb, residual, rb) || overlap(y_scale, sb, weight, wb) ||
        (residual != residual_out && overlap(residual_out, rb, residual, rb)))
        return fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps another buffer", fn);
    if (hidden > MOE_NORM_MAX_HIDDEN)
        return fail(MOE_ERR_UNSUPPORTED, "%s: hidden > %d", fn, MOE_NORM_MAX_HIDDEN);
    if (n_tokens > MOE_MAX_TOKENS)
        return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens > %d; split the batch", fn, MOE_MAX_TOKENS);
    a.T = n_tokens; a.H = hidden;
    a.residual = residual; a.residual_out = residual_out;
    a.res_kind = !residual ? moe::RES_NONE : res_dt == MOE_DT_F32 ? moe::RES_F32 : moe::RES_BF16;
    a.weight = weight; a.w_bf16 = w_dt == MOE_DT_BF16;
    a.eps = eps; a.inv_hidden = 1.0 / hidden;
    a.y = y; a.y_scale = y_scale;
    a.y_kind = y_dt == MOE_DT_F32 ? moe::NORM_F32 : y_dt == MOE_DT_BF16 ? moe::NORM_BF16
             : y_dt == MOE_DT_E4M3_BLOCK ? moe::NORM_MX8 : moe::NORM_ROW8;
    return MOE_OK;
}

// No output of a norm call may overlap its input `p` of `n` bytes.
static bool norm_writes(const moe::NormArgs &a, const void *p, size_t n) {
    const size_t e = (size_t)a.T * a.H;
    const size_t rb = a.res_kind == moe::RES_NONE ? 0 : e * (a.res_kind == moe::RES_F32 ? 4 : 2);
    const size_t yb = e * (a.y_kind == moe::NORM_F32 ? 4 : a.y_kind == moe::NORM_BF16 ? 2 : 1);
    const size_t sb = a.y_kind == moe::NORM_ROW8 ? 4 * (size_t)a.T : (size_t)a.T * (((size_t)a.H + 31) / 32);
    return overlap(p, n, a.residual_out, rb) || overlap(p, n, a.y, yb) || overlap(p, n, a.y_scale, sb);
}

moe_status moe_add_rms_norm(const void *x, int32_t x_dt, int32_t n_tokens, int32_t hidden, const void *residual,
                            void *residual_out, int32_t res_dt, const void *weight, int32_t w_dt, float eps, void *y,
                            int32_t y_dt, void *y_scale, void *stream) {
    const char *fn = "moe_add_rms_norm";
    if (!x) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (x_dt != MOE_DT_F32 && x_dt != MOE_DT_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!aligned(x, dt_bytes(x_dt))) return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    moe::NormArgs a;
    moe_status st = norm_args(fn, n_tokens, hidden, residual, residual_out, res_dt, weight, w_dt, eps, y, y_dt,
                              y_scale, a);
    if (st != MOE_OK) return st;
    if (norm_writes(a, x, (size_t)n_tokens * hidden * dt_bytes(x_dt)))
        return fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps x", fn);
    a.x = x; a.x_bf16 = x_dt == MOE_DT_BF16;
    return from_hip(moe::launch_norm(a, (hipStream_t)stream), fn, (hipStream_t)stream);
}

moe_status moe_combine_norm(const float *slot_out, const float *topk_w, const float *shared_out, int32_t n_tokens,
                            int32_t top_k, int32_t hidden, const float *steer_v, float steer_f, const void *residual,
                            void *residual_out, int32_t res_dt, const void *weight, int32_t w_dt, float eps, void *y,
                            int32_t y_dt, void *y_scale, void *stream) {
    const char *fn = "moe_combine_norm";
    if (!slot_out || !topk_w) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (top_k < 1) return fail(MOE_ERR_INVALID_ARG, "%s: bad shape", fn);
    if (!aligned(slot_out, 4) || !aligned(topk_w, 4) || (shared_out && !aligned(shared_out, 4)) ||
        (steer_v && !aligned(steer_v, 4)))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (steer_v && !std::isfinite(steer_f)) return fail(MOE_ERR_INVALID_ARG, "%s: steering strength not finite", fn);
    moe::NormArgs a;
    moe_status st = norm_args(fn, n_tokens, hidden, residual, residual_out, res_dt, weight, w_dt, eps, y, y_dt,
                              y_scale, a);
    if (st != MOE_OK) return st;
    const size_t row = (size_t)hidden * 4;
    if (norm_writes(a, slot_out, (size_t)n_tokens * top_k * row) || norm_writes(a, topk_w, (size_t)n_tokens * top_k * 4) ||
        (shared_out && norm_writes(a, shared_out, n_tokens * row)) || (steer_v && norm_writes(a, steer_v, row)))
        return fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    a.slot_out = slot_out; a.topk_w = topk_w; a.shared_out = shared_out; a.k = top_k;
    a.steer_v = steer_v; a.steer_f = steer_f;
    return from_hip(moe::launch_norm(a, (hipStream_t)stream), fn, (hipStream_t)stream);
}

// ---------------------------------------------------------------------------
// shared expert with low-rank adapters
// ---------------------------------------------------------------------------
static moe_status check_shared(const char *fn, const moe_layer_desc *L, const moe_adapter_desc *A, int32_t n_tokens) {
    if (!L) return fail(MOE_ERR_INVALID_ARG, "%s: null layer", fn);
    if (n_tokens < 1) return fail(MOE_ERR_INVALID_ARG, "%s: n_tokens < 1", fn);
    if (L->hidden < 8 || L->shared_inter < 8 || L->hidden % 8 || L->shared_inter % 8)
        return fail(MOE_ERR_INVALID_ARG, "%s: hidden and shared_inter must be positive multiples of 8", fn);
    if (L->hidden > MOE_SHARED_MAX_DIM || L->shared_inter > MOE_SHARED_MAX_DIM)
        return fail(MOE_ERR_UNSUPPORTED, "%s: hidden or shared_inter above %d", fn, MOE_SHARED_MAX_DIM);
    if (n_tokens > MOE_MAX_TOKENS)
        return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens > %d; split the batch", fn, MOE_MAX_TOKENS);
    if ((int64_t)n_tokens * (L->hidden > L->shared_inter ? L->hidden : L->shared_inter) >= (int64_t)1 << 30)
        return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens * hidden (or shared_inter) must be below 2^30; split the batch", fn);
    if (!L->shared_gate || !L->shared_up || !L->shared_down)
        return fail(MOE_ERR_INVALID_ARG, "%s: null shared expert weights", fn);
    if (!aligned(L->shared_gate, 16) || !aligned(L->shared_up, 16) || !aligned(L->shared_down, 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: shared expert weights not 16-byte aligned", fn);
    if (!A) return MOE_OK;
    if (A->n_adapters < 1 || A->n_adapters > MOE_MAX_ADAPTERS)
        return fail(MOE_ERR_INVALID_ARG, "%s: n_adapters outside [1, %d]", fn, MOE_MAX_ADAPTERS);
    if (A->max_rank < 8 || A->max_rank > MOE_MAX_RANK || A->max_rank % 8)
        return fail(MOE_ERR_INVALID_ARG, "%s: max_rank must be a multiple of 8 in [8, %d]", fn, MOE_MAX_RANK);
    const void *ab[3][2] = {{A->gate_a, A->gate_b}, {A->up_a, A->up_b}, {A->down_a, A->down_b}};
    for (const auto &p : ab) {
        if ((p[0] == nullptr) != (p[1] == nullptr))
            return fail(MOE_ERR_INVALID_ARG, "%s: both matrices of a projection's adapters, or neither", fn);
        if (!aligned(p[0], 16) || !aligned(p[1], 16))
            return fail(MOE_ERR_INVALID_ARG, "%s: adapter weights not 16-byte aligned", fn);
    }
    if (!aligned(A->rank, 4) || !aligned(A->scale, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer (adapter ranks or scales)", fn);
    return MOE_OK;
}

size_t moe_shared_ffn_workspace(const moe_layer_desc *L, const moe_adapter_desc *A, int32_t n_tokens) {
    if (check_shared("moe_shared_ffn_workspace", L, A, n_tokens) != MOE_OK) return 0;
    return moe::shared_workspace(n_tokens, L->hidden, L->shared_inter, A ? A->n_adapters : 0, A ? A->max_rank : 0);
}

moe_status moe_shared_ffn(const moe_layer_desc *L, const moe_adapter_desc *A, const void *x, int32_t x_dt,
                          int32_t n_tokens, const int32_t *token_adapter, void *out, int32_t out_dt, void *ws,
                          size_t ws_bytes, void *stream) {
    const char *fn = "moe_shared_ffn";
    moe_status st = check_shared(fn, L, A, n_tokens);
    if (st != MOE_OK) return st;
    if (!x || !out || !ws || (A && !token_adapter)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((x_dt != MOE_DT_F32 && x_dt != MOE_DT_BF16) || (out_dt != MOE_DT_F32 && out_dt != MOE_DT_BF16))
        return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(ws, 256) || !aligned(token_adapter, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer (x/out 16 B, ws 256 B)", fn);
    const size_t need = moe_shared_ffn_workspace(L, A, n_tokens);
    if (ws_bytes < need) return fail(MOE_ERR_INVALID_ARG, "%s: workspace too small (%zu < %zu)", fn, ws_bytes, need);
    const size_t n = (size_t)n_tokens * L->hidden, xb = n * dt_bytes(x_dt), ob = n * dt_bytes(out_dt);
    const size_t ib = A ? (size_t)n_tokens * 4 : 0;
    if (overlap(out, ob, x, xb) || overlap(ws, need, x, xb) || overlap(ws, need, out, ob) ||
        overlap(out, ob, token_adapter, ib) || overlap(ws, need, token_adapter, ib))
        return fail(MOE_ERR_INVALID_ARG, "%s: out or ws overlaps another buffer", fn);
    const size_t H = (size_t)L->hidden, Is = (size_t)L->shared_inter, wb = 2 * H * Is;
    const size_t an = A ? 2 * (size_t)A->n_adapters * A->max_rank : 0, sb = A ? 4 * (size_t)A->n_adapters : 0;
    const std::pair<const void *, size_t> weights[] = {
        {L->shared_gate, wb}, {L->shared_up, wb}, {L->shared_down, wb},
        {A ? A->gate_a : nullptr, an * H}, {A ? A->gate_b : nullptr, an * Is},
        {A ? A->up_a : nullptr, an * H}, {A ? A->up_b : nullptr, an * Is},
        {A ? A->down_a : nullptr, an * Is}, {A ? A->down_b : nullptr, an * H},
        {A ? A->rank : nullptr, sb}, {A ? A->scale : nullptr, sb}};
    for (const auto &w : weights)
        if (overlap(out, ob, w.first, w.second) || overlap(ws, need, w.first, w.second))
            return fail(MOE_ERR_INVALID_ARG, "%s: out or ws overlaps the layer's or the adapters' weights", fn);
    moe::SharedArgs a;
    memset(&a, 0, sizeof a);
    a.T = n_tokens; a.H = L->hidden; a.Is = L->shared_inter;
    a.x = x; a.x_bf16 = x_dt == MOE_DT_BF16;
    a.gate = static_cast<const uint16_t *>(L->shared_gate);
    a.up = static_cast<const uint16_t *>(L->shared_up);
    a.down = static_cast<const uint16_t *>(L->shared_down);
    if (A) {
        a.n = A->n_adapters; a.R = A->max_rank; a.rank = A->rank; a.scale = A->scale;
        a.gate_a = static_cast<const uint16_t *>(A->gate_a); a.gate_b = static_cast<const uint16_t *>(A->gate_b);
        a.up_a = static_cast<const uint16_t *>(A->up_a); a.up_b = static_cast<const uint16_t *>(A->up_b);
        a.down_a = static_cast<const uint16_t *>(A->down_a); a.down_b = static_cast<const uint16_t *>(A->down_b);
        a.token_adapter = token_adapter;
    }
    a.out = out; a.out_bf16 = out_dt == MOE_DT_BF16;
    return from_hip(moe::launch_shared(a, ws, (hipStream_t)stream), fn, (hipStream_t)stream);
}

// ---------------------------------------------------------------------------
// products over rows grouped by expert
// ---------------------------------------------------------------------------
struct Buffer {
    const void *p;
    size_t bytes;
};

static moe_status check_groups(const char *fn, const moe_group_desc *g, moe::Groups &o) {
    if (!g) return fail(MOE_ERR_INVALID_ARG, "%s: null group description", fn);
    if (g->n_groups < 1 || g->n_groups > MOE_MAX_GROUPS)
        return fail(MOE_ERR_INVALID_ARG, "%s: n_groups outside [1, %d]", fn, MOE_MAX_GROUPS);
    if (g->n_rows < 1) return fail(MOE_ERR_INVALID_ARG, "%s: n_rows < 1", fn);
    if (g->n_rows > MOE_MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_rows > %d; split the batch", fn, MOE_MAX_ROWS);
    if (!g->offsets && g->n_groups != 1)
        return fail(MOE_ERR_INVALID_ARG, "%s: offsets may be null for one group only", fn);
    if (g->in_div < 1) return fail(MOE_ERR_INVALID_ARG, "%s: in_div < 1", fn);
    if (!aligned(g->offsets, 4) || !aligned(g->in_index, 4) || !aligned(g->out_index, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer (offsets or indices)", fn);
    o.n = g->n_groups; o.rows = g->n_rows; o.offsets = g->offsets;
    o.in_index = g->in_index; o.in_div = g->in_div; o.out_index = g->out_index;
    // with 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d), m d - 2^(31+s) < d <= 2^s, so i m / 2^(31+s) is off i / d by less
    // than i / 2^31 / d < 1 / d: its integer part is that of i / d
    int shift = 0;
    while (((int64_t)1 << shift) < g->in_div) ++shift;
    o.div_mul = (uint32_t)((((uint64_t)1 << (31 + shift)) + g->in_div - 1) / g->in_div);
    o.div_shift = shift ? shift - 1 : 0;
    return MOE_OK;
}

// The output of a grouped product against what it reads.
static moe_status check_output(const char *fn, const moe::Groups &g, Buffer out, std::initializer_list<Buffer> read) {
    for (const Buffer &r : read)
        if (overlap(out.p, out.bytes, r.p, r.bytes)) return fail(MOE_ERR_INVALID_ARG, "%s: the output overlaps an input", fn);
    const size_t n = (size_t)g.rows * 4;
    if (overlap(out.p, out.bytes, g.offsets, ((size_t)g.n + 1) * 4) || overlap(out.p, out.bytes, g.in_index, n) ||
        overlap(out.p, out.bytes, g.out_index, n))
        return fail(MOE_ERR_INVALID_ARG, "%s: the output overlaps the offsets or an index", fn);
    return MOE_OK;
}

static moe_status check_dims(const char *fn, int32_t n_out, int32_t n_in) {
    if (n_out < 8 || n_in < 8 || n_out % 8 || n_in % 8)
        return fail(MOE_ERR_INVALID_ARG, "%s: n_out and n_in must be positive multiples of 8", fn);
    if (n_out > MOE_GROUPED_MAX_DIM || n_in > MOE_GROUPED_MAX_DIM)
        return fail(MOE_ERR_UNSUPPORTED, "%s: n_out or n_in above %d", fn, MOE_GROUPED_MAX_DIM);
    return MOE_OK;
}

static moe_status grouped_call(const char *fn, int op, const moe_group_desc *g, const void *a, int32_t a_rows,
                               const void *b, int32_t b_rows, int32_t n_out, int32_t n_in, int32_t act,
                               int32_t accumulate, void *out, int32_t out_dt, int32_t out_rows, void *stream) {
    moe::GroupedArgs p;
    memset(&p, 0, sizeof p);
    moe_status st = check_groups(fn, g, p.g);
    if (st != MOE_OK || (st = check_dims(fn, n_out, n_in)) != MOE_OK) return st;
    const bool wgrad = op == moe::GROUPED_WGRAD;
    if (!a || !b || !out) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer (16 B)", fn);
    if (a_rows < 1 || (wgrad && b_rows < 1) || (!wgrad && out_rows < 1))
        return fail(MOE_ERR_INVALID_ARG, "%s: a buffer without rows", fn);
    if (out_dt != MOE_DT_F32 && out_dt != MOE_DT_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown output dtype", fn);
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return fail(MOE_ERR_INVALID_ARG, "%s: unknown activation", fn);
    const size_t weights = (size_t)g->n_groups * n_out * n_in * (act == MOE_ACT_SWIGLU ? 2 : 1);
    const size_t in_cols = op == moe::GROUPED_DGRAD ? n_out : n_in, out_cols = op == moe::GROUPED_DGRAD ? n_in : n_out;
    const Buffer o{out, (wgrad ? weights : (size_t)out_rows * out_cols) * dt_bytes(out_dt)};
    st = check_output(fn, p.g, o, {{a, (size_t)a_rows * in_cols * 2}, {b, (wgrad ? (size_t)b_rows * n_out : weights) * 2}});
    if (st != MOE_OK) return st;
    p.a = static_cast<const uint16_t *>(a); p.a_rows = a_rows;
    p.b = static_cast<const uint16_t *>(b); p.b_rows = b_rows;
    p.n_out = n_out; p.n_in = n_in;
    p.swiglu = act == MOE_ACT_SWIGLU; p.accumulate = accumulate != 0;
    p.out = out; p.out_bf16 = out_dt == MOE_DT_BF16; p.out_rows = out_rows;
    const hipError_t e = moe::launch_grouped(op, p, (hipStream_t)stream);
    if (e == hipErrorInvalidConfiguration) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles; split the batch", fn);
    return from_hip(e, fn, (hipStream_t)stream);
}

moe_status moe_grouped_linear(const moe_group_desc *g, const void *x, int32_t x_rows, const void *w, int32_t n_out,
                              int32_t n_in, int32_t act, void *out, int32_t out_dt, int32_t out_rows, void *stream) {
    return grouped_call("moe_grouped_linear", moe::GROUPED_FWD, g, x, x_rows, w, 0, n_out, n_in, act, 0, out, out_dt,
                        out_rows, stream);
}

moe_status moe_grouped_dgrad(const moe_group_desc *g, const void *dy, int32_t dy_rows, const void *w, int32_t n_out,
                             int32_t n_in, void *dx, int32_t dx_dt, int32_t dx_rows, void *stream) {
    return grouped_call("moe_grouped_dgrad", moe::GROUPED_DGRAD, g, dy, dy_rows, w, 0, n_out, n_in, MOE_ACT_NONE, 0, dx,
                        dx_dt, dx_rows, stream);
}

moe_status moe_grouped_wgrad(const moe_group_desc *g, const void *x, int32_t x_rows, const void *dy, int32_t dy_rows,
                             int32_t n_out, int32_t n_in, int32_t accumulate, void *dw, int32_t dw_dt, void *stream) {
    return grouped_call("moe_grouped_wgrad", moe::GROUPED_WGRAD, g, x, x_rows, dy, dy_rows, n_out, n_in, MOE_ACT_NONE,
                        accumulate, dw, dw_dt, 0, stream);
}

moe_status moe_q4_linear(const moe_group_desc *g, const moe_q4_desc *w, const void *x, int32_t x_rows, int32_t act,
                         void *out, int32_t out_dt, int32_t out_rows, void *stream) {
    const char *fn = "moe_q4_linear";
    moe::Q4Args p;
    memset(&p, 0, sizeof p);
    moe_status st = check_groups(fn, g, p.g);
    if (st != MOE_OK) return st;
    if (!w || !x || !out || !w->codes || !w->scale) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (w->n_mats != g->n_groups) return fail(MOE_ERR_INVALID_ARG, "%s: %d matrices for %d groups", fn, w->n_mats, g->n_groups);
    if (w->group != 32 && w->group != 64 && w->group != 128)
        return fail(MOE_ERR_INVALID_ARG, "%s: group must be 32, 64 or 128", fn);
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return fail(MOE_ERR_INVALID_ARG, "%s: unknown activation", fn);
    if (w->rows < 1 || w->cols < 1 || w->cols % w->group || (act == MOE_ACT_SWIGLU && w->rows % 2))
        return fail(MOE_ERR_INVALID_ARG, "%s: cols must be a positive multiple of group, rows positive (SwiGLU: even)", fn);
    if (w->rows > MOE_GROUPED_MAX_DIM || w->cols > MOE_GROUPED_MAX_DIM)
        return fail(MOE_ERR_UNSUPPORTED, "%s: rows or cols above %d", fn, MOE_GROUPED_MAX_DIM);
    if ((w->scale_dt != MOE_DT_F32 && w->scale_dt != MOE_DT_BF16 && w->scale_dt != MOE_DT_F16) ||
        (out_dt != MOE_DT_F32 && out_dt != MOE_DT_BF16))
        return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    const size_t sb = w->scale_dt == MOE_DT_F32 ? 4 : 2;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(w->codes, 16) || !aligned(w->scale, sb))
        return fail(MOE_ERR_INVALID_ARG, "%s: misaligned pointer (x, out and codes 16 B)", fn);
    if (x_rows < 1 || out_rows < 1) return fail(MOE_ERR_INVALID_ARG, "%s: a buffer without rows", fn);
    p.N = act == MOE_ACT_SWIGLU ? w->rows / 2 : w->rows;
    p.K = w->cols; p.group = w->group;
    const size_t values = (size_t)w->n_mats * w->rows * w->cols, groups = values / w->group;
    st = check_output(fn, p.g, {out, (size_t)out_rows * p.N * dt_bytes(out_dt)},
                      {{x, (size_t)x_rows * p.K * 2}, {w->codes, values / 2}, {w->scale, groups * sb}, {w->zero, groups}});
    if (st != MOE_OK) return st;
    p.x = static_cast<const uint16_t *>(x); p.x_rows = x_rows;
    p.codes = static_cast<const uint8_t *>(w->codes);
    p.scale = w->scale; p.zero = w->zero;
    p.scale_kind = w->scale_dt == MOE_DT_F32 ? moe::Q4_F32 : w->scale_dt == MOE_DT_BF16 ? moe::Q4_BF16 : moe::Q4_F16;
    p.swiglu = act == MOE_ACT_SWIGLU;
    p.out = out; p.out_bf16 = out_dt == MOE_DT_BF16; p.out_rows = out_rows;
    const hipError_t e = moe::launch_q4(p, (hipStream_t)stream);
    if (e == hipErrorInvalidConfiguration) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles; split the batch", fn);
    return from_hip(e, fn, (hipStream_t)stream);
}

moe_status moe_probe_stream_read(const void *buf, size_t bytes, uint32_t *sink, int32_t n_blocks, void *stream) {
    if (!buf || !sink) return fail(MOE_ERR_INVALID_ARG, "moe_probe_stream_read: null pointer");
    if (bytes < 16 || bytes % 16 || !aligned(buf, 16) || !aligned(sink, 4))
        return fail(MOE_ERR_INVALID_ARG, "moe_probe_stream_read: need a 16-byte aligned, non-empty multiple of 16 bytes");
    if (n_blocks < 1 || n_blocks > (1 << 20))
        return fail(MOE_ERR_INVALID_ARG, "moe_probe_stream_read: n_blocks outside [1, 2^20]");
    return from_hip(moe::launch_stream_read(buf, (int64_t)bytes, sink, n_blocks, (hipStream_t)stream),
                    "moe_probe_stream_read", (hipStream_t)stream);
}

}  // extern "C"
