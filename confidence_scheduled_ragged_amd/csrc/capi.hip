// capi.hip - the exported C ABI: host-side argument checks, then launches on
// the caller's stream. No allocation, no synchronisation, no per-call state.
#include <atomic>
#include <cmath>
#include <mutex>

#include "forward.hpp"

#define DSPARK_API extern "C" __attribute__((visibility("default")))

namespace dspark {

int device_cu_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) dev = 0;
    if (dev >= 0 && dev < 64) {
        int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n <= 0)
        n = 256;
    if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(u32x4 *p, size_t n16) {
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16;
         i += (size_t)gridDim.x * blockDim.x)
        p[i] = u32x4{0u, 0u, 0u, 0u};
}

__global__ void step_status_kernel(unsigned *flag, int32_t *status) {
    if (threadIdx.x == 0)
        *status = (int32_t)__hip_atomic_exchange(flag, 0u, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT);
}

hipError_t launch_step_status(void *ws, int32_t *status, hipStream_t s) {
    unsigned *flag = reinterpret_cast<unsigned *>(static_cast<char *>(ws) + ws_ctrl_offset() +
                                                  kCtrlTimedOutOffset);
    hipLaunchKernelGGL(step_status_kernel, dim3(1), dim3(64), 0, s, flag, status);
    return hipGetLastError();
}

hipError_t launch_fill_zero(void *ws, size_t bytes, hipStream_t s) {
    const size_t n16 = bytes / 16;
    if (n16 == 0) return hipSuccess;
    size_t g = (n16 + 255) / 256;
    g = g > 1024 ? 1024 : g;
    hipLaunchKernelGGL(fill_zero_kernel, dim3((unsigned)g), dim3(256), 0, s,
                       static_cast<u32x4 *>(ws), n16);
    return hipGetLastError();
}

}  // namespace dspark

using namespace dspark;

namespace {

constexpr int kMaxD = 1 << 20;
constexpr int kMaxTiers = 4096;

inline bool misaligned(const void *p, size_t a) { return p && ((uintptr_t)p % a) != 0; }

inline dspark_status check_bg(int B, int gamma) {
    if (B < 1 || gamma < 1 || gamma > DSPARK_MAX_GAMMA) return DSPARK_ERR_SHAPE;
    if ((int64_t)B * (gamma + 1) > (int64_t)DSPARK_MAX_ROWS) return DSPARK_ERR_SHAPE;
    return DSPARK_OK;
}

inline bool valid_mode(int mode) {
    return mode == DSPARK_CUT_THRESHOLD || mode == DSPARK_CUT_BUDGET ||
           mode == DSPARK_CUT_STATIC || mode == DSPARK_CUT_COMBINED;
}

inline bool needs_cutoff(int mode) {
    return mode == DSPARK_CUT_THRESHOLD || mode == DSPARK_CUT_COMBINED;
}

inline bool needs_budget(int mode) {
    return mode == DSPARK_CUT_BUDGET || mode == DSPARK_CUT_COMBINED;
}

inline dspark_status launched(hipError_t e) { return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP; }

inline hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

}  // namespace

DSPARK_API const char *dspark_status_string(int status) {
    switch (status) {
        case DSPARK_OK: return "ok";
        case DSPARK_ERR_NULL: return "a required pointer is NULL";
        case DSPARK_ERR_SHAPE: return "a size is out of range";
        case DSPARK_ERR_ARG: return "an argument value is invalid";
        case DSPARK_ERR_ALIGN: return "a pointer is misaligned for its element type";
        case DSPARK_ERR_WORKSPACE: return "the workspace is too small";
        case DSPARK_ERR_HIP: return "a HIP kernel launch failed";
        default: return "unknown status";
    }
}

DSPARK_API size_t dspark_workspace_bytes(int B, int gamma, int V) {
    if (check_bg(B, gamma) != DSPARK_OK || V < 1) return 0;
    return ws_total_bytes(B, gamma);
}

DSPARK_API dspark_status dspark_workspace_init(void *ws, size_t ws_bytes, void *stream) {
    if (!ws) return DSPARK_ERR_NULL;
    if (misaligned(ws, 16)) return DSPARK_ERR_ALIGN;
    return launched(launch_fill_zero(ws, ws_bytes & ~(size_t)15, as_stream(stream)));
}

DSPARK_API dspark_status dspark_confidence(const dspark_bf16 *hidden, const dspark_bf16 *w,
                                           float bias, const float *temps, int B, int gamma, int d,
                                           float *conf, float *survival, void *stream) {
    if (!hidden || !w || !temps || !conf || !survival) return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (d < 1 || d > kMaxD) return DSPARK_ERR_SHAPE;
    if (!std::isfinite(bias)) return DSPARK_ERR_ARG;
    if (misaligned(hidden, 2) || misaligned(w, 2) || misaligned(temps, 4) || misaligned(conf, 4) ||
        misaligned(survival, 4))
        return DSPARK_ERR_ALIGN;
    return launched(launch_confidence(hidden, w, bias, temps, B, gamma, d, conf, survival,
                                      as_stream(stream)));
}

DSPARK_API dspark_status dspark_schedule(const float *survival, int B, int gamma, int mode,
                                         const float *cutoff, long long budget, int32_t *lengths,
                                         void *stream) {
    if (!survival || !lengths) return DSPARK_ERR_NULL;
    if (needs_cutoff(mode) && !cutoff) return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (!valid_mode(mode)) return DSPARK_ERR_ARG;
    if (needs_budget(mode) && budget < 0) return DSPARK_ERR_ARG;
    if (misaligned(survival, 4) || misaligned(cutoff, 4) || misaligned(lengths, 4))
        return DSPARK_ERR_ALIGN;
    return launched(launch_schedule(survival, B, gamma, mode, cutoff, budget, lengths,
                                    as_stream(stream)));
}

DSPARK_API dspark_status dspark_compact(const int32_t *lengths, const int32_t *tokens, int B,
                                        int gamma, int32_t *cu_seqlens, int32_t *packed_tokens,
                                        int32_t *packed_src_row, const dspark_bf16 *logits, int V,
                                        dspark_bf16 *packed_logits, void *stream) {
    if (!lengths || !tokens || !cu_seqlens || !packed_tokens || !packed_src_row)
        return DSPARK_ERR_NULL;
    if ((logits == nullptr) != (packed_logits == nullptr)) return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (logits && V < 1) return DSPARK_ERR_SHAPE;
    if (misaligned(lengths, 4) || misaligned(tokens, 4) || misaligned(cu_seqlens, 4) ||
        misaligned(packed_tokens, 4) || misaligned(packed_src_row, 4) || misaligned(logits, 2) ||
        misaligned(packed_logits, 2))
        return DSPARK_ERR_ALIGN;
    hipStream_t s = as_stream(stream);
    hipError_t e = launch_compact(lengths, tokens, B, gamma, cu_seqlens, packed_tokens,
                                  packed_src_row, s);
    if (e == hipSuccess && logits)
        e = launch_gather_rows(logits, packed_src_row, cu_seqlens, B, gamma, (int64_t)V * 2,
                               packed_logits, s);
    return launched(e);
}

DSPARK_API dspark_status dspark_gather_rows(const void *src, const int32_t *packed_src_row,
                                            const int32_t *cu_seqlens, int B, int gamma,
                                            long long row_bytes, void *dst, void *stream) {
    if (!src || !packed_src_row || !cu_seqlens || !dst) return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    // the source and destination each span B*(gamma+1) rows: keep their byte size
    // within 2^48 so no offset computation can overflow
    if (row_bytes < 1 || row_bytes > ((long long)1 << 48) / ((long long)B * (gamma + 1)))
        return DSPARK_ERR_SHAPE;
    if (misaligned(packed_src_row, 4) || misaligned(cu_seqlens, 4)) return DSPARK_ERR_ALIGN;
    return launched(launch_gather_rows(src, packed_src_row, cu_seqlens, B, gamma,
                                       (int64_t)row_bytes, dst, as_stream(stream)));
}

DSPARK_API dspark_status dspark_tier_select(const int32_t *cu_seqlens, int B, int gamma,
                                            const int32_t *tiers, int ntiers, int32_t pad_token,
                                            int32_t *padded_total, int32_t *tier_index,
                                            int32_t *packed_tokens, int32_t *packed_src_row,
                                            void *stream) {
    if (!cu_seqlens || !tiers || !padded_total || !tier_index) return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (ntiers < 1 || ntiers > kMaxTiers) return DSPARK_ERR_SHAPE;
    if (misaligned(cu_seqlens, 4) || misaligned(tiers, 4) || misaligned(padded_total, 4) ||
        misaligned(tier_index, 4) || misaligned(packed_tokens, 4) || misaligned(packed_src_row, 4))
        return DSPARK_ERR_ALIGN;
    return launched(launch_tier_select(cu_seqlens, B, gamma, tiers, ntiers, pad_token,
                                       padded_total, tier_index, packed_tokens, packed_src_row,
                                       as_stream(stream)));
}

DSPARK_API dspark_status dspark_cost_cutoff(const float *table, int n, const int32_t *load,
                                            int B, float *cutoff, void *stream) {
    if (!table || !load || !cutoff) return DSPARK_ERR_NULL;
    if (n < 1 || B < 1 || B > DSPARK_MAX_ROWS) return DSPARK_ERR_SHAPE;
    if (misaligned(table, 4) || misaligned(load, 4) || misaligned(cutoff, 4))
        return DSPARK_ERR_ALIGN;
    return launched(launch_cost_cutoff(table, n, load, B, cutoff, as_stream(stream)));
}

DSPARK_API dspark_status dspark_accept(const dspark_bf16 *logits, const int32_t *packed_src_row,
                                       const int32_t *cu_seqlens, const int32_t *tokens, int B,
                                       int gamma, int V, int32_t *packed_argmax, int32_t *accepted,
                                       int32_t *bonus, void *ws, size_t ws_bytes, void *stream) {
    if (!logits || !cu_seqlens || !tokens || !packed_argmax || !accepted || !bonus || !ws)
        return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (V < 1) return DSPARK_ERR_SHAPE;
    if (misaligned(logits, 2) || misaligned(packed_src_row, 4) || misaligned(cu_seqlens, 4) ||
        misaligned(tokens, 4) || misaligned(packed_argmax, 4) || misaligned(accepted, 4) ||
        misaligned(bonus, 4) || misaligned(ws, 16))
        return DSPARK_ERR_ALIGN;
    if (ws_bytes < ws_total_bytes(B, gamma)) return DSPARK_ERR_WORKSPACE;
    return launched(launch_accept(logits, packed_src_row, cu_seqlens, tokens, B, gamma, V,
                                  packed_argmax, accepted, bonus, ws, as_stream(stream)));
}

DSPARK_API dspark_status dspark_cap_accept(const int32_t *packed_argmax_full,
                                           const int32_t *tokens, const int32_t *lengths, int B,
                                           int gamma, int32_t *accepted, int32_t *bonus,
                                           int32_t *accepted_full, long long *sums,
                                           void *stream) {
    if (!packed_argmax_full || !tokens || !lengths || !accepted || !bonus || !accepted_full)
        return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (misaligned(packed_argmax_full, 4) || misaligned(tokens, 4) || misaligned(lengths, 4) ||
        misaligned(accepted, 4) || misaligned(bonus, 4) || misaligned(accepted_full, 4) ||
        misaligned(sums, 8))
        return DSPARK_ERR_ALIGN;
    return launched(launch_cap_accept(packed_argmax_full, tokens, lengths, B, gamma, accepted,
                                      bonus, accepted_full, sums, as_stream(stream)));
}

// Host-side checks of the fused step's arguments (every one but the workspace).
static dspark_status step_check(const dspark_bf16 *hidden, const dspark_bf16 *w, float bias,
                                const float *temps, const int32_t *tokens,
                                const dspark_bf16 *logits, int B, int gamma, int d, int V,
                                int mode, const float *cutoff, long long budget, float *conf,
                                float *survival, int32_t *lengths, int32_t *cu_seqlens,
                                int32_t *packed_tokens, int32_t *packed_src_row,
                                int32_t *packed_argmax, int32_t *accepted, int32_t *bonus,
                                int launches) {
    if (!hidden || !w || !temps || !tokens || !logits || !lengths || !cu_seqlens ||
        !packed_tokens || !packed_src_row || !packed_argmax || !accepted || !bonus)
        return DSPARK_ERR_NULL;
    if (needs_cutoff(mode) && !cutoff) return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (d < 1 || d > kMaxD || V < 1) return DSPARK_ERR_SHAPE;
    if (!valid_mode(mode)) return DSPARK_ERR_ARG;
    if (needs_budget(mode) && budget < 0) return DSPARK_ERR_ARG;
    if (!std::isfinite(bias)) return DSPARK_ERR_ARG;
    if (launches < 0 || launches > 2) return DSPARK_ERR_ARG;
    if (misaligned(hidden, 2) || misaligned(w, 2) || misaligned(temps, 4) ||
        misaligned(tokens, 4) || misaligned(logits, 2) || misaligned(cutoff, 4) ||
        misaligned(conf, 4) || misaligned(survival, 4) || misaligned(lengths, 4) ||
        misaligned(cu_seqlens, 4) || misaligned(packed_tokens, 4) ||
        misaligned(packed_src_row, 4) || misaligned(packed_argmax, 4) ||
        misaligned(accepted, 4) || misaligned(bonus, 4))
        return DSPARK_ERR_ALIGN;
    return DSPARK_OK;
}

// The fused step's launches, after every check has passed.
static dspark_status step_launch(const dspark_bf16 *hidden, const dspark_bf16 *w, float bias,
                                 const float *temps, const int32_t *tokens,
                                 const dspark_bf16 *logits, int B, int gamma, int d, int V,
                                 int mode, const float *cutoff, long long budget, float *conf,
                                 float *survival, int32_t *lengths, int32_t *cu_seqlens,
                                 int32_t *packed_tokens, int32_t *packed_src_row,
                                 int32_t *packed_argmax, int32_t *accepted, int32_t *bonus,
                                 void *ws, hipStream_t s, void *ev_start, void *ev_stop,
                                 int launches, unsigned long long wait_ticks) {
    char *wsb = static_cast<char *>(ws);
    float *surv = survival ? survival : reinterpret_cast<float *>(wsb + ws_surv_offset(B, gamma));
    float *cf = conf ? conf : reinterpret_cast<float *>(wsb + ws_conf_offset(B, gamma));
    hipEvent_t es = static_cast<hipEvent_t>(ev_start), et = static_cast<hipEvent_t>(ev_stop);
    auto fused = fused_slots_fit_32(B, gamma, V, logits) ? slots32::launch_fused_step
                                                         : slots64::launch_fused_step;
    hipError_t e = fused(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode, cutoff,
                         budget, cf, surv, lengths, cu_seqlens, packed_tokens, packed_src_row,
                         packed_argmax, accepted, bonus, ws, s, es, et, launches, wait_ticks);
    if (e != hipErrorNotSupported) return launched(e);
    // sizes outside the fused kernels' limits: the same step through the stage kernels
    e = launch_confidence(hidden, w, bias, temps, B, gamma, d, cf, surv, s);
    if (e == hipSuccess) e = launch_schedule(surv, B, gamma, mode, cutoff, budget, lengths, s);
    if (e == hipSuccess)
        e = launch_compact(lengths, tokens, B, gamma, cu_seqlens, packed_tokens, packed_src_row, s);
    if (e == hipSuccess && es) e = hipEventRecord(es, s);
    if (e == hipSuccess)
        e = launch_accept(logits, packed_src_row, cu_seqlens, tokens, B, gamma, V, packed_argmax,
                          accepted, bonus, ws, s);
    if (e == hipSuccess && et) e = hipEventRecord(et, s);
    return launched(e);
}

static dspark_status step_impl(const dspark_bf16 *hidden, const dspark_bf16 *w, float bias,
                               const float *temps, const int32_t *tokens,
                               const dspark_bf16 *logits, int B, int gamma, int d, int V,
                               int mode, const float *cutoff, long long budget, float *conf,
                               float *survival, int32_t *lengths, int32_t *cu_seqlens,
                               int32_t *packed_tokens, int32_t *packed_src_row,
                               int32_t *packed_argmax, int32_t *accepted, int32_t *bonus,
                               void *ws, size_t ws_bytes, void *stream, void *ev_start,
                               void *ev_stop, int launches, unsigned long long wait_ticks) {
    if (dspark_status st = step_check(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode,
                                      cutoff, budget, conf, survival, lengths, cu_seqlens,
                                      packed_tokens, packed_src_row, packed_argmax, accepted,
                                      bonus, launches))
        return st;
    if (!ws) return DSPARK_ERR_NULL;
    if (misaligned(ws, 16)) return DSPARK_ERR_ALIGN;
    if (ws_bytes < ws_total_bytes(B, gamma)) return DSPARK_ERR_WORKSPACE;
    return step_launch(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode, cutoff,
                       budget, conf, survival, lengths, cu_seqlens, packed_tokens, packed_src_row,
                       packed_argmax, accepted, bonus, ws, as_stream(stream), ev_start, ev_stop,
                       launches, wait_ticks);
}

DSPARK_API dspark_status dspark_step(const dspark_bf16 *hidden, const dspark_bf16 *w, float bias,
                                     const float *temps, const int32_t *tokens,
                                     const dspark_bf16 *logits, int B, int gamma, int d, int V,
                                     int mode, const float *cutoff, long long budget, float *conf,
                                     float *survival, int32_t *lengths, int32_t *cu_seqlens,
                                     int32_t *packed_tokens, int32_t *packed_src_row,
                                     int32_t *packed_argmax, int32_t *accepted, int32_t *bonus,
                                     void *ws, size_t ws_bytes, void *stream) {
    return step_impl(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode, cutoff, budget,
                     conf, survival, lengths, cu_seqlens, packed_tokens, packed_src_row,
                     packed_argmax, accepted, bonus, ws, ws_bytes, stream, nullptr, nullptr, 0, 0);
}

DSPARK_API dspark_status dspark_step_ex(
    const dspark_bf16 *hidden, const dspark_bf16 *w, float bias, const float *temps,
    const int32_t *tokens, const dspark_bf16 *logits, int B, int gamma, int d, int V, int mode,
    const float *cutoff, long long budget, float *conf, float *survival, int32_t *lengths,
    int32_t *cu_seqlens, int32_t *packed_tokens, int32_t *packed_src_row, int32_t *packed_argmax,
    int32_t *accepted, int32_t *bonus, void *ws, size_t ws_bytes, void *stream, void *ev_start,
    void *ev_stop, int launches, unsigned long long wait_ticks) {
    return step_impl(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode, cutoff, budget,
                     conf, survival, lengths, cu_seqlens, packed_tokens, packed_src_row,
                     packed_argmax, accepted, bonus, ws, ws_bytes, stream, ev_start, ev_stop,
                     launches, wait_ticks);
}

DSPARK_API dspark_status dspark_step_status(void *ws, int32_t *status, void *stream) {
    if (!ws || !status) return DSPARK_ERR_NULL;
    if (misaligned(ws, 16) || misaligned(status, 4)) return DSPARK_ERR_ALIGN;
    return launched(launch_step_status(ws, status, as_stream(stream)));
}

// ------------------------------------------------------------ no allocation

// The workspace of dspark_step_noalloc: one array per device, in the code
// object's own device memory, so the call allocates nothing. In host code the
// name `scratch` is only a stand-in for the symbol; its device address (one per
// device) comes from hipGetSymbolAddress and is the only pointer ever passed to
// a kernel or a fill.
constexpr size_t kNoallocScratchBytes = (size_t)4 << 20;
static __device__ __align__(256) unsigned char scratch[kNoallocScratchBytes];

namespace {
std::mutex g_scratch_mu;
void *g_scratch_ptr[64];  // device address of `scratch` per device, once set up
}  // namespace

// The current device's scratch address. The first call on a device looks it up
// and zero-fills the array on `s` (the fused step's control words and counters
// must start at zero; every call returns them to zero).
static dspark_status noalloc_scratch(void **out, hipStream_t s) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return DSPARK_ERR_HIP;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p)
            return DSPARK_ERR_HIP;
        if (launch_fill_zero(p, kNoallocScratchBytes, s) != hipSuccess) return DSPARK_ERR_HIP;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return DSPARK_OK;
}

DSPARK_API dspark_status dspark_step_noalloc(
    const dspark_bf16 *hidden, const dspark_bf16 *w, float bias, const float *temps,
    const int32_t *tokens, const dspark_bf16 *logits, int B, int gamma, int d, int V, int mode,
    const float *cutoff, long long budget, float *conf, float *survival, int32_t *lengths,
    int32_t *cu_seqlens, int32_t *packed_tokens, int32_t *packed_src_row, int32_t *packed_argmax,
    int32_t *accepted, int32_t *bonus, int32_t *status, void *stream) {
    if (dspark_status st = step_check(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode,
                                      cutoff, budget, conf, survival, lengths, cu_seqlens,
                                      packed_tokens, packed_src_row, packed_argmax, accepted,
                                      bonus, 0))
        return st;
    if (ws_total_bytes(B, gamma) > kNoallocScratchBytes) return DSPARK_ERR_WORKSPACE;
    if (misaligned(status, 4)) return DSPARK_ERR_ALIGN;
    hipStream_t s = as_stream(stream);
    void *ws = nullptr;
    if (dspark_status st = noalloc_scratch(&ws, s)) return st;
    dspark_status st = step_launch(hidden, w, bias, temps, tokens, logits, B, gamma, d, V, mode,
                                   cutoff, budget, conf, survival, lengths, cu_seqlens,
                                   packed_tokens, packed_src_row, packed_argmax, accepted, bonus,
                                   ws, s, nullptr, nullptr, 0, 0);
    if (st == DSPARK_OK && status) st = launched(launch_step_status(ws, status, s));
    return st;
}

namespace {

constexpr int kMaxHeads = 4096;

// The checks that appending to the paged cache and reading it share.
dspark_status check_paged(const void *k_cache, const void *v_cache, int cache_type, int pages,
                          int page_size, long long page_stride, long long head_stride,
                          long long slot_stride, float k_scale, float v_scale, int table_width,
                          int B, int rows, int Hq, int Hkv, int D, int max_d) {
    if (B < 1 || rows < 1 || rows > DSPARK_MAX_ROWS || B > DSPARK_MAX_ROWS) return DSPARK_ERR_SHAPE;
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > kMaxHeads) return DSPARK_ERR_SHAPE;
    if (D < 1 || D > max_d || pages < 1 || page_size < 1 || table_width < 1) return DSPARK_ERR_SHAPE;
    if ((long long)rows * Hq > 0x7FFFFFFFll) return DSPARK_ERR_SHAPE;
    // positions are 32-bit
    if ((long long)table_width * page_size > 0x7FFFFFFFll) return DSPARK_ERR_SHAPE;
    if (cache_type != DSPARK_CACHE_BF16 && cache_type != DSPARK_CACHE_E4M3) return DSPARK_ERR_ARG;
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f)
        return DSPARK_ERR_ARG;
    if (page_stride < 0 || head_stride < 0 || slot_stride < 0) return DSPARK_ERR_ARG;
    const size_t item = cache_type == DSPARK_CACHE_E4M3 ? 1 : 2;
    if (misaligned(k_cache, item) || misaligned(v_cache, item)) return DSPARK_ERR_ALIGN;
    return DSPARK_OK;
}

PagedCache paged(const void *k_cache, const void *v_cache, int pages, int page_size,
                 long long page_stride, long long head_stride, long long slot_stride,
                 float k_scale, float v_scale, bool scaled, const int32_t *table,
                 int table_width) {
    PagedCache c;
    c.k = const_cast<void *>(k_cache);
    c.v = const_cast<void *>(v_cache);
    c.table = table;
    c.table_width = table_width;
    c.pages = pages;
    set_page_size(c, page_size);
    c.page_stride = page_stride;
    c.head_stride = head_stride;
    c.slot_stride = slot_stride;
    c.k_scale = scaled ? k_scale : 1.f;
    c.v_scale = scaled ? v_scale : 1.f;
    return c;
}

}  // namespace

// depths: of the nodes of drafted trees, or NULL for chains.
static dspark_status append_rows(
    const dspark_bf16 *q, const dspark_bf16 *k, const dspark_bf16 *v, long long q_stride,
    long long k_stride, long long v_stride, const float *cos, const float *sin, int positions,
    int half, int interleaved, const int32_t *depths, const int32_t *cu_seqlens,
    const int32_t *ctx_lens, int B, int rows, int Hq, int Hkv, int D, void *k_cache,
    void *v_cache, int cache_type, int pages, int page_size, long long page_stride,
    long long head_stride, long long slot_stride, float k_scale, float v_scale,
    const int32_t *block_table, int table_width, dspark_bf16 *q_out, void *stream) {
    if (!q || !k || !v || !cu_seqlens || !ctx_lens || !k_cache || !v_cache || !block_table || !q_out)
        return DSPARK_ERR_NULL;
    if (half > 0 && (!cos || !sin)) return DSPARK_ERR_NULL;
    if (dspark_status st = check_paged(k_cache, v_cache, cache_type, pages, page_size, page_stride,
                                       head_stride, slot_stride, k_scale, v_scale, table_width, B,
                                       rows, Hq, Hkv, D, 1024))
        return st;
    if (positions < 1 || half < 0 || 2 * (long long)half > D) return DSPARK_ERR_SHAPE;
    if (q_stride < 0 || k_stride < 0 || v_stride < 0) return DSPARK_ERR_ARG;
    if (misaligned(q, 2) || misaligned(k, 2) || misaligned(v, 2) || misaligned(q_out, 2) ||
        misaligned(cos, 4) || misaligned(sin, 4) || misaligned(cu_seqlens, 4) ||
        misaligned(ctx_lens, 4) || misaligned(block_table, 4) || misaligned(depths, 4))
        return DSPARK_ERR_ALIGN;
    AppendParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cos = cos;
    p.sin = sin;
    p.positions = positions;
    p.half = half;
    p.cu = cu_seqlens;
    p.ctx = ctx_lens;
    p.B = B;
    p.rows = rows;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    const bool e4m3 = cache_type == DSPARK_CACHE_E4M3;
    p.c = paged(k_cache, v_cache, pages, page_size, page_stride, head_stride, slot_stride, k_scale,
                v_scale, e4m3, block_table, table_width);
    p.out = q_out;
    p.depths = depths;
    return launched(launch_append_kv(p, interleaved != 0, e4m3, as_stream(stream)));
}

DSPARK_API dspark_status dspark_append_kv(
    const dspark_bf16 *q, const dspark_bf16 *k, const dspark_bf16 *v, long long q_stride,
    long long k_stride, long long v_stride, const float *cos, const float *sin, int positions,
    int half, int interleaved, const int32_t *cu_seqlens, const int32_t *ctx_lens, int B, int rows,
    int Hq, int Hkv, int D, void *k_cache, void *v_cache, int cache_type, int pages, int page_size,
    long long page_stride, long long head_stride, long long slot_stride, float k_scale,
    float v_scale, const int32_t *block_table, int table_width, dspark_bf16 *q_out, void *stream) {
    return append_rows(q, k, v, q_stride, k_stride, v_stride, cos, sin, positions, half,
                       interleaved, nullptr, cu_seqlens, ctx_lens, B, rows, Hq, Hkv, D, k_cache,
                       v_cache, cache_type, pages, page_size, page_stride, head_stride,
                       slot_stride, k_scale, v_scale, block_table, table_width, q_out, stream);
}

DSPARK_API dspark_status dspark_append_tree_kv(
    const dspark_bf16 *q, const dspark_bf16 *k, const dspark_bf16 *v, long long q_stride,
    long long k_stride, long long v_stride, const float *cos, const float *sin, int positions,
    int half, int interleaved, const int32_t *depths, const int32_t *cu_seqlens,
    const int32_t *ctx_lens, int B, int rows, int Hq, int Hkv, int D, void *k_cache,
    void *v_cache, int cache_type, int pages, int page_size, long long page_stride,
    long long head_stride, long long slot_stride, float k_scale, float v_scale,
    const int32_t *block_table, int table_width, dspark_bf16 *q_out, void *stream) {
    if (!depths) return DSPARK_ERR_NULL;
    return append_rows(q, k, v, q_stride, k_stride, v_stride, cos, sin, positions, half,
                       interleaved, depths, cu_seqlens, ctx_lens, B, rows, Hq, Hkv, D, k_cache,
                       v_cache, cache_type, pages, page_size, page_stride, head_stride,
                       slot_stride, k_scale, v_scale, block_table, table_width, q_out, stream);
}

DSPARK_API size_t dspark_attention_workspace_bytes(int B, int max_rows, int Hq, int Hkv, int D) {
    if (B < 1 || B > DSPARK_MAX_ROWS || max_rows < 1 || max_rows > DSPARK_MAX_ROWS || Hkv < 1 ||
        Hq < Hkv || Hq % Hkv != 0 || Hq > kMaxHeads || D < 8 || D > 256 || D % 8 != 0)
        return 0;
    return attention_ws_bytes(B, max_rows, Hq, Hkv, D);
}

// The checks and parameters that both attention entry points share.
static dspark_status attend_params(
    const dspark_bf16 *q, long long q_row, long long q_head, const void *k_cache,
    const void *v_cache, int cache_type, int pages, int page_size, long long page_stride,
    long long head_stride, long long slot_stride, float k_scale, float v_scale,
    const int32_t *block_table, int table_width, const int32_t *cu_seqlens,
    const int32_t *ctx_lens, int B, int rows, int max_rows, int Hq, int Hkv, int D, int window,
    float scale, dspark_bf16 *out, void *ws, size_t ws_bytes, AttendParams &p) {
    if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens || !ctx_lens || !out || !ws)
        return DSPARK_ERR_NULL;
    if (dspark_status st = check_paged(k_cache, v_cache, cache_type, pages, page_size, page_stride,
                                       head_stride, slot_stride, k_scale, v_scale, table_width, B,
                                       rows, Hq, Hkv, D, 256))
        return st;
    if (D % 8 != 0 || max_rows < 1) return DSPARK_ERR_SHAPE;
    if (q_row < 0 || q_head < 0 || window < 0 || !std::isfinite(scale)) return DSPARK_ERR_ARG;
    const bool e4m3 = cache_type == DSPARK_CACHE_E4M3;
    const size_t item = e4m3 ? 1 : 2;
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(ws, 16) || q_row % 8 != 0 ||
        q_head % 8 != 0 || misaligned(k_cache, 8 * item) || misaligned(v_cache, 8 * item) ||
        page_stride % 8 != 0 || head_stride % 8 != 0 || slot_stride % 8 != 0 ||
        misaligned(block_table, 4) || misaligned(cu_seqlens, 4) || misaligned(ctx_lens, 4))
        return DSPARK_ERR_ALIGN;
    // a request has at most `rows` rows
    max_rows = max_rows < rows ? max_rows : rows;
    if (ws_bytes < attention_ws_bytes(B, max_rows, Hq, Hkv, D)) return DSPARK_ERR_WORKSPACE;
    p.q = q;
    p.q_row = q_row;
    p.q_head = q_head;
    p.cu = cu_seqlens;
    p.ctx = ctx_lens;
    p.B = B;
    p.rows = rows;
    p.max_rows = max_rows;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.window = window;
    p.scale = scale;
    p.c = paged(k_cache, v_cache, pages, page_size, page_stride, head_stride, slot_stride, k_scale,
                v_scale, e4m3, block_table, table_width);
    p.out = out;
    return DSPARK_OK;
}

DSPARK_API dspark_status dspark_verify_attention(
    const dspark_bf16 *q, long long q_row, long long q_head, const void *k_cache,
    const void *v_cache, int cache_type, int pages, int page_size, long long page_stride,
    long long head_stride, long long slot_stride, float k_scale, float v_scale,
    const int32_t *block_table, int table_width, const int32_t *cu_seqlens,
    const int32_t *ctx_lens, int B, int rows, int max_rows, int Hq, int Hkv, int D, int window,
    float scale, dspark_bf16 *out, void *ws, size_t ws_bytes, void *stream) {
    AttendParams p;
    if (dspark_status st = attend_params(
            q, q_row, q_head, k_cache, v_cache, cache_type, pages, page_size, page_stride,
            head_stride, slot_stride, k_scale, v_scale, block_table, table_width, cu_seqlens,
            ctx_lens, B, rows, max_rows, Hq, Hkv, D, window, scale, out, ws, ws_bytes, p))
        return st;
    return launched(launch_attention(p, cache_type == DSPARK_CACHE_E4M3, ws, as_stream(stream)));
}

DSPARK_API dspark_status dspark_tree_attention(
    const dspark_bf16 *q, long long q_row, long long q_head, const void *k_cache,
    const void *v_cache, int cache_type, int pages, int page_size, long long page_stride,
    long long head_stride, long long slot_stride, float k_scale, float v_scale,
    const int32_t *block_table, int table_width, const int32_t *cu_seqlens,
    const int32_t *ctx_lens, int B, int rows, int max_rows, int Hq, int Hkv, int D, int window,
    int sinks, const int32_t *depths, const int32_t *masks, int mask_words, float scale,
    dspark_bf16 *out, void *ws, size_t ws_bytes, void *stream) {
    if (!depths != !masks) return DSPARK_ERR_NULL;
    AttendParams p;
    if (dspark_status st = attend_params(
            q, q_row, q_head, k_cache, v_cache, cache_type, pages, page_size, page_stride,
            head_stride, slot_stride, k_scale, v_scale, block_table, table_width, cu_seqlens,
            ctx_lens, B, rows, max_rows, Hq, Hkv, D, window, scale, out, ws, ws_bytes, p))
        return st;
    if (sinks < 0) return DSPARK_ERR_ARG;
    if (masks && (mask_words < 1 || mask_words > DSPARK_MAX_ROWS / 32 ||
                  (long long)mask_words * 32 < p.max_rows))
        return DSPARK_ERR_SHAPE;
    if (misaligned(depths, 4) || misaligned(masks, 4)) return DSPARK_ERR_ALIGN;
    TreeView v;
    v.depths = depths;
    v.masks = reinterpret_cast<const uint32_t *>(masks);
    v.words = masks ? mask_words : 0;
    v.sinks = window > 0 ? sinks : 0;
    return launched(launch_tree_attention(p, v, cache_type == DSPARK_CACHE_E4M3, ws,
                                          as_stream(stream)));
}

DSPARK_API dspark_status dspark_sample_accept(
    const dspark_bf16 *logits, const int32_t *packed_src_row, const int32_t *cu_seqlens,
    const int32_t *tokens, const float *uniforms, const float *temperature, const int32_t *top_k,
    const float *top_p, const float *min_p, int B, int gamma, int V, int32_t *packed_sample,
    int32_t *accepted, int32_t *bonus, void *ws, size_t ws_bytes, void *stream) {
    if (!logits || !cu_seqlens || !tokens || !uniforms || !packed_sample || !accepted || !bonus ||
        !ws)
        return DSPARK_ERR_NULL;
    if (dspark_status st = check_bg(B, gamma)) return st;
    if (V < 1) return DSPARK_ERR_SHAPE;
    if (misaligned(logits, 2) || misaligned(packed_src_row, 4) || misaligned(cu_seqlens, 4) ||
        misaligned(tokens, 4) || misaligned(uniforms, 4) || misaligned(temperature, 4) ||
        misaligned(top_k, 4) || misaligned(top_p, 4) || misaligned(min_p, 4) ||
        misaligned(packed_sample, 4) || misaligned(accepted, 4) || misaligned(bonus, 4) ||
        misaligned(ws, 16))
        return DSPARK_ERR_ALIGN;
    if (ws_bytes < ws_total_bytes(B, gamma)) return DSPARK_ERR_WORKSPACE;
    SampleParams p;
    p.logits = logits;
    p.psrc = packed_src_row;
    p.cu = cu_seqlens;
    p.tokens = tokens;
    p.uniforms = uniforms;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.B = B;
    p.gamma = gamma;
    p.V = V;
    p.sample = packed_sample;
    p.acc = accepted;
    p.bonus = bonus;
    return launched(launch_sample_accept(p, ws, as_stream(stream)));
}

namespace {

// Requests, rows and tree sizes that the calls on drafted trees share.
dspark_status check_tree(int B, int rows, int max_rows) {
    if (B < 1 || B > DSPARK_MAX_ROWS || rows < 1 || rows > DSPARK_MAX_ROWS) return DSPARK_ERR_SHAPE;
    if (max_rows < 1 || max_rows > DSPARK_MAX_TREE) return DSPARK_ERR_SHAPE;
    return DSPARK_OK;
}

// The pools of all layers, as moves of whole rows see them.
dspark_status page_moves(void *k_cache, void *v_cache, int cache_type, int layers,
                         long long layer_stride, int pages, int page_size, long long page_stride,
                         long long head_stride, long long slot_stride, int Hkv, int D,
                         PageMoveParams &p) {
    if (layers < 1 || layers > 32767 || pages < 1 || page_size < 1 || Hkv < 1 || Hkv > kMaxHeads ||
        D < 1 || D > 1024)
        return DSPARK_ERR_SHAPE;
    if (cache_type != DSPARK_CACHE_BF16 && cache_type != DSPARK_CACHE_E4M3) return DSPARK_ERR_ARG;
    if (layer_stride < 0 || page_stride < 0 || head_stride < 0 || slot_stride < 0)
        return DSPARK_ERR_ARG;
    const int item = cache_type == DSPARK_CACHE_E4M3 ? 1 : 2;
    if (misaligned(k_cache, item) || misaligned(v_cache, item)) return DSPARK_ERR_ALIGN;
    p.k = k_cache;
    p.v = v_cache;
    p.layers = layers;
    p.pages = pages;
    p.page = page_size;
    p.heads = Hkv;
    p.row_bytes = D * item;
    p.layer_stride = layer_stride * item;
    p.page_stride = page_stride * item;
    p.head_stride = head_stride * item;
    p.slot_stride = slot_stride * item;
    return DSPARK_OK;
}

dspark_status check_pool(const int32_t *table, const int32_t *held, const int32_t *lens, int R,
                         int width, int page_size, const int32_t *refs, int pages) {
    if (!table || !held || !lens || !refs) return DSPARK_ERR_NULL;
    if (R < 1 || R > DSPARK_MAX_TABLE_ROWS || width < 1 || page_size < 1 || pages < 1 ||
        pages > (1 << 30) || (long long)width * page_size > 0x7FFFFFFFll ||
        (long long)R * width > (1ll << 30))
        return DSPARK_ERR_SHAPE;
    if (misaligned(table, 4) || misaligned(held, 4) || misaligned(lens, 4) || misaligned(refs, 4))
        return DSPARK_ERR_ALIGN;
    return DSPARK_OK;
}

PoolParams pool_params(int32_t *table, int32_t *held, const int32_t *lens, int R, int width,
                       int page_size, int32_t *refs, int pages) {
    PoolParams p = {};
    p.table = table;
    p.held = held;
    p.lens = lens;
    p.R = R;
    p.width = width;
    p.page = page_size;
    p.refs = refs;
    p.pages = pages;
    return p;
}

}  // namespace

DSPARK_API dspark_status dspark_tree_masks(const int32_t *parents, const int32_t *cu_seqlens,
                                           const int32_t *ctx_lens, int B, int rows, int max_rows,
                                           int window, int sinks, int mask_words, int32_t *depths,
                                           int32_t *masks, void *stream) {
    if (!parents || !cu_seqlens || !depths || !masks) return DSPARK_ERR_NULL;
    if (dspark_status st = check_tree(B, rows, max_rows)) return st;
    max_rows = max_rows < rows ? max_rows : rows;
    if (mask_words < 1 || mask_words > DSPARK_MAX_TREE / 32 || mask_words * 32 < max_rows)
        return DSPARK_ERR_SHAPE;
    if (window < 0 || sinks < 0) return DSPARK_ERR_ARG;
    if (window > 0 && sinks > 0 && !ctx_lens) return DSPARK_ERR_NULL;
    if (misaligned(parents, 4) || misaligned(cu_seqlens, 4) || misaligned(ctx_lens, 4) ||
        misaligned(depths, 4) || misaligned(masks, 4))
        return DSPARK_ERR_ALIGN;
    TreeMaskParams p;
    p.parents = parents;
    p.cu = cu_seqlens;
    p.ctx = ctx_lens;
    p.B = B;
    p.rows = rows;
    p.max_rows = max_rows;
    p.words = mask_words;
    p.window = window;
    p.sinks = window > 0 ? sinks : 0;
    p.depths = depths;
    p.masks = reinterpret_cast<uint32_t *>(masks);
    return launched(launch_tree_masks(p, as_stream(stream)));
}

DSPARK_API dspark_status dspark_tree_accept(const int32_t *packed_choice,
                                            const int32_t *packed_tokens, const int32_t *parents,
                                            const int32_t *cu_seqlens, int B, int rows,
                                            int max_rows, int width, int32_t *accepted,
                                            int32_t *bonus, int32_t *path, void *stream) {
    if (!packed_choice || !packed_tokens || !parents || !cu_seqlens || !accepted || !bonus || !path)
        return DSPARK_ERR_NULL;
    if (dspark_status st = check_tree(B, rows, max_rows)) return st;
    if (width < 1 || width > DSPARK_MAX_TREE) return DSPARK_ERR_SHAPE;
    if (misaligned(packed_choice, 4) || misaligned(packed_tokens, 4) || misaligned(parents, 4) ||
        misaligned(cu_seqlens, 4) || misaligned(accepted, 4) || misaligned(bonus, 4) ||
        misaligned(path, 4))
        return DSPARK_ERR_ALIGN;
    TreeAcceptParams p;
    p.choice = packed_choice;
    p.tokens = packed_tokens;
    p.parents = parents;
    p.cu = cu_seqlens;
    p.B = B;
    p.rows = rows;
    p.max_rows = max_rows;
    p.width = width;
    p.accepted = accepted;
    p.bonus = bonus;
    p.path = path;
    return launched(launch_tree_accept(p, as_stream(stream)));
}

DSPARK_API dspark_status dspark_move_kv(void *k_cache, void *v_cache, int cache_type, int layers,
                                        long long layer_stride, int pages, int page_size,
                                        long long page_stride, long long head_stride,
                                        long long slot_stride, int Hkv, int D, const int32_t *path,
                                        const int32_t *accepted, int width,
                                        const int32_t *ctx_lens, const int32_t *block_table,
                                        int table_width, int B, void *stream) {
    if (!k_cache || !v_cache || !path || !accepted || !ctx_lens || !block_table)
        return DSPARK_ERR_NULL;
    if (B < 1 || B > DSPARK_MAX_ROWS || width < 1 || width > DSPARK_MAX_TREE || table_width < 1 ||
        page_size < 1 || (long long)table_width * page_size > 0x7FFFFFFFll)
        return DSPARK_ERR_SHAPE;
    PageMoveParams p = {};
    if (dspark_status st = page_moves(k_cache, v_cache, cache_type, layers, layer_stride, pages,
                                      page_size, page_stride, head_stride, slot_stride, Hkv, D, p))
        return st;
    if (misaligned(path, 4) || misaligned(accepted, 4) || misaligned(ctx_lens, 4) ||
        misaligned(block_table, 4))
        return DSPARK_ERR_ALIGN;
    p.c = paged(k_cache, v_cache, pages, page_size, p.page_stride, p.head_stride, p.slot_stride,
                1.f, 1.f, false, block_table, table_width);
    p.path = path;
    p.accepted = accepted;
    p.width = width;
    p.ctx = ctx_lens;
    p.n = B;
    return launched(launch_move_kv(p, as_stream(stream)));
}

DSPARK_API dspark_status dspark_copy_pages(void *k_cache, void *v_cache, int cache_type,
                                           int layers, long long layer_stride, int pages,
                                           int page_size, long long page_stride,
                                           long long head_stride, long long slot_stride, int Hkv,
                                           int D, const int32_t *src, const int32_t *dst,
                                           const int32_t *slots, int n, void *stream) {
    if (!k_cache || !v_cache || !src || !dst) return DSPARK_ERR_NULL;
    if (n < 1 || n > (1 << 20)) return DSPARK_ERR_SHAPE;
    PageMoveParams p = {};
    if (dspark_status st = page_moves(k_cache, v_cache, cache_type, layers, layer_stride, pages,
                                      page_size, page_stride, head_stride, slot_stride, Hkv, D, p))
        return st;
    if (misaligned(src, 4) || misaligned(dst, 4) || misaligned(slots, 4)) return DSPARK_ERR_ALIGN;
    p.src = src;
    p.dst = dst;
    p.slots = slots;
    p.n = n;
    return launched(launch_copy_pages(p, as_stream(stream)));
}

DSPARK_API dspark_status dspark_resize_pages(int32_t *table, int32_t *held, const int32_t *lens,
                                             int R, int width, int page_size, int32_t *refs,
                                             int pages, int32_t *granted, void *stream) {
    if (!granted) return DSPARK_ERR_NULL;
    if (dspark_status st = check_pool(table, held, lens, R, width, page_size, refs, pages))
        return st;
    if (misaligned(granted, 4)) return DSPARK_ERR_ALIGN;
    PoolParams p = pool_params(table, held, lens, R, width, page_size, refs, pages);
    p.granted = granted;
    return launched(launch_resize_pages(p, as_stream(stream)));
}

DSPARK_API dspark_status dspark_fork_pages(int32_t *table, int32_t *held, const int32_t *lens,
                                           int R, int width, int page_size, int32_t *refs,
                                           int pages, const int32_t *src, const int32_t *dst,
                                           int n, int32_t *copy_src, int32_t *copy_dst,
                                           int32_t *copy_slots, int32_t *granted, void *stream) {
    if (!src || !dst || !copy_src || !copy_dst || !copy_slots || !granted) return DSPARK_ERR_NULL;
    if (dspark_status st = check_pool(table, held, lens, R, width, page_size, refs, pages))
        return st;
    if (n < 1 || n > DSPARK_MAX_FORKS) return DSPARK_ERR_SHAPE;
    if (misaligned(src, 4) || misaligned(dst, 4) || misaligned(copy_src, 4) ||
        misaligned(copy_dst, 4) || misaligned(copy_slots, 4) || misaligned(granted, 4))
        return DSPARK_ERR_ALIGN;
    PoolParams p = pool_params(table, held, lens, R, width, page_size, refs, pages);
    p.src = src;
    p.dst = dst;
    p.n = n;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.copy_slots = copy_slots;
    p.granted = granted;
    return launched(launch_fork_pages(p, as_stream(stream)));
}
