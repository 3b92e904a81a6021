// C ABI of libgdn2 (declared in include/gdn2.h): argument validation, the
// per-thread stream, and dispatch to the kernels. Nothing is enqueued unless
// every check passes.
#include "../../include/gdn2.h"
#include "gdn2_launch.hpp"

#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <vector>

namespace {

thread_local hipStream_t g_stream = nullptr;

// Per-thread kernel timing state (gdn2_profile_*).
struct Prof {
    bool on = false;          // recording requested
    bool active = false;      // the current call is being recorded
    int max_calls = 0, calls = 0;
    std::vector<hipEvent_t> ev;
    size_t used = 0;
    struct Rec { const char *name; size_t e0; };
    std::vector<Rec> recs;
    void release() {
        for (hipEvent_t e : ev) (void)hipEventDestroy(e);
        ev.clear();
        recs.clear();
        used = 0;
        calls = 0;
        on = active = false;
    }
    // no destructor: events are left to the process teardown, whose order
    // relative to the HIP runtime's is not defined
};
thread_local Prof g_prof;

// Events created up front per recorded call; the pool grows past this on
// demand (a segmented prefill launches two kernels per segment), up to a cap.
constexpr size_t kEventsPerCall = 64;
constexpr size_t kMaxProfEvents = 1u << 17;

bool prof_grow(size_t n)
{
    while (g_prof.ev.size() < n) {
        hipEvent_t e = nullptr;
        if (g_prof.ev.size() >= kMaxProfEvents || hipEventCreate(&e) != hipSuccess) return false;
        g_prof.ev.push_back(e);
    }
    return true;
}

// Marks the start of a library call: decides whether its kernels are timed.
void prof_call()
{
    g_prof.active = g_prof.on && g_prof.calls < g_prof.max_calls;
    if (g_prof.active) ++g_prof.calls;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

bool head_dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

} // namespace

namespace gdn2 {

void prof_before(const char *kernel, hipStream_t st)
{
    if (!g_prof.active || !prof_grow(g_prof.used + 2)) return;
    (void)hipEventRecord(g_prof.ev[g_prof.used], st);
    g_prof.recs.push_back({kernel, g_prof.used});
    g_prof.used += 1;
}

void prof_after(hipStream_t st)
{
    if (!g_prof.active || g_prof.recs.empty() || g_prof.recs.back().e0 + 1 != g_prof.used) return;
    (void)hipEventRecord(g_prof.ev[g_prof.used], st);
    g_prof.used += 1;
}

} // namespace gdn2

extern "C" {

int gdn2_profile_begin(int max_calls)
{
    if (max_calls < 1 || max_calls > 4096) return GDN2_ERR_INVALID;
    g_prof.release();
    if (!prof_grow(std::min((size_t)max_calls * kEventsPerCall, kMaxProfEvents))) {
        g_prof.release();
        return GDN2_ERR_HIP;
    }
    g_prof.max_calls = max_calls;
    g_prof.on = true;
    return GDN2_OK;
}

int gdn2_profile_end(void)
{
    g_prof.on = g_prof.active = false;
    return g_prof.calls;
}

int gdn2_profile_kernel(int idx, const char **name, int *launches, double *total_ms)
{
    // distinct names in order of first launch
    std::vector<const char *> names;
    for (const auto &r : g_prof.recs) {
        bool seen = false;
        for (const char *n : names) seen = seen || strcmp(n, r.name) == 0;
        if (!seen) names.push_back(r.name);
    }
    if (idx < 0 || idx >= (int)names.size()) return GDN2_ERR_INVALID;
    int cnt = 0;
    double tot = 0.0;
    for (const auto &r : g_prof.recs) {
        if (strcmp(r.name, names[idx]) != 0 || r.e0 + 1 >= g_prof.used) continue;
        float ms = 0.f;
        if (hipEventSynchronize(g_prof.ev[r.e0 + 1]) != hipSuccess) return GDN2_ERR_HIP;
        if (hipEventElapsedTime(&ms, g_prof.ev[r.e0], g_prof.ev[r.e0 + 1]) != hipSuccess) return GDN2_ERR_HIP;
        ++cnt;
        tot += ms;
    }
    if (name) *name = names[idx];
    if (launches) *launches = cnt;
    if (total_ms) *total_ms = tot;
    return GDN2_OK;
}

int gdn2_set_stream(void *hip_stream)
{
    g_stream = (hipStream_t)hip_stream;
    return GDN2_OK;
}

void *gdn2_get_stream(void) { return (void *)g_stream; }

const char *gdn2_status_string(int status)
{
    switch (status) {
    case GDN2_OK: return "GDN2_OK";
    case GDN2_ERR_INVALID: return "GDN2_ERR_INVALID: invalid argument";
    case GDN2_ERR_UNSUPPORTED: return "GDN2_ERR_UNSUPPORTED: sizes or dtypes not supported";
    case GDN2_ERR_WORKSPACE: return "GDN2_ERR_WORKSPACE: workspace missing or too small";
    case GDN2_ERR_HIP: return "GDN2_ERR_HIP: HIP runtime error";
    }
    return "GDN2: unknown status";
}

static int chunk_fwd_impl(const void *q, const void *k, const void *v, const float *log_alpha,
                          const void *b, const void *w, int gates, const gdn2_short_conv *conv, const float *S0,
                          void *o, float *ST, const int32_t *cu_seqlens, int B, int T, int N, int H, int dk,
                          int dv, int in_dtype, int out_dtype, void *workspace,
                          size_t workspace_bytes, int chunk = 64);

static int chunk_check(int B, int T, int N, int H, int dk, int dv, int in_dtype, int varlen,
                       gdn2::ChunkPlan *plan, int chunk = 64)
{
    if (chunk != 32 && chunk != 64 && chunk != 128) return GDN2_ERR_INVALID;
    if (B <= 0 || T < 0 || N <= 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_INVALID;
    if (in_dtype != GDN2_F32 && in_dtype != GDN2_BF16) return GDN2_ERR_INVALID;
    if (varlen ? B != 1 : N != B) return GDN2_ERR_INVALID;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN2_ERR_UNSUPPORTED;
    if (H > 65535) return GDN2_ERR_UNSUPPORTED;   // grid y dimension
    if ((long long)B * T > 0x7fffffffLL) return GDN2_ERR_UNSUPPORTED;
    // (each factor is bounded above, so the product cannot overflow)
    if ((long long)B * T * H * (dk > dv ? dk : dv) > 0x7fffffffLL * 16LL) return GDN2_ERR_UNSUPPORTED;
    if (!gdn2::chunk_plan(B, T, N, H, dk, dv, in_dtype == GDN2_BF16, varlen != 0, plan, chunk))
        return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

size_t gdn2_chunk_fwd_sized_workspace_bytes(int B, int T, int N, int H, int dk, int dv, int in_dtype,
                                            int varlen, int chunk)
{
    gdn2::ChunkPlan plan;
    if (chunk_check(B, T, N, H, dk, dv, in_dtype, varlen, &plan, chunk) != GDN2_OK) return 0;
    return plan.total_bytes > 0 ? plan.total_bytes : 256;
}

size_t gdn2_chunk_fwd_workspace_bytes(int B, int T, int N, int H, int dk, int dv,
                                      int in_dtype, int varlen)
{
    gdn2::ChunkPlan plan;
    if (chunk_check(B, T, N, H, dk, dv, in_dtype, varlen, &plan) != GDN2_OK) return 0;
    return plan.total_bytes > 0 ? plan.total_bytes : 256;
}

int gdn2_chunk_fwd(const void *q, const void *k, const void *v, const float *log_alpha,
                   const void *b, const void *w, const float *S0, void *o, float *ST,
                   const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                   int in_dtype, int out_dtype, void *workspace,
                   size_t workspace_bytes)
{
    return gdn2_chunk_fwd_gates(q, k, v, log_alpha, b, w, GDN2_GATES_PER_CHANNEL, S0, o, ST, cu_seqlens, B, T,
                                N, H, dk, dv, in_dtype, out_dtype, workspace, workspace_bytes);
}

} // extern "C"

// Workspace of gdn2_chunk_fwd_noalloc, for callers that cannot allocate:
// one copy per device, held until the process ends, shared by every call on
// that device (calls that overlap on one device race on it).
static constexpr size_t kScratchBytes = (size_t)GDN2_NOALLOC_WORKSPACE_MAX;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

// Device address of `scratch` on the current device, looked up with that
// device current on its first use and kept per device. (In host code the
// array's name stands for a host-side shadow, not for device memory.)
static int scratch_address(void **out)
{
    constexpr int kMaxDev = 64;
    static std::atomic<void *> addr[kMaxDev];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDev) return GDN2_ERR_HIP;
    void *p = addr[dev].load(std::memory_order_acquire);
    if (!p) {
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return GDN2_ERR_HIP;
        addr[dev].store(p, std::memory_order_release);
    }
    *out = p;
    return GDN2_OK;
}

extern "C" {

int gdn2_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const float *log_alpha,
                           const void *b, const void *w, const float *S0, void *o, float *ST,
                           const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                           int in_dtype, int out_dtype)
{
    const size_t need = gdn2_chunk_fwd_workspace_bytes(B, T, N, H, dk, dv, in_dtype, cu_seqlens != nullptr);
    if (need == 0 || need > kScratchBytes) {
        // invalid sizes report their own status; valid ones over the limit
        // report the workspace (nothing is launched either way)
        const int st = chunk_fwd_impl(q, k, v, log_alpha, b, w, GDN2_GATES_PER_CHANNEL, nullptr, S0, o, ST,
                                      cu_seqlens, B, T, N, H, dk, dv, in_dtype, out_dtype, nullptr, 0);
        return st == GDN2_OK ? GDN2_ERR_WORKSPACE : st;
    }
    void *ws = nullptr;
    const int st = scratch_address(&ws);
    if (st != GDN2_OK) return st;
    return chunk_fwd_impl(q, k, v, log_alpha, b, w, GDN2_GATES_PER_CHANNEL, nullptr, S0, o, ST, cu_seqlens, B, T,
                          N, H, dk, dv, in_dtype, out_dtype, ws, kScratchBytes);
}

// The convolution parameters of a *_prologue call: weights required, biases
// optional, history in / out each all-or-none.
static int conv_args(const gdn2_short_conv *c, gdn2::Prologue *p)
{
    if (!c) return GDN2_ERR_INVALID;
    const void *req[] = {c->weight_q, c->weight_k, c->weight_v};
    for (const void *x : req)
        if (!x || !aligned16(x)) return GDN2_ERR_INVALID;
    const void *opt[] = {c->bias_q, c->bias_k, c->bias_v, c->state_in_q, c->state_in_k, c->state_in_v,
                         c->state_out_q, c->state_out_k, c->state_out_v};
    for (const void *x : opt)
        if (x && !aligned16(x)) return GDN2_ERR_INVALID;
    const int nin = !!c->state_in_q + !!c->state_in_k + !!c->state_in_v;
    const int nout = !!c->state_out_q + !!c->state_out_k + !!c->state_out_v;
    if ((nin != 0 && nin != 3) || (nout != 0 && nout != 3)) return GDN2_ERR_INVALID;
    p->on = true;
    p->q = {c->weight_q, c->bias_q, c->state_in_q, c->state_out_q};
    p->k = {c->weight_k, c->bias_k, c->state_in_k, c->state_out_k};
    p->v = {c->weight_v, c->bias_v, c->state_in_v, c->state_out_v};
    return GDN2_OK;
}

static int chunk_fwd_impl(const void *q, const void *k, const void *v, const float *log_alpha,
                          const void *b, const void *w, int gates, const gdn2_short_conv *conv, const float *S0,
                          void *o, float *ST, const int32_t *cu_seqlens, int B, int T, int N, int H, int dk,
                          int dv, int in_dtype, int out_dtype, void *workspace,
                          size_t workspace_bytes, int chunk)
{
    if (gates & ~(GDN2_GATE_B_PER_HEAD | GDN2_GATE_W_PER_HEAD | GDN2_GATE_ALPHA_PER_HEAD)) return GDN2_ERR_INVALID;
    gdn2::ChunkPlan plan;
    const int varlen = cu_seqlens != nullptr;
    int st = chunk_check(B, T, N, H, dk, dv, in_dtype, varlen, &plan, chunk);
    if (st != GDN2_OK) return st;
    if (out_dtype != GDN2_F32) return out_dtype == GDN2_BF16 ? GDN2_ERR_UNSUPPORTED : GDN2_ERR_INVALID;
    const bool have_tokens = (long long)B * T > 0;
    if (have_tokens && (!q || !k || !v || !log_alpha || !b || !w || !o)) return GDN2_ERR_INVALID;
    const void *ptrs[] = {q, k, v, log_alpha, b, w, S0, o, ST, cu_seqlens, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    gdn2::ChunkArgs a;
    if (conv && (st = conv_args(conv, &a.pro)) != GDN2_OK) return st;
    if (!workspace || workspace_bytes < plan.total_bytes) return GDN2_ERR_WORKSPACE;

    a.q = q; a.k = k; a.v = v; a.b = b; a.w = w;
    a.log_alpha = log_alpha;
    a.S0 = S0;
    a.o = o;
    a.ST = ST;
    a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.N = N; a.H = H; a.dk = dk; a.dv = dv;
    a.gates = gates;
    a.bf16 = in_dtype == GDN2_BF16;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    prof_call();
    if (gdn2::launch_chunk_fwd(a, plan, g_stream) != hipSuccess) return GDN2_ERR_HIP;
    return GDN2_OK;
}

int gdn2_chunk_fwd_gates(const void *q, const void *k, const void *v, const float *log_alpha,
                         const void *b, const void *w, int gates, const float *S0, void *o, float *ST,
                         const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                         int in_dtype, int out_dtype, void *workspace,
                         size_t workspace_bytes)
{
    return chunk_fwd_impl(q, k, v, log_alpha, b, w, gates, nullptr, S0, o, ST, cu_seqlens, B, T, N, H, dk, dv,
                          in_dtype, out_dtype, workspace, workspace_bytes);
}

int gdn2_chunk_fwd_sized(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                         const void *w, const float *S0, void *o, float *ST, const int32_t *cu_seqlens, int B,
                         int T, int N, int H, int dk, int dv, int in_dtype, int out_dtype,
                         int chunk, void *workspace, size_t workspace_bytes)
{
    return chunk_fwd_impl(q, k, v, log_alpha, b, w, GDN2_GATES_PER_CHANNEL, nullptr, S0, o, ST, cu_seqlens, B, T,
                          N, H, dk, dv, in_dtype, out_dtype, workspace, workspace_bytes, chunk);
}

int gdn2_chunk_fwd_prologue(const void *q_raw, const void *k_raw, const void *v_raw, const float *log_alpha,
                            const void *b_logit, const void *w_logit, const gdn2_short_conv *conv,
                            const float *S0, void *o, float *ST, const int32_t *cu_seqlens, int B, int T,
                            int N, int H, int dk, int dv, int in_dtype, int out_dtype,
                            void *workspace, size_t workspace_bytes)
{
    if (!conv) return GDN2_ERR_INVALID;
    return chunk_fwd_impl(q_raw, k_raw, v_raw, log_alpha, b_logit, w_logit, GDN2_GATES_PER_CHANNEL, conv, S0, o,
                          ST, cu_seqlens, B, T, N, H, dk, dv, in_dtype, out_dtype, workspace, workspace_bytes);
}

int gdn2_decode_step(const void *q, const void *k, const void *v, const float *log_alpha,
                     const void *b, const void *w, float *S, void *o, int N, int H, int dk,
                     int dv, int in_dtype, int out_dtype)
{
    return gdn2_decode_step_gates(q, k, v, log_alpha, b, w, GDN2_GATES_PER_CHANNEL, S, o, N, H, dk, dv, in_dtype,
                                  out_dtype);
}

size_t gdn2_chunk_bwd_workspace_bytes(int B, int T, int N, int H, int dk, int dv,
                                      int in_dtype, int varlen)
{
    gdn2::ChunkPlan plan;
    if (chunk_check(B, T, N, H, dk, dv, in_dtype, varlen, &plan) != GDN2_OK) return 0;
    gdn2::BwdPlan bp;
    if (!gdn2::chunk_bwd_plan(B, T, N, H, dk, dv, in_dtype == GDN2_BF16, varlen != 0, &bp)) return 0;
    return bp.total_bytes > 0 ? bp.total_bytes : 256;
}

// gdn2_chunk_bwd and its two halves (part: gdn2::kBwdAll, kBwdForward,
// kBwdFromKept); every check runs before anything is launched
static int chunk_bwd_impl(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                          const void *w, const float *S0, const float *dO, const float *dST,
                          const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv, int in_dtype,
                          float *dq, float *dk_, float *dv_, float *dlog_alpha, float *db, float *dw, float *dS0,
                          void *o, float *ST, int part, void *workspace, size_t workspace_bytes)
{
    gdn2::ChunkPlan plan;
    const int varlen = cu_seqlens != nullptr;
    int st = chunk_check(B, T, N, H, dk, dv, in_dtype, varlen, &plan);
    if (st != GDN2_OK) return st;
    gdn2::BwdPlan bp;
    if (!gdn2::chunk_bwd_plan(B, T, N, H, dk, dv, in_dtype == GDN2_BF16, varlen != 0, &bp))
        return GDN2_ERR_UNSUPPORTED;
    const bool have_tokens = (long long)B * T > 0;
    if (have_tokens && (!q || !k || !v || !log_alpha || !b || !w)) return GDN2_ERR_INVALID;
    if (part == gdn2::kBwdForward && have_tokens && !o) return GDN2_ERR_INVALID;
    if (part != gdn2::kBwdForward && have_tokens && (!dO || !dq || !dk_ || !dv_ || !dlog_alpha || !db || !dw))
        return GDN2_ERR_INVALID;
    const void *ptrs[] = {q, k, v, log_alpha, b, w, S0, dO, dST, cu_seqlens, dq, dk_, dv_, dlog_alpha, db, dw, dS0,
                          o, ST, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (!workspace || workspace_bytes < bp.total_bytes) return GDN2_ERR_WORKSPACE;
    gdn2::ChunkBwdArgs a;
    a.q = q; a.k = k; a.v = v; a.b = b; a.w = w;
    a.log_alpha = log_alpha;
    a.S0 = S0;
    a.dO = dO;
    a.dST = dST;
    a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.N = N; a.H = H; a.dk = dk; a.dv = dv;
    a.bf16 = in_dtype == GDN2_BF16;
    a.dq = dq; a.dk_ = dk_; a.dv_ = dv_; a.dlog_alpha = dlog_alpha; a.db = db; a.dw = dw;
    a.dS0 = dS0;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    a.part = part;
    a.o = o;
    a.ST = ST;
    prof_call();
    if (gdn2::launch_chunk_bwd(a, bp, g_stream) != hipSuccess) return GDN2_ERR_HIP;
    return GDN2_OK;
}

int gdn2_chunk_bwd(const void *q, const void *k, const void *v, const float *log_alpha,
                   const void *b, const void *w, const float *S0, const float *dO, const float *dST,
                   const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                   int in_dtype, float *dq, float *dk_, float *dv_, float *dlog_alpha,
                   float *db, float *dw, float *dS0, void *workspace, size_t workspace_bytes)
{
    return chunk_bwd_impl(q, k, v, log_alpha, b, w, S0, dO, dST, cu_seqlens, B, T, N, H, dk, dv, in_dtype, dq, dk_,
                          dv_, dlog_alpha, db, dw, dS0, nullptr, nullptr, gdn2::kBwdAll, workspace, workspace_bytes);
}

int gdn2_chunk_fwd_keep(const void *q, const void *k, const void *v, const float *log_alpha,
                        const void *b, const void *w, const float *S0, void *o, float *ST,
                        const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                        int in_dtype, int out_dtype, void *workspace, size_t workspace_bytes)
{
    if (out_dtype != GDN2_F32) return out_dtype == GDN2_BF16 ? GDN2_ERR_UNSUPPORTED : GDN2_ERR_INVALID;
    return chunk_bwd_impl(q, k, v, log_alpha, b, w, S0, nullptr, nullptr, cu_seqlens, B, T, N, H, dk, dv, in_dtype,
                          nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, o, ST, gdn2::kBwdForward,
                          workspace, workspace_bytes);
}

int gdn2_chunk_bwd_kept(const void *q, const void *k, const void *v, const float *log_alpha,
                        const void *b, const void *w, const float *S0, const float *dO, const float *dST,
                        const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                        int in_dtype, float *dq, float *dk_, float *dv_, float *dlog_alpha,
                        float *db, float *dw, float *dS0, void *workspace, size_t workspace_bytes)
{
    return chunk_bwd_impl(q, k, v, log_alpha, b, w, S0, dO, dST, cu_seqlens, B, T, N, H, dk, dv, in_dtype, dq, dk_,
                          dv_, dlog_alpha, db, dw, dS0, nullptr, nullptr, gdn2::kBwdFromKept, workspace,
                          workspace_bytes);
}

static int decode_impl(const void *q, const void *k, const void *v, const float *log_alpha,
                       const void *b, const void *w, int gates, const gdn2_short_conv *conv, float *S, void *o,
                       int N, int H, int dk, int dv, int in_dtype, int out_dtype)
{
    if (gates & ~(GDN2_GATE_B_PER_HEAD | GDN2_GATE_W_PER_HEAD | GDN2_GATE_ALPHA_PER_HEAD)) return GDN2_ERR_INVALID;
    if (N <= 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_INVALID;
    if (in_dtype != GDN2_F32 && in_dtype != GDN2_BF16) return GDN2_ERR_INVALID;
    if (out_dtype != GDN2_F32) return out_dtype == GDN2_BF16 ? GDN2_ERR_UNSUPPORTED : GDN2_ERR_INVALID;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN2_ERR_UNSUPPORTED;
    if ((long long)N * H > 0x7fffffffLL) return GDN2_ERR_UNSUPPORTED;
    const void *ptrs[] = {q, k, v, log_alpha, b, w, S, o};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return GDN2_ERR_INVALID;
    gdn2::DecodeArgs a;
    int st;
    if (conv && (st = conv_args(conv, &a.pro)) != GDN2_OK) return st;
    a.q = q; a.k = k; a.v = v; a.b = b; a.w = w;
    a.log_alpha = log_alpha;
    a.S = S;
    a.o = o;
    a.N = N; a.H = H; a.dk = dk; a.dv = dv;
    a.gates = gates;
    a.bf16 = in_dtype == GDN2_BF16;
    prof_call();
    if (gdn2::launch_decode(a, g_stream) != hipSuccess) return GDN2_ERR_HIP;
    return GDN2_OK;
}

int gdn2_decode_step_gates(const void *q, const void *k, const void *v, const float *log_alpha,
                           const void *b, const void *w, int gates, float *S, void *o, int N, int H, int dk,
                           int dv, int in_dtype, int out_dtype)
{
    return decode_impl(q, k, v, log_alpha, b, w, gates, nullptr, S, o, N, H, dk, dv, in_dtype, out_dtype);
}

int gdn2_decode_step_prologue(const void *q_raw, const void *k_raw, const void *v_raw, const float *log_alpha,
                              const void *b_logit, const void *w_logit, const gdn2_short_conv *conv, float *S,
                              void *o, int N, int H, int dk, int dv, int in_dtype, int out_dtype)
{
    if (!conv) return GDN2_ERR_INVALID;
    return decode_impl(q_raw, k_raw, v_raw, log_alpha, b_logit, w_logit, GDN2_GATES_PER_CHANNEL, conv, S, o, N, H,
                       dk, dv, in_dtype, out_dtype);
}

// ---- operators around the mixer ------------------------------------------------

static bool dtype_ok(int t) { return t == GDN2_F32 || t == GDN2_BF16; }

// Whether an output is an input's own memory (partial overlaps are the caller's).
using Ptrs = std::initializer_list<const void *>;
static bool same_memory(Ptrs outs, Ptrs ins)
{
    for (const void *o : outs)
        for (const void *i : ins)
            if (o && o == i) return true;
    return false;
}

// Whether two outputs are one.
static bool twice(Ptrs outs)
{
    for (auto o = outs.begin(); o != outs.end(); ++o)
        for (auto p = outs.begin(); p != o; ++p)
            if (*o && *o == *p) return true;
    return false;
}

// Sizes whose launch would have too many threads are found where it is laid out.
static int launch_status(hipError_t err)
{
    return err == hipSuccess ? GDN2_OK : err == hipErrorInvalidConfiguration ? GDN2_ERR_UNSUPPORTED : GDN2_ERR_HIP;
}

// Sizes shared by the recurrence on slots and the prologue.
static int serve_check(int B, int T, int N, int H, int HK, int dk, int dv, int in_dtype, int varlen)
{
    if (B <= 0 || T < 0 || N <= 0 || H <= 0 || HK <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_INVALID;
    if (!dtype_ok(in_dtype) || H % HK != 0) return GDN2_ERR_INVALID;
    if (varlen ? B != 1 : N != B) return GDN2_ERR_INVALID;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return GDN2_ERR_UNSUPPORTED;
    if (H > 65535) return GDN2_ERR_UNSUPPORTED;
    const long long rows = (long long)B * T > N ? (long long)B * T : N;
    if (rows > 0x7fffffffLL) return GDN2_ERR_UNSUPPORTED;
    // (each factor is bounded above, so the product cannot overflow)
    if (rows * H * (dk > dv ? dk : dv) > 0x7fffffffLL * 16LL) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

int gdn2_recurrent_fwd(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                       const void *w, int gates, float *state, const int32_t *slot_in, const int32_t *slot_out,
                       const int32_t *commit, void *o, const int32_t *cu_seqlens, int B, int T, int N, int H, int HK,
                       int slots, int dk, int dv, int in_dtype, int out_dtype)
{
    if (gates & ~(GDN2_GATE_B_PER_HEAD | GDN2_GATE_W_PER_HEAD | GDN2_GATE_ALPHA_PER_HEAD)) return GDN2_ERR_INVALID;
    const int st = serve_check(B, T, N, H, HK, dk, dv, in_dtype, cu_seqlens != nullptr);
    if (st != GDN2_OK) return st;
    if (!dtype_ok(out_dtype) || slots < 1 || (!slot_in && slots < N)) return GDN2_ERR_INVALID;
    // (a wave has 16 columns of a chain, and a launch fewer than 2^32 threads)
    if ((long long)N * H * (dv / 16) * 64 > 0xffffffffLL) return GDN2_ERR_UNSUPPORTED;
    const bool have_tokens = (long long)B * T > 0;
    if (!state || (have_tokens && (!q || !k || !v || !log_alpha || !b || !w || !o))) return GDN2_ERR_INVALID;
    const void *ptrs[] = {q, k, v, log_alpha, b, w, state, slot_in, slot_out, commit, o, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (!have_tokens) o = nullptr;   // (nothing is written there)
    if (o == state || same_memory({o, state}, {q, k, v, log_alpha, b, w, slot_in, slot_out, commit, cu_seqlens}))
        return GDN2_ERR_INVALID;
    gdn2::RecurrentArgs a;
    a.q = q; a.k = k; a.v = v; a.b = b; a.w = w;
    a.log_alpha = log_alpha;
    a.state = state;
    a.slot_in = slot_in;
    a.slot_out = slot_out;
    a.commit = commit;
    a.o = o;
    a.cu_seqlens = cu_seqlens;
    a.T = T; a.N = N; a.H = H; a.HK = HK; a.slots = slots; a.dk = dk; a.dv = dv;
    a.gates = gates;
    a.bf16 = in_dtype == GDN2_BF16;
    a.out_bf16 = out_dtype == GDN2_BF16;
    prof_call();
    return gdn2::launch_recurrent(a, g_stream) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

// What gdn2_prologue_fwd and gdn2_prologue_bwd have in common.
static int prologue_args(const void *q_raw, const void *k_raw, const void *v_raw, const void *b_logit,
                         const void *w_logit, int gates, const gdn2_short_conv *conv, const int32_t *slot_in,
                         const int32_t *cu_seqlens, int B, int T, int N, int H, int HK, int slots, int dk, int dv,
                         int in_dtype, gdn2::PrologueArgs *a)
{
    if (gates & ~(GDN2_GATE_B_PER_HEAD | GDN2_GATE_W_PER_HEAD)) return GDN2_ERR_INVALID;
    int st = serve_check(B, T, N, H, HK, dk, dv, in_dtype, cu_seqlens != nullptr);
    if (st != GDN2_OK) return st;
    gdn2::Prologue pro;
    if ((st = conv_args(conv, &pro)) != GDN2_OK) return st;
    if ((pro.q.hist_in || pro.q.hist_out) && (slots < 1 || (!slot_in && slots < N))) return GDN2_ERR_INVALID;
    const bool have_tokens = (long long)B * T > 0;
    if (have_tokens && (!q_raw || !k_raw || !v_raw || !b_logit || !w_logit)) return GDN2_ERR_INVALID;
    const void *ptrs[] = {q_raw, k_raw, v_raw, b_logit, w_logit, slot_in, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    const void *xs[3] = {q_raw, k_raw, v_raw};
    const gdn2::ConvTensor *ct[3] = {&pro.q, &pro.k, &pro.v};
    for (int z = 0; z < 3; ++z) {
        a->x[z] = xs[z];
        a->weight[z] = ct[z]->w;
        a->bias[z] = ct[z]->bias;
        a->hist_in[z] = ct[z]->hist_in;
        a->hist_out[z] = ct[z]->hist_out;
        a->heads[z] = z < 2 ? HK : H;
        a->d[z] = z < 2 ? dk : dv;
    }
    a->logit[0] = b_logit;
    a->logit[1] = w_logit;
    a->nlogit[0] = H * (gates & GDN2_GATE_B_PER_HEAD ? 1 : dk);
    a->nlogit[1] = H * (gates & GDN2_GATE_W_PER_HEAD ? 1 : dv);
    a->slot_in = slot_in;
    a->cu_seqlens = cu_seqlens;
    a->T = T;
    a->N = N;
    a->slots = slots;
    a->bf16 = in_dtype == GDN2_BF16;
    return GDN2_OK;
}

int gdn2_prologue_fwd(const void *q_raw, const void *k_raw, const void *v_raw, const void *b_logit,
                      const void *w_logit, int gates, const gdn2_short_conv *conv, const int32_t *slot_in,
                      const int32_t *slot_out, const int32_t *commit, void *q, void *k, void *v, void *b, void *w,
                      const int32_t *cu_seqlens, int B, int T, int N, int H, int HK, int slots, int dk, int dv,
                      int in_dtype)
{
    gdn2::PrologueArgs a = {};
    const int st = prologue_args(q_raw, k_raw, v_raw, b_logit, w_logit, gates, conv, slot_in, cu_seqlens, B, T, N, H, HK,
                                 slots, dk, dv, in_dtype, &a);
    if (st != GDN2_OK) return st;
    if ((long long)B * T > 0 && (!q || !k || !v || !b || !w)) return GDN2_ERR_INVALID;
    const void *ptrs[] = {q, k, v, b, w, slot_out, commit};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if ((long long)B * T == 0) q = k = v = b = w = nullptr;   // (nothing is written there)
    // gates may take their own logits' place, histories their own pool's
    const Ptrs outs = {q, k, v, b, w, a.hist_out[0], a.hist_out[1], a.hist_out[2]};
    if (twice(outs) ||
        same_memory(outs, {q_raw, k_raw, v_raw, a.weight[0], a.weight[1], a.weight[2], a.bias[0], a.bias[1], a.bias[2],
                           slot_in, slot_out, commit, cu_seqlens}) ||
        same_memory({q, k, v, b, w}, {a.hist_in[0], a.hist_in[1], a.hist_in[2]}) ||
        same_memory({a.hist_out[0], a.hist_out[1], a.hist_out[2]}, {b_logit, w_logit}) ||
        same_memory({q, k, v}, {b_logit, w_logit}) || same_memory({b}, {w_logit}) || same_memory({w}, {b_logit}) ||
        same_memory({a.hist_out[0]}, {a.hist_in[1], a.hist_in[2]}) ||
        same_memory({a.hist_out[1]}, {a.hist_in[0], a.hist_in[2]}) ||
        same_memory({a.hist_out[2]}, {a.hist_in[0], a.hist_in[1]}))
        return GDN2_ERR_INVALID;
    a.y[0] = q; a.y[1] = k; a.y[2] = v;
    a.gate[0] = b; a.gate[1] = w;
    a.slot_out = slot_out;
    a.commit = commit;
    prof_call();
    return launch_status(gdn2::launch_prologue_fwd(a, g_stream));
}

size_t gdn2_prologue_bwd_workspace_bytes(int B, int T, int N, int H, int HK, int dk, int dv, int varlen)
{
    if (serve_check(B, T, N, H, HK, dk, dv, GDN2_F32, varlen) != GDN2_OK) return 0;
    const size_t need = gdn2::prologue_bwd_workspace((long long)B * T, 2LL * HK * dk + (long long)H * dv);
    return need > 0 ? need : 256;
}

int gdn2_prologue_bwd(const void *q_raw, const void *k_raw, const void *v_raw, const void *b_logit,
                      const void *w_logit, int gates, const gdn2_short_conv *conv, const int32_t *slot_in,
                      const float *dq, const float *dk_, const float *dv_, const float *db, const float *dw,
                      void *dq_raw, void *dk_raw, void *dv_raw, void *db_logit, void *dw_logit, float *dweight_q,
                      float *dweight_k, float *dweight_v, float *dbias_q, float *dbias_k, float *dbias_v,
                      const int32_t *cu_seqlens, int B, int T, int N, int H, int HK, int slots, int dk, int dv,
                      int in_dtype, int grad_dtype, void *workspace, size_t workspace_bytes)
{
    gdn2::PrologueBwdArgs a = {};
    const int st = prologue_args(q_raw, k_raw, v_raw, b_logit, w_logit, gates, conv, slot_in, cu_seqlens, B, T, N, H, HK,
                                 slots, dk, dv, in_dtype, &a.f);
    if (st != GDN2_OK) return st;
    if (!dtype_ok(grad_dtype) || !dweight_q || !dweight_k || !dweight_v) return GDN2_ERR_INVALID;
    if ((long long)B * T > 0 &&
        (!dq || !dk_ || !dv_ || !db || !dw || !dq_raw || !dk_raw || !dv_raw || !db_logit || !dw_logit))
        return GDN2_ERR_INVALID;
    const void *ptrs[] = {dq, dk_, dv_, db, dw, dq_raw, dk_raw, dv_raw, db_logit, dw_logit, dweight_q, dweight_k,
                          dweight_v, dbias_q, dbias_k, dbias_v, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (!workspace || workspace_bytes < gdn2_prologue_bwd_workspace_bytes(B, T, N, H, HK, dk, dv, cu_seqlens != nullptr))
        return GDN2_ERR_WORKSPACE;
    if ((long long)B * T == 0) dq_raw = dk_raw = dv_raw = db_logit = dw_logit = nullptr;   // (nothing is written there)
    const Ptrs outs = {dq_raw, dk_raw, dv_raw, db_logit, dw_logit, dweight_q, dweight_k, dweight_v,
                       dbias_q, dbias_k, dbias_v, workspace};
    if (twice(outs) ||
        same_memory(outs, {q_raw, k_raw, v_raw, b_logit, w_logit, dq, dk_, dv_, db, dw, a.f.weight[0], a.f.weight[1],
                           a.f.weight[2], a.f.bias[0], a.f.bias[1], a.f.bias[2], a.f.hist_in[0], a.f.hist_in[1],
                           a.f.hist_in[2], slot_in, cu_seqlens}))
        return GDN2_ERR_INVALID;
    a.dy[0] = dq; a.dy[1] = dk_; a.dy[2] = dv_;
    a.dgate[0] = db; a.dgate[1] = dw;
    a.dx[0] = dq_raw; a.dx[1] = dk_raw; a.dx[2] = dv_raw;
    a.dlogit[0] = db_logit; a.dlogit[1] = dw_logit;
    a.out_bf16 = grad_dtype == GDN2_BF16;
    a.dweight[0] = dweight_q; a.dweight[1] = dweight_k; a.dweight[2] = dweight_v;
    a.dbias[0] = dbias_q; a.dbias[1] = dbias_k; a.dbias[2] = dbias_v;
    a.workspace = workspace;
    prof_call();
    return launch_status(gdn2::launch_prologue_bwd(a, g_stream));
}

static int layer_norm_check(int64_t rows, int cols, float eps, int in_dtype, int out_dtype)
{
    if (rows < 0 || cols < 1 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return GDN2_ERR_INVALID;
    if (!(eps > 0.f && eps <= 3.4e38f)) return GDN2_ERR_INVALID;
    if (cols > GDN2_LAYER_NORM_MAX_COLS || rows > (int64_t)1 << 40) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

int gdn2_layer_norm_fwd(const void *x, const void *residual, const float *weight, const float *bias, void *y, void *sum,
                        int64_t rows, int cols, float eps, int in_dtype, int out_dtype)
{
    const int st = layer_norm_check(rows, cols, eps, in_dtype, out_dtype);
    if (st != GDN2_OK) return st;
    if (rows > 0 && (!x || !weight || !y || y == sum)) return GDN2_ERR_INVALID;
    const void *ptrs[] = {x, residual, weight, bias, y, sum};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    // (in place only where the elements have one size; weights are never outputs)
    if (in_dtype != out_dtype && same_memory({y}, {x, residual})) return GDN2_ERR_INVALID;
    if (same_memory({y, sum}, {weight, bias})) return GDN2_ERR_INVALID;
    gdn2::LayerNormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.sum = sum;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.in_bf16 = in_dtype == GDN2_BF16;
    a.out_bf16 = out_dtype == GDN2_BF16;
    prof_call();
    return gdn2::launch_layer_norm_fwd(a, g_stream) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

size_t gdn2_layer_norm_bwd_workspace_bytes(int64_t rows, int cols)
{
    if (layer_norm_check(rows, cols, 1.f, GDN2_F32, GDN2_F32) != GDN2_OK) return 0;
    const size_t need = (size_t)gdn2::ln_bwd_parts(rows, cols) * 2 * cols * sizeof(float);
    return need > 0 ? need : 256;
}

int gdn2_layer_norm_bwd(const void *dy, const void *h, const float *weight, const void *dsum, void *dh, float *dweight,
                        float *dbias, int64_t rows, int cols, float eps, int in_dtype, int out_dtype, void *workspace,
                        size_t workspace_bytes)
{
    const int st = layer_norm_check(rows, cols, eps, in_dtype, out_dtype);
    if (st != GDN2_OK) return st;
    if (!dweight || (rows > 0 && (!dy || !h || !weight || !dh))) return GDN2_ERR_INVALID;
    const void *ptrs[] = {dy, h, weight, dsum, dh, dweight, dbias, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (!workspace || workspace_bytes < gdn2_layer_norm_bwd_workspace_bytes(rows, cols)) return GDN2_ERR_WORKSPACE;
    if (in_dtype != out_dtype && same_memory({dh}, {dy})) return GDN2_ERR_INVALID;
    if (rows == 0) dh = nullptr;   // (nothing is written there)
    if (twice({dh, dweight, dbias, workspace}) || same_memory({dh, dweight, dbias, workspace}, {weight}) ||
        same_memory({dweight, dbias, workspace}, {dy, h, dsum}))
        return GDN2_ERR_INVALID;
    gdn2::LayerNormBwdArgs a;
    a.dy = dy;
    a.h = h;
    a.weight = weight;
    a.dsum = dsum;
    a.dh = dh;
    a.dweight = dweight;
    a.dbias = dbias;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.in_bf16 = in_dtype == GDN2_BF16;
    a.out_bf16 = out_dtype == GDN2_BF16;
    a.workspace = workspace;
    prof_call();
    return gdn2::launch_layer_norm_bwd(a, g_stream) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

} // extern "C"
