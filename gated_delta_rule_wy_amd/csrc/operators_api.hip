// C ABI of the operators around the mixer (declared in include/gdn2.h): argument
// validation and dispatch to the kernels. Nothing is enqueued unless every check
// passes.
#include "operators_checks.hpp"
#include "operators_launch.hpp"

using namespace gdn2;

extern "C" {

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
    return gdn2::launch_recurrent(a, stream()) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
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
    return launch_status(gdn2::launch_prologue_fwd(a, stream()));
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
    return launch_status(gdn2::launch_prologue_bwd(a, stream()));
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
    return gdn2::launch_layer_norm_fwd(a, stream()) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
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
    return gdn2::launch_layer_norm_bwd(a, stream()) == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

} // extern "C"
