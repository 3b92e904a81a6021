// C ABI of a layer's dense half (declared in include/gdn2.h): projections, RMS
// norm, gradient clipping. Argument validation and dispatch; nothing is enqueued
// unless every check passes.
#include "dense_launch.hpp"
#include "operators_checks.hpp"

#include <algorithm>
#include <new>

using namespace gdn2;

extern "C" {

// ---- linear ------------------------------------------------------------------

static int linear_check(int64_t rows, int in_features, int out_features, int activation)
{
    if (rows < 0 || in_features < 1 || out_features < 1) return GDN2_ERR_INVALID;
    if (activation < GDN2_ACT_NONE || activation > GDN2_ACT_GELU_TANH) return GDN2_ERR_INVALID;
    if (in_features > GDN2_LINEAR_MAX_FEATURES || out_features > GDN2_LINEAR_MAX_FEATURES || rows > 0x7fff0000LL)
        return GDN2_ERR_UNSUPPORTED;
    // (one launch: tiles of 128 x 128, 512 threads each)
    auto tiles = [](int64_t a, int64_t b) { return ((a + 127) / 128) * ((b + 127) / 128) > 0x7fffffLL; };
    if (tiles(rows, out_features) || tiles(rows, in_features) || tiles(in_features, out_features))
        return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

int gdn2_linear_fwd(const void *x, const void *weight, const float *bias, const void *residual, const float *x_scale,
                    const float *weight_scale, void *y, void *preact, int64_t rows, int in_features, int out_features,
                    int activation, int in_dtype, int out_dtype)
{
    const int st = linear_check(rows, in_features, out_features, activation);
    if (st != GDN2_OK) return st;
    const bool e4m3 = in_dtype == GDN2_E4M3;
    if ((!dtype_ok(in_dtype) && !e4m3) || !dtype_ok(out_dtype)) return GDN2_ERR_INVALID;
    if (e4m3 && preact) return GDN2_ERR_INVALID;
    if (!e4m3 && (x_scale || weight_scale)) return GDN2_ERR_INVALID;
    if (rows > 0 && (!x || !weight || !y || (e4m3 && (!x_scale || !weight_scale)))) return GDN2_ERR_INVALID;
    const void *ptrs[] = {x, weight, bias, residual, x_scale, weight_scale, y, preact};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (rows == 0) return GDN2_OK;
    // y may be the residual
    if (twice({y, preact}) || same_memory({y, preact}, {x, weight, bias, x_scale, weight_scale}) ||
        same_memory({preact}, {residual}))
        return GDN2_ERR_INVALID;
    GemmArgs a = {};
    a.x = x;
    a.w = weight;
    a.ldx = a.ldw = a.kbytes = (int64_t)in_features * elt_size(e4m3 ? Elt::kE4m3 : in_dtype == GDN2_BF16 ? Elt::kBf16 : Elt::kF32);
    a.M = rows;
    a.N = out_features;
    a.sx = x_scale;
    a.sw = weight_scale;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    a.preact = preact;
    a.act = activation;
    a.out_bf16 = out_dtype == GDN2_BF16;
    a.preact_bf16 = in_dtype == GDN2_BF16;
    a.splits = 1;
    prof_call();
    return launch_status(launch_gemm(e4m3 ? Elt::kE4m3 : in_dtype == GDN2_BF16 ? Elt::kBf16 : Elt::kF32, a,
                                     "gdn2_linear_fwd", stream()));
}

size_t gdn2_linear_bwd_workspace_bytes(int64_t rows, int in_features, int out_features, int activation, int in_dtype,
                                       int dy_dtype, int need_dx, int need_dweight, int need_dbias)
{
    if (linear_check(rows, in_features, out_features, activation) != GDN2_OK) return 0;
    if (!dtype_ok(in_dtype) || !dtype_ok(dy_dtype) || rows > GDN2_LINEAR_BWD_MAX_ROWS) return 0;
    const size_t need = linear_bwd_workspace(rows, out_features, in_features, activation, in_dtype == GDN2_BF16,
                                             dy_dtype == GDN2_BF16, need_dx, need_dweight, need_dbias);
    return need > 0 ? need : 256;
}

int gdn2_linear_bwd(const void *dy, const void *x, const void *weight, const void *preact, void *dx, void *dweight,
                    float *dbias, int64_t rows, int in_features, int out_features, int activation, int in_dtype,
                    int dy_dtype, void *workspace, size_t workspace_bytes)
{
    const int st = linear_check(rows, in_features, out_features, activation);
    if (st != GDN2_OK) return st;
    if (!dtype_ok(in_dtype) || !dtype_ok(dy_dtype)) return GDN2_ERR_INVALID;
    if (!dx && !dweight && !dbias) return GDN2_ERR_INVALID;
    if (rows > GDN2_LINEAR_BWD_MAX_ROWS) return GDN2_ERR_UNSUPPORTED;
    if (rows > 0 && (!dy || (dweight && !x) || (dx && !weight) || (activation != GDN2_ACT_NONE && !preact)))
        return GDN2_ERR_INVALID;
    const void *ptrs[] = {dy, x, weight, preact, dx, dweight, dbias, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (!workspace || workspace_bytes < gdn2_linear_bwd_workspace_bytes(rows, in_features, out_features, activation, in_dtype,
                                                                       dy_dtype, dx != nullptr, dweight != nullptr,
                                                                       dbias != nullptr))
        return GDN2_ERR_WORKSPACE;
    const Ptrs outs = {rows > 0 ? dx : nullptr, dweight, dbias, workspace};
    if (twice(outs) || same_memory(outs, {dy, x, weight, preact})) return GDN2_ERR_INVALID;
    LinearBwdArgs a;
    a.dy = dy;
    a.x = x;
    a.w = weight;
    a.preact = preact;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.M = rows;
    a.N = out_features;
    a.K = in_features;
    a.act = activation;
    a.bf16 = in_dtype == GDN2_BF16;
    a.dy_bf16 = dy_dtype == GDN2_BF16;
    a.workspace = workspace;
    prof_call();
    return launch_status(launch_linear_bwd(a, stream()));
}

// ---- RMS norm ----------------------------------------------------------------

static int rms_norm_check(int64_t rows, int cols, float eps, int in_dtype)
{
    if (rows < 0 || cols < 1 || !dtype_ok(in_dtype)) return GDN2_ERR_INVALID;
    if (!(eps > 0.f && eps <= 3.4e38f)) return GDN2_ERR_INVALID;
    if (cols > GDN2_LAYER_NORM_MAX_COLS || rows > (int64_t)1 << 40) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

int gdn2_rms_norm_fwd(const void *x, const void *residual, const float *weight, void *y, float *scale, void *sum,
                      int64_t rows, int cols, float eps, int in_dtype, int out_dtype)
{
    const int st = rms_norm_check(rows, cols, eps, in_dtype);
    if (st != GDN2_OK) return st;
    const bool e4m3 = out_dtype == GDN2_E4M3;
    if (!dtype_ok(out_dtype) && !e4m3) return GDN2_ERR_INVALID;
    if (!e4m3 && scale) return GDN2_ERR_INVALID;
    if (rows > 0 && (!x || !weight || !y || (e4m3 && !scale))) return GDN2_ERR_INVALID;
    const void *ptrs[] = {x, residual, weight, y, scale, sum};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    // (in place only where the elements have one size; weights are never outputs)
    if (rows > 0 && (twice({y, scale, sum}) || same_memory({y, scale, sum}, {weight}) || same_memory({scale}, {x, residual}) ||
                     (in_dtype != out_dtype && same_memory({y}, {x, residual}))))
        return GDN2_ERR_INVALID;
    RmsNormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.sum = sum;
    a.scale = scale;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.in_bf16 = in_dtype == GDN2_BF16;
    a.out_bf16 = out_dtype == GDN2_BF16;
    prof_call();
    return launch_status(launch_rms_norm_fwd(a, stream()));
}

size_t gdn2_rms_norm_bwd_workspace_bytes(int64_t rows, int cols)
{
    if (rms_norm_check(rows, cols, 1.f, GDN2_F32) != GDN2_OK) return 0;
    const size_t need = rms_bwd_workspace(rows, cols);
    return need > 0 ? need : 256;
}

int gdn2_rms_norm_bwd(const void *dy, const void *h, const float *weight, const void *dsum, void *dh, float *dweight,
                      int64_t rows, int cols, float eps, int in_dtype, int out_dtype, void *workspace,
                      size_t workspace_bytes)
{
    const int st = rms_norm_check(rows, cols, eps, in_dtype);
    if (st != GDN2_OK) return st;
    if (!dtype_ok(out_dtype)) return GDN2_ERR_INVALID;
    if (!dweight || (rows > 0 && (!dy || !h || !weight || !dh))) return GDN2_ERR_INVALID;
    const void *ptrs[] = {dy, h, weight, dsum, dh, dweight, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_INVALID;
    if (!workspace || workspace_bytes < gdn2_rms_norm_bwd_workspace_bytes(rows, cols)) return GDN2_ERR_WORKSPACE;
    if (in_dtype != out_dtype && same_memory({dh}, {dy})) return GDN2_ERR_INVALID;
    if (rows == 0) dh = nullptr;   // (nothing is written there)
    if (twice({dh, dweight, workspace}) || same_memory({dh, dweight, workspace}, {weight}) ||
        same_memory({dweight, workspace}, {dy, h, dsum}))
        return GDN2_ERR_INVALID;
    RmsNormBwdArgs a;
    a.dy = dy;
    a.h = h;
    a.weight = weight;
    a.dsum = dsum;
    a.dh = dh;
    a.dweight = dweight;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.in_bf16 = in_dtype == GDN2_BF16;
    a.out_bf16 = out_dtype == GDN2_BF16;
    a.workspace = workspace;
    prof_call();
    return launch_status(launch_rms_norm_bwd(a, stream()));
}

// ---- gradient norm and clipping ------------------------------------------------

size_t gdn2_clip_grads_workspace_bytes(void) { return kClipGrid * sizeof(double); }

// One tensor's address range; out: it is written.
namespace {
struct Range {
    uintptr_t begin, end;
    int index;
    bool out;
};
}

// Whether an output (out: or null, the norm alone) shares memory with anything but its own gradient,
// in place; the norm (written or read) and the workspace (written, or null) among them.
static int clip_overlap(const void *const *grads, void *const *out, const int64_t *sizes, const int32_t *in_types,
                        const int32_t *out_types, int count, const float *norm, bool norm_given, const void *workspace, bool *bad)
{
    Range *r = new (std::nothrow) Range[2 * (size_t)count + 2];
    if (!r) return GDN2_ERR_HIP;
    int n = 0;
    r[n++] = {(uintptr_t)norm, (uintptr_t)norm + 4, -1, !norm_given};
    if (workspace) r[n++] = {(uintptr_t)workspace, (uintptr_t)workspace + gdn2_clip_grads_workspace_bytes(), -1, true};
    for (int i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        auto add = [&](const void *p, int type, bool o) {
            r[n++] = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)sizes[i] * (type == GDN2_BF16 ? 2 : 4), i, o};
        };
        if (out) add(out[i], out_types[i], true);
        if (!out || grads[i] != out[i] || in_types[i] != out_types[i]) add(grads[i], in_types[i], false);
    }
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.begin < b.begin; });
    // (the furthest end so far of the written ranges, and of all of them)
    uintptr_t out_end = 0, any_end = 0;
    *bad = false;
    for (int i = 0; i < n && !*bad; ++i) {
        *bad = r[i].begin < out_end || (r[i].out && r[i].begin < any_end);
        any_end = std::max(any_end, r[i].end);
        if (r[i].out) out_end = std::max(out_end, r[i].end);
    }
    delete[] r;
    return GDN2_OK;
}

static int clip_check(const void *const *grads, const int64_t *sizes, const int32_t *types, int count)
{
    if (count < 0 || (count > 0 && (!grads || !sizes || !types))) return GDN2_ERR_INVALID;
    for (int i = 0; i < count; ++i) {
        if (!dtype_ok(types[i]) || sizes[i] < 0) return GDN2_ERR_INVALID;
        if (sizes[i] > (int64_t)1 << 40) return GDN2_ERR_UNSUPPORTED;
        if (sizes[i] > 0 && (!grads[i] || (uintptr_t)grads[i] % (types[i] == GDN2_BF16 ? 2 : 4))) return GDN2_ERR_INVALID;
    }
    return GDN2_OK;
}

int gdn2_grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes, int count, float *norm,
                   void *workspace, size_t workspace_bytes)
{
    int st = clip_check(grads, sizes, dtypes, count);
    if (st != GDN2_OK) return st;
    if (!norm || (uintptr_t)norm % 4) return GDN2_ERR_INVALID;
    if (workspace && !aligned16(workspace)) return GDN2_ERR_INVALID;
    if (!workspace || workspace_bytes < gdn2_clip_grads_workspace_bytes()) return GDN2_ERR_WORKSPACE;
    bool bad;
    if ((st = clip_overlap(grads, nullptr, sizes, dtypes, nullptr, count, norm, false, workspace, &bad)) != GDN2_OK) return st;
    if (bad) return GDN2_ERR_INVALID;
    ClipArgs a = {};
    a.in = grads;
    a.sizes = sizes;
    a.in_types = dtypes;
    a.count = count;
    a.norm_out = norm;
    a.partial = (double *)workspace;
    prof_call();
    return launch_status(launch_clip(a, stream()));
}

int gdn2_clip_grads(const void *const *grads, void *const *out, const int64_t *sizes, const int32_t *dtypes,
                    const int32_t *out_dtypes, int count, float max_norm, float *norm, int norm_given, void *workspace,
                    size_t workspace_bytes)
{
    int st = clip_check(grads, sizes, dtypes, count);
    if (st != GDN2_OK) return st;
    if ((st = clip_check(out, sizes, out_dtypes, count)) != GDN2_OK) return st;
    if (!(max_norm >= 0.f && max_norm <= 3.4e38f) || !norm || (uintptr_t)norm % 4) return GDN2_ERR_INVALID;
    if (workspace && !aligned16(workspace)) return GDN2_ERR_INVALID;
    if (!norm_given && (!workspace || workspace_bytes < gdn2_clip_grads_workspace_bytes())) return GDN2_ERR_WORKSPACE;
    bool bad;
    if ((st = clip_overlap(grads, out, sizes, dtypes, out_dtypes, count, norm, norm_given, norm_given ? nullptr : workspace, &bad)) !=
        GDN2_OK)
        return st;
    if (bad) return GDN2_ERR_INVALID;
    ClipArgs a = {};
    a.in = grads;
    a.out = out;
    a.sizes = sizes;
    a.in_types = dtypes;
    a.out_types = out_dtypes;
    a.count = count;
    a.max_norm = max_norm;
    a.norm_in = norm_given ? norm : nullptr;
    a.norm_out = norm_given ? nullptr : norm;
    a.partial = (double *)workspace;
    prof_call();
    return launch_status(launch_clip(a, stream()));
}

} // extern "C"
