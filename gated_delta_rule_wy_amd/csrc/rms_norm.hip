// Root-mean-square norm of x + residual over rows of `cols` elements, its output
// in bf16, fp32 or e4m3 with a scale a row, and its gradient: the norm before a
// layer's projections (linear_impl.hpp takes the e4m3 rows and their scales).
//
//   h = x + residual,  rstd = 1 / sqrt(sum h^2 / n + eps),  y = h rstd weight
//   e4m3: scale = max |y| / 448 (at least 2^-126), stored y / scale
//
//   backward, with xh = h rstd and g = dy weight:
//   dh = rstd (g - xh sum(g xh) / n) [+ dsum],  dweight = sum over rows of dy xh
//
// A row is read once and held in registers (row_parts.hpp, as in layer_norm.hip),
// so the largest |y| is known before the first element is stored and the 8-bit
// form costs no second pass. Bound by memory. Everything is fp32; y, the sum and dh are rounded
// once, as they are stored (e4m3 from the fp32 y, not from a bf16 one). The
// backward adds each workgroup's rows' terms of dweight in registers, in row
// order, and writes one partial row; column_sums.hip adds those in a fixed order.
#include "dense_launch.hpp"
#include "operators_launch.hpp"
#include "row_parts.hpp"

namespace gdn2 {

constexpr float kTopE4m3 = 448.f, kLeastScale = 1.17549435e-38f;

// A row's scale from its largest |y|, and the row's elements by it. y / scale = y 448 / top is taken with
// the roundings of its factors beside it and rounded once: an element next to a border between two e4m3 numbers
// falls to the right side of it (rstd's own error is in top as well). No slower: 65536 x 2048 157 us, 158 without.
struct RowScale {
    float scale, by, rest;   // 448 / top = by + rest
    __device__ __forceinline__ explicit RowScale(float top)
    {
        const float own = top / kTopE4m3;
        scale = fmaxf(own, kLeastScale);
        by = own >= kLeastScale ? kTopE4m3 / top : 1.f / scale;
        // (none of it where the row holds infinities or is scaled by the least scale, a power of two)
        rest = own >= kLeastScale && by > 0.f ? fmaf(-by, top, kTopE4m3) * (by * (1.f / kTopE4m3)) : 0.f;
    }
    __device__ __forceinline__ float operator()(float h, float rstd, float w) const
    {
        const float xh = h * rstd, y = xh * w, low = fmaf(fmaf(h, rstd, -xh), w, fmaf(xh, w, -y));
        return fmaf(y, by, fmaf(low, by, y * rest));
    }
};

template <typename In, typename Out, Packs P, int TPR, int E, bool RES>
__global__ __launch_bounds__((RowShape<TPR>::NT)) void rms_fwd_kernel(
    const In *x, const In *res, const float *__restrict__ weight, Out *y, float *scale, In *sum, int64_t rows, int cols,
    float inv_n, float eps)
{
    constexpr int RPB = RowShape<TPR>::RPB;
    constexpr bool kScaled = sizeof(Out) == 1;
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    const int grp = threadIdx.x / TPR;
    const RowPart<TPR, P> part = {(int)threadIdx.x % TPR, cols};
    float wv[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        Pack8<float> pw;
        part.template load<false>(pw, weight, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) wv[e][i] = pw.get(i);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
        // groups past the last row repeat it and store nothing
        const bool live = r0 + grp < rows;
        const int64_t row = live ? r0 + grp : rows - 1, base = row * (int64_t)cols;
        Pack8<In> px[E], pr[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            part.load(px[e], x + base, e);
            if (RES) part.load(pr[e], res + base, e);
        }
        float h[E][8], s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[e][i] = RES ? px[e].get(i) + pr[e].get(i) : px[e].get(i);
                s[0] += part.own(h[e][i] * h[e][i], e, i);
            }
        row_sums<TPR>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        if (live && sum)
#pragma unroll
            for (int e = 0; e < E; ++e) part.store(sum + base, h[e], e);
        if constexpr (kScaled) {
            float top = 0.f;   // (what a lane holds twice, or beyond the row as zeros, changes nothing)
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (P != Packs::kFew || part.mine(e, i)) top = fmaxf(top, fabsf(h[e][i] * rstd * wv[e][i]));
            const RowScale sc(row_max<TPR>(top, red));
            if (live && part.p == 0) scale[row] = sc.scale;
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i) h[e][i] = sc(h[e][i], rstd, wv[e][i]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i) h[e][i] = h[e][i] * rstd * wv[e][i];
        }
        if (live)
#pragma unroll
            for (int e = 0; e < E; ++e) part.store(y + base, h[e], e);
    }
}

// Rows longer than the registers hold: one workgroup a row, read again for each pass.
template <typename In, typename Out>
__global__ __launch_bounds__(1024) void rms_fwd_long_kernel(const In *x, const In *res, const float *__restrict__ weight,
                                                            Out *y, float *scale, In *sum, int64_t rows, int cols,
                                                            float inv_n, float eps)
{
    __shared__ float red[16];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * (int64_t)cols;
        auto at = [&](int c) { return in2f<In>(x[base + c]) + (res ? in2f<In>(res[base + c]) : 0.f); };
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < cols; c += 1024) s[0] += at(c) * at(c);
        row_sums<1024>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        float top = 0.f;
        if constexpr (sizeof(Out) == 1) {
            for (int c = threadIdx.x; c < cols; c += 1024) top = fmaxf(top, fabsf(at(c) * rstd * weight[c]));
            top = row_max<1024>(top, red);
        }
        const RowScale sc(top);
        if (sizeof(Out) == 1 && threadIdx.x == 0) scale[r] = sc.scale;
        for (int c = threadIdx.x; c < cols; c += 1024) {
            const float h = at(c);
            store1(y + base + c, sizeof(Out) == 1 ? sc(h, rstd, weight[c]) : h * rstd * weight[c]);
            if (sum) store1(sum + base + c, h);
        }
    }
}

// Gradient. partial: [gridDim.x][cols], this workgroup's sums of dy xh.
template <typename In, typename Dy, Packs P, int TPR, int E, bool SUM>
__global__ __launch_bounds__((RowShape<TPR>::NT)) __attribute__((amdgpu_waves_per_eu(TPR > 256 ? 4 : 2))) void rms_bwd_kernel(
    const Dy *dy, const In *h, const float *__restrict__ weight, const In *dsum, In *dh, float *__restrict__ partial,
    int64_t rows, int cols, float inv_n, float eps)
{
    constexpr int RPB = RowShape<TPR>::RPB;
    __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
    const int grp = threadIdx.x / TPR;
    const RowPart<TPR, P> part = {(int)threadIdx.x % TPR, cols};
    float wv[E][8], dw[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        Pack8<float> pw;
        part.template load<false>(pw, weight, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wv[e][i] = pw.get(i);
            dw[e][i] = 0.f;
        }
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
        const bool live = r0 + grp < rows;
        const int64_t base = (live ? r0 + grp : rows - 1) * (int64_t)cols;
        Pack8<In> ph[E], pa[E];
        Pack8<Dy> pd[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            part.load(ph[e], h + base, e);
            part.load(pd[e], dy + base, e);
            if (SUM) part.load(pa[e], dsum + base, e);
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = ph[e].get(i);
                s[0] += part.own(x * x, e, i);
                s[1] += part.own(x * (pd[e].get(i) * wv[e][i]), e, i);
            }
        row_sums<TPR>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        const float gx = s[1] * rstd * inv_n;   // mean of g xh
        if (live)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = ph[e].get(i) * rstd, d = pd[e].get(i);
                    o[i] = rstd * (d * wv[e][i] - xh * gx);
                    if (SUM) o[i] += pa[e].get(i);
                    dw[e][i] += d * xh;
                }
                part.store(dh + base, o, e);
            }
    }
    // the groups' sums, in group order, to this workgroup's partial row
    float *pw = partial + (size_t)blockIdx.x * cols;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) part.store(pw, dw[e], e);
    } else {
        // (element i of thread p at i * PITCH + p: no two of a step's lanes on one bank)
        constexpr int PITCH = TPR + 8;
        __shared__ float acc[RPB][8 * PITCH];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int back = part.col(e) - part.at(e);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (P != Packs::kOdd || part.mine(e, i)) acc[grp][(i - back) * PITCH + part.p] = dw[e][i];
            __syncthreads();
            for (int c = threadIdx.x; c < TPR * 8; c += RowShape<TPR>::NT) {
                const int cc = e * TPR * 8 + c;
                if (cc < cols) {
                    float t = 0.f;
#pragma unroll
                    for (int g = 0; g < RPB; ++g) t += acc[g][c % 8 * PITCH + c / 8];
                    pw[cc] = t;
                }
            }
            __syncthreads();
        }
    }
}

// Long rows: one workgroup a row at a time; its partial row is added to in
// place (the same thread owns a column throughout).
template <typename In, typename Dy>
__global__ __launch_bounds__(1024) void rms_bwd_long_kernel(const Dy *dy, const In *h, const float *__restrict__ weight,
                                                            const In *dsum, In *dh, float *part, int64_t rows, int cols,
                                                            float inv_n, float eps)
{
    __shared__ float red[32];
    float *pw = part + (size_t)blockIdx.x * cols;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * (int64_t)cols;
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < cols; c += 1024) {
            const float x = in2f<In>(h[base + c]);
            s[0] += x * x;
            s[1] += x * (in2f<Dy>(dy[base + c]) * weight[c]);
        }
        row_sums<1024>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        const float gx = s[1] * rstd * inv_n;
        const bool first = r == blockIdx.x;
        for (int c = threadIdx.x; c < cols; c += 1024) {
            const float xh = in2f<In>(h[base + c]) * rstd, d = in2f<Dy>(dy[base + c]);
            float o = rstd * (d * weight[c] - xh * gx);
            if (dsum) o += in2f<In>(dsum[base + c]);
            store1(dh + base + c, o);
            pw[c] = (first ? 0.f : pw[c]) + d * xh;
        }
    }
}

// ---- launch ------------------------------------------------------------------

template <typename In, typename Out> static void rms_fwd(const RmsNormArgs &a, hipStream_t st)
{
    const float inv_n = 1.f / (float)a.cols;
    auto args = [&](auto kern, int grid, int nt) {
        hipLaunchKernelGGL(kern, dim3(grid), dim3(nt), 0, st, (const In *)a.x, (const In *)a.residual, a.weight,
                           (Out *)a.y, a.scale, (In *)a.sum, a.rows, a.cols, inv_n, a.eps);
    };
    const bool held = for_row_shape(a.cols, [&](auto packs, auto t, auto e) {
        constexpr Packs P = decltype(packs)::value;
        constexpr int T = decltype(t)::value, E = decltype(e)::value;
        const int grid = row_grid(a.rows, RowShape<T>::RPB, kLnFwdGrid);
        if (a.residual) args(rms_fwd_kernel<In, Out, P, T, E, true>, grid, RowShape<T>::NT);
        else args(rms_fwd_kernel<In, Out, P, T, E, false>, grid, RowShape<T>::NT);
    });
    if (!held) args(rms_fwd_long_kernel<In, Out>, row_grid(a.rows, 1, kLnFwdGrid), 1024);
}

template <typename In, typename Dy> static void rms_bwd(const RmsNormBwdArgs &a, hipStream_t st)
{
    const float inv_n = 1.f / (float)a.cols;
    auto args = [&](auto kern, int grid, int nt) {
        hipLaunchKernelGGL(kern, dim3(grid), dim3(nt), 0, st, (const Dy *)a.dy, (const In *)a.h, a.weight,
                           (const In *)a.dsum, (In *)a.dh, (float *)a.workspace, a.rows, a.cols, inv_n, a.eps);
    };
    const int grid = ln_bwd_parts(a.rows, a.cols);
    const bool held = for_row_shape(a.cols, [&](auto packs, auto t, auto e) {
        constexpr Packs P = decltype(packs)::value;
        constexpr int T = decltype(t)::value, E = decltype(e)::value;
        if (a.dsum) args(rms_bwd_kernel<In, Dy, P, T, E, true>, grid, RowShape<T>::NT);
        else args(rms_bwd_kernel<In, Dy, P, T, E, false>, grid, RowShape<T>::NT);
    });
    if (!held) args(rms_bwd_long_kernel<In, Dy>, grid, 1024);
}

size_t rms_bwd_workspace(int64_t rows, int cols) { return (size_t)ln_bwd_parts(rows, cols) * cols * sizeof(float); }

hipError_t launch_rms_norm_fwd(const RmsNormArgs &a, hipStream_t st)
{
    if (a.rows == 0) return hipSuccess;
    prof_before("gdn2_rms_norm_fwd", st);
    if (a.in_bf16) {
        if (a.scale) rms_fwd<uint16_t, uint8_t>(a, st);
        else if (a.out_bf16) rms_fwd<uint16_t, uint16_t>(a, st);
        else rms_fwd<uint16_t, float>(a, st);
    } else {
        if (a.scale) rms_fwd<float, uint8_t>(a, st);
        else if (a.out_bf16) rms_fwd<float, uint16_t>(a, st);
        else rms_fwd<float, float>(a, st);
    }
    prof_after(st);
    return hipGetLastError();
}

hipError_t launch_rms_norm_bwd(const RmsNormBwdArgs &a, hipStream_t st)
{
    if (a.rows > 0) {
        prof_before("gdn2_rms_norm_bwd", st);
        if (a.in_bf16) {
            if (a.out_bf16) rms_bwd<uint16_t, uint16_t>(a, st);
            else rms_bwd<uint16_t, float>(a, st);
        } else {
            if (a.out_bf16) rms_bwd<float, uint16_t>(a, st);
            else rms_bwd<float, float>(a, st);
        }
        prof_after(st);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    // (no rows: no parts, and the weight's gradient is zeros)
    ColumnSums c = {};
    c.part[0] = (const float *)a.workspace;
    c.out0[0] = a.dweight;
    c.n0[0] = a.cols;
    c.parts = ln_bwd_parts(a.rows, a.cols);
    c.jobs = 1;
    return launch_column_sums(c, "gdn2_rms_norm_reduce", st);
}

} // namespace gdn2
