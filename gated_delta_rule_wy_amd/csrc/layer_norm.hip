// LayerNorm(x + residual) over rows of `cols` elements and its gradient: the
// layer's closing step (aifetchly-blog.pages.dev, "Gated DeltaNet-2 Guide",
// "End-to-End PyTorch Implementation": LayerNorm(x + out_proj(y))).
//
//   h = x + residual,  mean = sum h / n,  var = sum (h - mean)^2 / n,
//   rstd = 1 / sqrt(var + eps),  y = (h - mean) rstd weight + bias
//
//   backward, with xh = (h - mean) rstd and g = dy weight:
//   dh = rstd (g - sum(g) / n - xh sum(g xh) / n) [+ dsum]
//   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
//
// A row is read once and held in registers by TPR threads (a part of a wave,
// a wave or a workgroup), E packs of eight elements each; mean and variance are
// two passes over the registers, so an offset far from zero costs no
// precision. Rows pass through once, so they are loaded and stored past the
// caches (65536 x 2048 bf16 with residual and sum 193 us instead of 201, and 182
// with the weights loaded as vectors, 5.9 TB/s; backward 143 us instead of 159,
// now 137, 5.9 TB/s). Everything is fp32; y, sum and dh are rounded once, as
// they are stored. The statistics are those of the unrounded sum. Rows too long
// for the registers are read again for each pass (they stay in the L2).
//
// The backward takes the sum h and forms its statistics anew: the row is in
// registers anyway, and its gradient is then that of the h it was given.
// Each workgroup adds its rows' terms of dweight and dbias in registers, in
// row order, and writes one partial row; a second kernel adds the partial
// rows in a fixed order (no atomics: the same inputs give the same bits).
#include "operators_launch.hpp"
#include "row_parts.hpp"

#include <algorithm>

namespace gdn2 {

template <typename In, typename Out, Packs P, int TPR, int E, bool RES>
__global__ __launch_bounds__((RowShape<TPR>::NT)) void ln_fwd_kernel(
    const In *x, const In *res, const float *__restrict__ weight, const float *__restrict__ bias, Out *y, In *sum,
    int64_t rows, int cols, float inv_n, float eps)
{
    constexpr int RPB = RowShape<TPR>::RPB;
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    const int grp = threadIdx.x / TPR;
    const RowPart<TPR, P> part = {(int)threadIdx.x % TPR, cols};
    float wv[E][8], bv[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        Pack8<float> pw, pb;
        part.template load<false>(pw, weight, e);
        pb.zero();
        if (bias) part.template load<false>(pb, bias, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wv[e][i] = pw.get(i);
            bv[e][i] = pb.get(i);
        }
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
        // groups past the last row repeat it and store nothing
        const bool live = r0 + grp < rows;
        const int64_t base = (live ? r0 + grp : rows - 1) * (int64_t)cols;
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
                s[0] += part.own(h[e][i], e, i);
            }
        row_sums<TPR>(s, red);
        const float mean = s[0] * inv_n;
        s[0] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += part.mine(e, i) ? (h[e][i] - mean) * (h[e][i] - mean) : 0.f;
        row_sums<TPR>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        if (live)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = (h[e][i] - mean) * rstd * wv[e][i] + bv[e][i];
                part.store(y + base, o, e);
                if (sum) part.store(sum + base, h[e], e);
            }
    }
}

// Rows longer than the registers hold: one workgroup a row, three passes.
template <typename In, typename Out>
__global__ __launch_bounds__(1024) void ln_fwd_long_kernel(
    const In *x, const In *res, const float *__restrict__ weight, const float *__restrict__ bias, Out *y, In *sum,
    int64_t rows, int cols, float inv_n, float eps)
{
    __shared__ float red[16];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * (int64_t)cols;
        auto at = [&](int c) { return in2f<In>(x[base + c]) + (res ? in2f<In>(res[base + c]) : 0.f); };
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < cols; c += 1024) s[0] += at(c);
        row_sums<1024>(s, red);
        const float mean = s[0] * inv_n;
        s[0] = 0.f;
        for (int c = threadIdx.x; c < cols; c += 1024) s[0] += (at(c) - mean) * (at(c) - mean);
        row_sums<1024>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        for (int c = threadIdx.x; c < cols; c += 1024) {
            const float h = at(c), o = (h - mean) * rstd * weight[c] + (bias ? bias[c] : 0.f);
            store1(y + base + c, o);
            if (sum) store1(sum + base + c, h);
        }
    }
}

// Gradient. part: [gridDim.x][2][cols], this workgroup's sums of dy xh and dy.
template <typename In, typename Dy, Packs P, int TPR, int E, bool SUM>
__global__ __launch_bounds__((RowShape<TPR>::NT)) __attribute__((amdgpu_waves_per_eu(TPR > 256 ? 4 : 2))) void ln_bwd_kernel(
    const Dy *dy, const In *h, const float *__restrict__ weight, const In *dsum, In *dh, float *__restrict__ partial,
    int64_t rows, int cols, float inv_n, float eps)
{
    constexpr int RPB = RowShape<TPR>::RPB;
    __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
    const int grp = threadIdx.x / TPR;
    const RowPart<TPR, P> part = {(int)threadIdx.x % TPR, cols};
    float wv[E][8], dw[E][8], db[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        Pack8<float> pw;
        part.template load<false>(pw, weight, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wv[e][i] = pw.get(i);
            dw[e][i] = db[e][i] = 0.f;
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
                s[0] += part.own(ph[e].get(i), e, i);
                s[1] += part.own(pd[e].get(i) * wv[e][i], e, i);
            }
        row_sums<TPR>(s, red);
        const float mean = s[0] * inv_n, gm = s[1] * inv_n;
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = part.mine(e, i) ? ph[e].get(i) - mean : 0.f;
                s[0] += c * c;
                s[1] += c * (pd[e].get(i) * wv[e][i]);
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
                    const float xh = (ph[e].get(i) - mean) * rstd, d = pd[e].get(i);
                    o[i] = rstd * (d * wv[e][i] - gm - xh * gx);
                    if (SUM) o[i] += pa[e].get(i);
                    dw[e][i] += d * xh;
                    db[e][i] += d;
                }
                part.store(dh + base, o, e);
            }
    }
    // the groups' sums, in group order, to this workgroup's partial row
    float *pw = partial + (size_t)blockIdx.x * 2 * cols;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            part.store(pw, dw[e], e);
            part.store(pw + cols, db[e], e);
        }
    } else {
        // (element i of thread p at i * PITCH + p: eight lanes' stores and
        // eight columns' loads fall on different banks: 1111 x 1001 fp32 11.2
        // us, 11.8 with the columns in order)
        constexpr int PITCH = TPR + 8;
        __shared__ float acc[RPB][8 * PITCH];
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
            const int back = part.col(e % E) - part.at(e % E);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (P != Packs::kOdd || part.mine(e % E, i))
                    acc[grp][(i - back) * PITCH + part.p] = e < E ? dw[e % E][i] : db[e % E][i];
            __syncthreads();
            for (int c = threadIdx.x; c < TPR * 8; c += RowShape<TPR>::NT) {
                const int cc = (e % E) * TPR * 8 + c;
                if (cc < cols) {
                    float t = 0.f;
#pragma unroll
                    for (int g = 0; g < RPB; ++g) t += acc[g][c % 8 * PITCH + c / 8];
                    pw[(e < E ? 0 : cols) + cc] = t;
                }
            }
            __syncthreads();
        }
    }
}

// Long rows: one workgroup a row at a time; its partial row is added to in
// place (the same thread owns a column throughout).
template <typename In, typename Dy>
__global__ __launch_bounds__(1024) void ln_bwd_long_kernel(
    const Dy *dy, const In *h, const float *__restrict__ weight, const In *dsum, In *dh, float *part, int64_t rows,
    int cols, float inv_n, float eps)
{
    __shared__ float red[32];
    float *pw = part + (size_t)blockIdx.x * 2 * cols;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * (int64_t)cols;
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < cols; c += 1024) {
            s[0] += in2f<In>(h[base + c]);
            s[1] += in2f<Dy>(dy[base + c]) * weight[c];
        }
        row_sums<1024>(s, red);
        const float mean = s[0] * inv_n, gm = s[1] * inv_n;
        s[0] = s[1] = 0.f;
        for (int c = threadIdx.x; c < cols; c += 1024) {
            const float x = in2f<In>(h[base + c]) - mean;
            s[0] += x * x;
            s[1] += x * (in2f<Dy>(dy[base + c]) * weight[c]);
        }
        row_sums<1024>(s, red);
        const float rstd = 1.f / sqrtf(s[0] * inv_n + eps);
        const float gx = s[1] * rstd * inv_n;
        const bool first = r == blockIdx.x;
        for (int c = threadIdx.x; c < cols; c += 1024) {
            const float xh = (in2f<In>(h[base + c]) - mean) * rstd, d = in2f<Dy>(dy[base + c]);
            float o = rstd * (d * weight[c] - gm - xh * gx);
            if (dsum) o += in2f<In>(dsum[base + c]);
            store1(dh + base + c, o);
            pw[c] = (first ? 0.f : pw[c]) + d * xh;
            pw[cols + c] = (first ? 0.f : pw[cols + c]) + d;
        }
    }
}

// ---- launch ------------------------------------------------------------------

template <typename In, typename Out> static void ln_fwd(const LayerNormArgs &a, hipStream_t st)
{
    const float inv_n = 1.f / (float)a.cols;
    auto args = [&](auto kern, int grid, int nt) {
        hipLaunchKernelGGL(kern, dim3(grid), dim3(nt), 0, st, (const In *)a.x, (const In *)a.residual, a.weight, a.bias,
                           (Out *)a.y, (In *)a.sum, a.rows, a.cols, inv_n, a.eps);
    };
    const bool held = for_row_shape(a.cols, [&](auto packs, auto t, auto e) {
        constexpr Packs P = decltype(packs)::value;
        constexpr int T = decltype(t)::value, E = decltype(e)::value;
        const int grid = row_grid(a.rows, RowShape<T>::RPB, kLnFwdGrid);
        if (a.residual) args(ln_fwd_kernel<In, Out, P, T, E, true>, grid, RowShape<T>::NT);
        else args(ln_fwd_kernel<In, Out, P, T, E, false>, grid, RowShape<T>::NT);
    });
    if (!held) args(ln_fwd_long_kernel<In, Out>, row_grid(a.rows, 1, kLnFwdGrid), 1024);
}

template <typename In, typename Dy> static void ln_bwd(const LayerNormBwdArgs &a, hipStream_t st)
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
        if (a.dsum) args(ln_bwd_kernel<In, Dy, P, T, E, true>, grid, RowShape<T>::NT);
        else args(ln_bwd_kernel<In, Dy, P, T, E, false>, grid, RowShape<T>::NT);
    });
    if (!held) args(ln_bwd_long_kernel<In, Dy>, grid, 1024);
}

int ln_bwd_parts(int64_t rows, int cols)
{
    int rpb = 1;
    (void)for_row_shape(cols, [&](auto, auto t, auto) { rpb = RowShape<decltype(t)::value>::RPB; });
    // (wide rows: fewer parts, so that the partial rows stay within 64 MiB, or 32 rows)
    return row_grid(rows, rpb, std::max(32, std::min(kLnBwdGrid, (1 << 23) / cols)));
}

hipError_t launch_layer_norm_fwd(const LayerNormArgs &a, hipStream_t st)
{
    if (a.rows == 0) return hipSuccess;
    prof_before("gdn2_layer_norm_fwd", st);
    if (a.in_bf16) {
        if (a.out_bf16) ln_fwd<uint16_t, uint16_t>(a, st);
        else ln_fwd<uint16_t, float>(a, st);
    } else {
        if (a.out_bf16) ln_fwd<float, uint16_t>(a, st);
        else ln_fwd<float, float>(a, st);
    }
    prof_after(st);
    return hipGetLastError();
}

hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs &a, hipStream_t st)
{
    if (a.rows > 0) {
        prof_before("gdn2_layer_norm_bwd", st);
        if (a.in_bf16) {
            if (a.out_bf16) ln_bwd<uint16_t, uint16_t>(a, st);
            else ln_bwd<uint16_t, float>(a, st);
        } else {
            if (a.out_bf16) ln_bwd<float, uint16_t>(a, st);
            else ln_bwd<float, float>(a, st);
        }
        prof_after(st);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    // (no rows: no parts, and the weights' gradients are zeros)
    ColumnSums c = {};
    c.part[0] = (const float *)a.workspace;
    c.out0[0] = a.dweight;
    c.out1[0] = a.dbias;
    c.n0[0] = c.n1[0] = a.cols;
    c.parts = ln_bwd_parts(a.rows, a.cols);
    c.jobs = 1;
    return launch_column_sums(c, "gdn2_layer_norm_reduce", st);
}

} // namespace gdn2
