// Gradient of y = act(z) + residual, z = x w^T + bias:
//
//   dz = dy act'(z),  dx = dz w,  dw = dz^T x,  db = sum over rows of dz
//
// The products (linear_impl.hpp) contract along rows, or along columns: in bf16, where rows
// begin at whole 16 bytes, dw takes dz and x as they lie then, and in fp32 products that are too few tiles
// to fill the chip take theirs, dx's w too. Otherwise x and dz are turned around first, and w. The pass over dy and
// the forward's z that forms dz turns it as well, and leaves db's partial rows (added by
// column_sums.hip in a fixed order); without an activation and a bias there is none. It is
// bound by memory. (32768 x 2048 x 2048 bf16, sigmoid: 711 us with x and dz turned, 623 without.)
//
// dz is fp32 in that pass, where db takes it, and is rounded to the operands' type for
// the products: the matrix instructions take no wider bf16 operand, and the
// gradients that leave are rounded to the same type.
#include "dense_launch.hpp"
#include "operators_launch.hpp"
#include "rows.hpp"

#include <algorithm>

namespace gdn2 {

// act'(z), with e = exp(-|z|) so that nothing cancels for large |z|
static __device__ __forceinline__ float sigmoid_slope(float u, float &s)
{
    // (the exponent's product is rounded once, as u itself was; the reciprocal is off by its last bit)
    // (the instruction gives 0 below 2^-126, which z may still make a number of: 64 steps up and down again)
    const float p = fabsf(u) * -1.44269504f, up = p < -100.f ? 64.f : 0.f;
    const float e = __builtin_amdgcn_exp2f(p + up) * (p < -100.f ? 0x1p-64f : 1.f), d = __builtin_amdgcn_rcpf(1.f + e);
    s = u < 0.f ? e * d : d;
    return e * d * d;
}
static __device__ __forceinline__ float slope_of(int act, float z)
{
    float s;
    if (act == kActSigmoid) return sigmoid_slope(z, s);
    if (act == kActSilu) {
        const float d = sigmoid_slope(z, s);
        return s + z * d;
    }
    if (act == kActGelu) {
        // (beyond 16 the sigmoid's slope is below the smallest float; z^2 may overflow there)
        if (fabsf(z) > 16.f) return z > 0.f ? 1.f : 0.f;
        const float u = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        const float d = sigmoid_slope(u, s);
        return s + z * d * 1.5957691216057308f * (1.f + 0.134145f * z * z);
    }
    return 1.f;
}

struct TurnArgs {
    const void *in;        // [R][C]
    const void *preact;    // [R][C], type of the outputs; null: in itself is what is turned
    void *copy;            // [R][Cp] or null
    void *turned;          // [C][Rp]; null: dz_kernel takes it
    float *partial;        // [gridDim.y][C] column sums, or null
    int64_t R, Rp;
    int C, Cp, act;
};

// Tiles of 64 x 64; a workgroup takes every gridDim.y-th of its 64 columns' tiles.
// Rp, Cp: R, C rounded up to eight, what is behind R, C filled with zeros.
template <typename In, typename T> __global__ __launch_bounds__(256) void turn_kernel(TurnArgs a)
{
    constexpr int PITCH = 64 + 16 / (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) T tile[64][PITCH];
    __shared__ float sums[32][64 + 4];
    const int p = threadIdx.x % 8, row = threadIdx.x / 8, c0 = blockIdx.x * 64, c = c0 + p * 8;
    float db[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t r0 = (int64_t)blockIdx.y * 64; r0 < a.Rp; r0 += (int64_t)gridDim.y * 64) {
        Pack8<In> x[2];
        Pack8<T> z[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = r0 + h * 32 + row, at = r * a.C + c;
            const int cnt = r < a.R ? a.C - c : 0;
            z[h].zero();
            if (cnt >= 8) {
                x[h].template load<false, false>((const In *)a.in + at);
                if (a.preact) z[h].template load<false, false>((const T *)a.preact + at);
            } else {
                x[h].load_some((const In *)a.in + at, cnt);
                if (a.preact) z[h].load_some((const T *)a.preact + at, cnt);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = r0 + h * 32 + row;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = x[h].get(i);
                if (a.preact) v[i] *= slope_of(a.act, z[h].get(i));
                db[i] += v[i];
            }
            if (a.copy && r < a.R && c < a.Cp) store8<true>((T *)a.copy + r * a.Cp + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) store1(&tile[h * 32 + row][p * 8 + i], v[i]);
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tc = h * 32 + row;     // column of the tile, row of the outcome
            const int64_t r = r0 + p * 8;
            if (c0 + tc < a.C && r < a.Rp) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = in2f<T>(tile[p * 8 + i][tc]);
                store8<true>((T *)a.turned + (int64_t)(c0 + tc) * a.Rp + r, v);
            }
        }
        __syncthreads();
    }
    if (a.partial) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[row][p * 8 + i] = db[i];
        __syncthreads();
        if (threadIdx.x < 64 && c0 + (int)threadIdx.x < a.C) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
            a.partial[(int64_t)blockIdx.y * a.C + c0 + threadIdx.x] = s;
        }
    }
}

// The same without anything turned: TX lanes take 8 TX neighbours of a row (whole
// pieces of memory: 32768 x 2048 bf16 94 us in tiles, 75 so, 5.4 TB/s), four rows at a time.
template <typename In, typename T, int TX> __global__ __launch_bounds__(256) void dz_kernel(TurnArgs a)
{
    constexpr int TY = 256 / TX, ROWS = 4;
    __shared__ float sums[TY > 1 ? TY : 1][TX * 8 + 4];
    const int p = threadIdx.x % TX, y = threadIdx.x / TX, c = (blockIdx.x * TX + p) * 8, cnt = a.C - c;
    float db[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t r0 = (int64_t)blockIdx.y * (TY * ROWS); r0 < a.R && c < a.Cp; r0 += (int64_t)gridDim.y * (TY * ROWS)) {
        Pack8<In> x[ROWS];
        Pack8<T> z[ROWS];
#pragma unroll
        for (int h = 0; h < ROWS; ++h) {
            const int64_t r = r0 + h * TY + y, at = r * a.C + c;
            const int n = r < a.R ? cnt : 0;
            z[h].zero();
            if (n >= 8) {
                x[h].template load<false, true>((const In *)a.in + at);
                if (a.preact) z[h].template load<false, true>((const T *)a.preact + at);
            } else {
                x[h].load_some((const In *)a.in + at, n);
                if (a.preact) z[h].load_some((const T *)a.preact + at, n);
            }
        }
#pragma unroll
        for (int h = 0; h < ROWS; ++h) {
            const int64_t r = r0 + h * TY + y;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = x[h].get(i);
                if (a.preact) v[i] *= slope_of(a.act, z[h].get(i));
                db[i] += v[i];
            }
            if (a.copy && r < a.R) store8<true>((T *)a.copy + r * a.Cp + c, v);
        }
    }
    if (!a.partial) return;
    if constexpr (TY > 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[y][p * 8 + i] = db[i];
        __syncthreads();
        for (int i = threadIdx.x; i < TX * 8; i += 256) {
            const int at = blockIdx.x * TX * 8 + i;
            if (at < a.C) {
                float s = 0.f;
#pragma unroll
                for (int t = 0; t < TY; ++t) s += sums[t][i];
                a.partial[(int64_t)blockIdx.y * a.C + at] = s;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < cnt) a.partial[(int64_t)blockIdx.y * a.C + c + i] = db[i];
    }
}

// How the rows of dz are shared: lanes across, workgroups across and down. With something
// turned, tiles, eight workgroups a compute unit in all; without, four.
struct DzShape { int tx, across, down; };
static DzShape dz_shape(int64_t R, int C, bool turned)
{
    DzShape d;
    d.tx = turned || C <= 64 ? 8 : C <= 256 ? 32 : C <= 1024 ? 128 : 256;
    d.across = (C + d.tx * 8 - 1) / (d.tx * 8);
    const int64_t rows = turned ? 64 : 256 / d.tx * 4;
    d.down = (int)std::max<int64_t>(1, std::min((R + rows - 1) / rows, (turned ? 2048 : 1024) / (int64_t)d.across));
    return d;
}

static void turn(TurnArgs a, bool in_bf16, bool bf16, const char *name, hipStream_t st)
{
    const DzShape d = dz_shape(a.R, a.C, a.turned);
    const dim3 grid(d.across, d.down);
    auto run = [&](auto in, auto out) {
        using In = decltype(in);
        using T = decltype(out);
        if (a.turned) hipLaunchKernelGGL((turn_kernel<In, T>), grid, dim3(256), 0, st, a);
        else if (d.tx == 8) hipLaunchKernelGGL((dz_kernel<In, T, 8>), grid, dim3(256), 0, st, a);
        else if (d.tx == 32) hipLaunchKernelGGL((dz_kernel<In, T, 32>), grid, dim3(256), 0, st, a);
        else if (d.tx == 128) hipLaunchKernelGGL((dz_kernel<In, T, 128>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((dz_kernel<In, T, 256>), grid, dim3(256), 0, st, a);
    };
    prof_before(name, st);
    if (bf16) {
        if (in_bf16) run(uint16_t(0), uint16_t(0));
        else run(0.f, uint16_t(0));
    } else {
        if (in_bf16) run(uint16_t(0), 0.f);
        else run(0.f, 0.f);
    }
    prof_after(st);
}

// Where the workspace's parts lie.
struct BwdLayout {
    size_t copy = 0, dzt = 0, xt = 0, wt = 0, partial = 0, db = 0, bytes = 0;
    bool need_copy, columns, w_columns;   // dw's operands, dx's w are taken as they lie
    int dx_splits = 1, dw_splits = 1;
};
static BwdLayout bwd_layout(int64_t M, int N, int K, int act, bool bf16, bool dy_bf16, bool dx, bool dw, bool db)
{
    BwdLayout l;
    const size_t e = bf16 ? 2 : 4;
    const int64_t Mp = (M + 7) / 8 * 8, Np = (N + 7) / 8 * 8, Kp = (K + 7) / 8 * 8;
    auto take = [&](size_t n) {
        const size_t at = l.bytes;
        l.bytes += (n + 255) / 256 * 256;
        return at;
    };
    l.columns = dw && M > 0 && (bf16 ? K % 8 == 0 : gemm_columns_f32(N, K, M, true));
    l.w_columns = dx && !bf16 && gemm_columns_f32(M, K, N, false);
    // dz where dy is not it, as it stands
    l.need_copy = (dx || l.columns) && (act != kActNone || dy_bf16 != bf16 || N % 8 != 0);
    if (l.need_copy) l.copy = take((size_t)M * Np * e);
    if (dw && !l.columns) {
        l.dzt = take((size_t)N * Mp * e);
        l.xt = take((size_t)Kp * Mp * e);
    }
    if (dx && !l.w_columns) l.wt = take((size_t)Kp * Np * e);
    size_t part = 0;
    if (dx && !l.w_columns && (l.dx_splits = gemm_splits(M, K, Np * e)) > 1) part = (size_t)l.dx_splits * M * Kp * 4;
    if (dw && (bf16 || !l.columns) && (l.dw_splits = l.columns ? gemm_columns_splits(N, K, M * e) : gemm_splits(N, K, Mp * e)) > 1)
        part = std::max(part, (size_t)l.dw_splits * N * Kp * 4);
    if (part) l.partial = take(part);
    if (db) l.db = take((size_t)dz_shape(M, N, dw && !l.columns).down * N * 4);
    return l;
}

size_t linear_bwd_workspace(int64_t M, int N, int K, int act, bool bf16, bool dy_bf16, bool dx, bool dw, bool db)
{
    return bwd_layout(M, N, K, act, bf16, dy_bf16, dx, dw, db).bytes;
}

hipError_t launch_linear_bwd(const LinearBwdArgs &a, hipStream_t st)
{
    const BwdLayout l = bwd_layout(a.M, a.N, a.K, a.act, a.bf16, a.dy_bf16, a.dx, a.dweight, a.dbias);
    const Elt elt = a.bf16 ? Elt::kBf16 : Elt::kF32;
    const size_t e = a.bf16 ? 2 : 4;
    const int64_t Mp = (a.M + 7) / 8 * 8;
    const int Np = (a.N + 7) / 8 * 8, Kp = (a.K + 7) / 8 * 8;
    char *ws = (char *)a.workspace;
    if (l.need_copy || (a.dweight && !l.columns) || a.dbias) {
        TurnArgs t = {};
        t.in = a.dy;
        t.preact = a.act == kActNone ? nullptr : a.preact;
        t.copy = l.need_copy ? ws + l.copy : nullptr;
        t.turned = a.dweight && !l.columns ? ws + l.dzt : nullptr;
        t.partial = a.dbias ? (float *)(ws + l.db) : nullptr;
        t.R = a.M; t.Rp = Mp; t.C = a.N; t.Cp = Np;
        t.act = a.act;
        turn(t, a.dy_bf16, a.bf16, "gdn2_linear_bwd_dz", st);
    }
    if (a.dx && a.M > 0) {
        GemmArgs m = {};
        m.x = l.need_copy ? ws + l.copy : a.dy;
        m.ldx = (int64_t)Np * e;
        m.M = a.M; m.N = a.K;
        m.y = a.dx;
        m.out_bf16 = a.bf16;
        m.partial = (float *)(ws + l.partial);
        m.ldp = Kp;
        m.splits = l.dx_splits;
        hipError_t err;
        if (l.w_columns) {
            m.w = a.w;
            m.ldw = (int64_t)a.K * 4;
            m.kbytes = (int64_t)a.N * 4;
            prof_before("gdn2_linear_bwd_dx", st);
            err = launch_gemm_columns_f32(m, false, st);
            prof_after(st);
        } else {
            TurnArgs t = {};
            t.in = a.w;
            t.turned = ws + l.wt;
            t.R = a.N; t.Rp = Np; t.C = a.K; t.Cp = Kp;
            turn(t, a.bf16, a.bf16, "gdn2_linear_bwd_turn", st);
            m.w = ws + l.wt;
            m.ldw = m.kbytes = (int64_t)Np * e;
            err = launch_gemm(elt, m, "gdn2_linear_bwd_dx", st);
        }
        if (err != hipSuccess) return err;
    }
    if (a.dweight) {
        GemmArgs m = {};
        m.M = a.N; m.N = a.K;
        m.y = a.dweight;
        m.out_bf16 = a.bf16;
        m.partial = (float *)(ws + l.partial);
        m.ldp = Kp;
        m.splits = l.dw_splits;
        hipError_t err;
        if (l.columns) {
            m.x = l.need_copy ? ws + l.copy : a.dy;
            m.w = a.x;
            m.ldx = (int64_t)Np * e;
            m.ldw = (int64_t)a.K * e;
            m.kbytes = a.M * e;
            prof_before("gdn2_linear_bwd_dw", st);
            err = a.bf16 ? launch_gemm_columns(m, st) : launch_gemm_columns_f32(m, true, st);
            prof_after(st);
        } else {
            TurnArgs t = {};
            t.in = a.x;
            t.turned = ws + l.xt;
            t.R = a.M; t.Rp = Mp; t.C = a.K; t.Cp = Kp;
            turn(t, a.bf16, a.bf16, "gdn2_linear_bwd_turn", st);
            m.x = ws + l.dzt;
            m.w = ws + l.xt;
            m.ldx = m.ldw = m.kbytes = Mp * e;
            err = launch_gemm(elt, m, "gdn2_linear_bwd_dw", st);
        }
        if (err != hipSuccess) return err;
    }
    if (a.dbias) {
        ColumnSums c = {};
        c.part[0] = (const float *)(ws + l.db);
        c.out0[0] = a.dbias;
        c.n0[0] = a.N;
        c.parts = dz_shape(a.M, a.N, a.dweight && !l.columns).down;
        c.jobs = 1;
        return launch_column_sums(c, "gdn2_linear_bwd_db", st);
    }
    return hipGetLastError();
}

// ---- the choice of a product's form ---------------------------------------------

// (rows x cols: the smaller tiles that a product of few of them takes)
static int splits_of(int64_t M, int64_t N, int64_t kbytes, int rows, int cols)
{
    auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
    const int64_t steps = (kbytes + 127) / 128, big = tiles(256, 256), small = tiles(rows, cols);
    if (M == 0 || big >= 192) return 1;
    // one part a compute unit, each of 16 steps at least
    int64_t s = std::min((256 + big - 1) / big, steps / 16);
    if (s >= 1 && big * s >= 192) return (int)s;
    s = std::min((512 + small - 1) / small, steps / 16);
    return s >= 2 ? (int)s : 1;
}
int gemm_splits(int64_t M, int64_t N, int64_t kbytes) { return splits_of(M, N, kbytes, 128, 64); }
int gemm_columns_splits(int64_t M, int64_t N, int64_t kbytes) { return splits_of(M, N, kbytes, 128, 128); }

bool gemm_columns_f32(int64_t M, int64_t N, int64_t count, bool turned_x)
{
    // blocks of 64 x 64 that fill half the chip at least and are too few for tiles; offsets of 32 bits. (Fewer blocks: the
    // contraction is split into parts instead. 4096 x 512 x 512: 69 us, 108 with dw in its 64 blocks.)
    const int64_t blocks = ((M + 63) / 64) * ((N + 63) / 64), most = 0x7fffffffLL;
    return blocks >= 128 && blocks < 2048 && N >= 64 && count * N * 4 < most &&
           (!turned_x || (M >= 64 && count * ((M + 7) / 8 * 8) * 4 < most));
}

hipError_t launch_gemm(Elt e, const GemmArgs &a, const char *name, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    prof_before(name, st);
    const hipError_t err = e == Elt::kBf16 ? launch_gemm_bf16(a, st) : e == Elt::kF32 ? launch_gemm_f32(a, st)
                                                                                     : launch_gemm_e4m3(a, st);
    prof_after(st);
    return err;
}

} // namespace gdn2
