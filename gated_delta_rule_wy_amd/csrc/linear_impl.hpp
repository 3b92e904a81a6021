// Products of rows, y = act(x w^T ...) + residual, on the matrix cores (gfx950):
// x [M][K] and w [N][K] in one type (bf16, fp32, e4m3), sums in fp32.
//
// Both operands have the contracted axis along their rows, so a step is 128 bytes
// of each row whatever the type: 64 bf16, 32 fp32 or 128 e4m3 elements, eight
// chunks of 16 bytes. Which elements of a chunk meet in which matrix
// instruction is the same for both operands, and then no matter.
//
// The instructions' rows are w's, their columns x's: a lane's four sums
// are four neighbouring elements of a row of y.
#pragma once

#include "dense_launch.hpp"
#include "rows.hpp"

#include <algorithm>

namespace gdn2 {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef u4 u4_byte __attribute__((aligned(1)));

constexpr int kStep = 128;   // bytes of a row a step

// Products of two chunks of 16 w rows with two of 16 x rows (16 x 16 sums).
template <Elt T> struct Mm;
template <> struct Mm<Elt::kBf16> {
    static constexpr int kSize = 2;
    static __device__ __forceinline__ f4 mma(const u4 (&w)[2], const u4 (&x)[2], f4 c)
    {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, w[0]), __builtin_bit_cast(b8, x[0]), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, w[1]), __builtin_bit_cast(b8, x[1]), c, 0, 0, 0);
    }
};
template <> struct Mm<Elt::kF32> {
    static constexpr int kSize = 4;
    static __device__ __forceinline__ f4 mma(const u4 (&w)[2], const u4 (&x)[2], f4 c)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[j][i]), __uint_as_float(x[j][i]), c, 0, 0, 0);
        return c;
    }
};
template <> struct Mm<Elt::kE4m3> {
    static constexpr int kSize = 1;
    static __device__ __forceinline__ f4 mma(const u4 (&w)[2], const u4 (&x)[2], f4 c)
    {
        struct P { u4 a[2]; };
        const P pw = {{w[0], w[1]}}, px = {{x[0], x[1]}};
        // both e4m3, block scales 2^0
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i8v, pw), __builtin_bit_cast(i8v, px), c, 0,
                                                                0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
    }
};

// Chunk at byte `at` of a row of `bytes`, zeros behind its end. ODD: rows begin
// at any element, and a row's last chunk may be a part of one.
template <Elt T, bool ODD> static __device__ __forceinline__ u4 load_chunk(const char *row, int64_t at, int64_t bytes)
{
    u4 r = {0u, 0u, 0u, 0u};
    if constexpr (!ODD) {
        if (at < bytes) r = *reinterpret_cast<const u4 *>(row + at);
    } else {
        if (at + 16 <= bytes) {
            r = *reinterpret_cast<const u4_byte *>(row + at);
        } else {
            constexpr int S = Mm<T>::kSize;
#pragma unroll
            for (int i = 0; i < 16; i += S)
                if (at + i < bytes) {
                    uint32_t v;
                    if constexpr (S == 4) v = *reinterpret_cast<const uint32_t *>(row + at + i);
                    else if constexpr (S == 2) v = *reinterpret_cast<const uint16_t *>(row + at + i);
                    else v = *reinterpret_cast<const uint8_t *>(row + at + i);
                    r[i / 4] |= v << (8 * (i % 4));
                }
        }
    }
    return r;
}

// ---- the epilogue ----------------------------------------------------------------

// 1 / (1 + exp(-z)): exp overflows to infinity and its reciprocal to 0
static __device__ __forceinline__ float sigmoid_of(float z) { return __builtin_amdgcn_rcpf(1.f + expf(-z)); }

template <int ACT> static __device__ __forceinline__ float act_of(float z)
{
    if (ACT == kActSigmoid) return sigmoid_of(z);
    if (ACT == kActSilu) return z * sigmoid_of(z);
    // gelu's tanh form, 0.5 z (1 + tanh(u / 2)) = z sigmoid(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
    if (ACT == kActGelu) return z * sigmoid_of(1.5957691216057308f * (z + 0.044715f * z * z * z));
    return z;
}

// Calls f with the activation as a constant.
template <typename F> static __device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case kActSigmoid: f(std::integral_constant<int, kActSigmoid>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default: break;
    }
}

// Eight neighbours of a row (n: of them in the row; fewer than eight: one by
// one). Addresses are those of any element: rows of odd lengths follow each other.
static __device__ __forceinline__ void get8(const float *p, int n, float (&x)[8])
{
    Pack8<float> r;
    if (n >= 8) r.template load<false, false>(p);
    else r.load_some(p, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = r.get(i);
}
static __device__ __forceinline__ void get8(const uint16_t *p, int n, float (&x)[8])
{
    Pack8<uint16_t> r;
    if (n >= 8) r.template load<false, false>(p);
    else r.load_some(p, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = r.get(i);
}
template <typename T> static __device__ __forceinline__ void put8(T *p, int n, const float (&x)[8])
{
    if (n >= 8) {
        store8<false>(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) store1(p + i, x[i]);
    }
}
static __device__ __forceinline__ void put8(void *p, bool bf16, int64_t at, int n, const float (&x)[8])
{
    if (bf16) put8((uint16_t *)p + at, n, x);
    else put8((float *)p + at, n, x);
}

// The steps of the epilogue for eight sums of row m, columns n .. n + 7 (cnt of
// them in the row): up to z, and from act(z) on.
static __device__ __forceinline__ void to_preact(const GemmArgs &a, int64_t m, int64_t n, int cnt, float (&v)[8])
{
    float s[8];
    if (a.sw) {
        const float sx = a.sx[m];
        get8(a.sw + n, cnt, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sx * s[i];
    }
    if (a.bias) {
        get8(a.bias + n, cnt, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += s[i];
    }
    if (a.preact) put8(a.preact, a.preact_bf16, m * a.N + n, cnt, v);
}
static __device__ __forceinline__ void to_output(const GemmArgs &a, int64_t m, int64_t n, int cnt, float (&v)[8])
{
    const int64_t at = m * a.N + n;
    if (a.residual) {
        float s[8];
        if (a.out_bf16) get8((const uint16_t *)a.residual + at, cnt, s);
        else get8((const float *)a.residual + at, cnt, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += s[i];
    }
    put8(a.y, a.out_bf16, at, cnt, v);
}
static __device__ __forceinline__ void finish8(const GemmArgs &a, int64_t m, int64_t n, int cnt, float (&v)[8])
{
    to_preact(a, m, n, cnt, v);
    with_act(a.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_of<decltype(act)::value>(v[i]);
    });
    to_output(a, m, n, cnt, v);
}

// ---- few tiles: every wave a part of the contraction -----------------------------
//
// A workgroup of W waves owns 16 MB rows of x and 16 NB of w. Wave i takes the
// steps i, i + W, ... straight from memory into the instructions' operands
// (nothing is used twice that could be shared through LDS), and the waves' sums are
// added through LDS in wave order.
constexpr int kWaves = 8;

template <Elt T, int MB, int NB, bool ODD> __global__ __launch_bounds__(kWaves * 64) void gemm_split_kernel(GemmArgs a)
{
    constexpr int PITCH = NB * 16 + 4;                   // floats a row of the sums (16-byte aligned, banks apart)
    constexpr int ROUNDS = MB * NB > 4 ? 2 : 1, MR = MB / ROUNDS;   // blocks of rows a round through LDS
    static_assert(MB % ROUNDS == 0, "whole blocks of rows a round");
    __shared__ __attribute__((aligned(16))) float sums[kWaves][MR * 16 * PITCH];
    const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * (MB * 16), n0 = (int64_t)blockIdx.x * (NB * 16);
    const char *px[MB], *pw[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) px[i] = (const char *)a.x + min(m0 + i * 16 + r, a.M - 1) * a.ldx;
#pragma unroll
    for (int i = 0; i < NB; ++i) pw[i] = (const char *)a.w + min(n0 + i * 16 + r, a.N - 1) * a.ldw;
    f4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = f4zero();
    const int steps = (int)((a.kbytes + kStep - 1) / kStep);
#pragma unroll 2
    for (int s = wv; s < steps; s += kWaves) {
        const int64_t k = (int64_t)s * kStep + g * 32;
        u4 fx[MB][2], fw[NB][2];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) fw[j][c] = load_chunk<T, ODD>(pw[j], k + c * 16, a.kbytes);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) fx[i][c] = load_chunk<T, ODD>(px[i], k + c * 16, a.kbytes);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < MB; ++i) acc[j][i] = Mm<T>::mma(fw[j], fx[i], acc[j][i]);
    }
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
        if (q) __syncthreads();
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < MR; ++i)
                *reinterpret_cast<f4 *>(&sums[wv][(i * 16 + r) * PITCH + j * 16 + g * 4]) = acc[j][q * MR + i];
        __syncthreads();
        for (int e = threadIdx.x; e < MR * 16 * NB * 2; e += kWaves * 64) {
            const int row = e / (NB * 2), col = e % (NB * 2) * 8;
            const int64_t m = m0 + q * MR * 16 + row, n = n0 + col;
            if (m < a.M && n < a.N) {
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kWaves; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f4 s = *reinterpret_cast<const f4 *>(&sums[i][row * PITCH + col + h * 4]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[h * 4 + c] += s[c];
                    }
                finish8(a, m, n, (int)min((int64_t)8, a.N - n), v);
            }
        }
    }
}

// ---- many tiles -------------------------------------------------------------------
//
// A workgroup of WM x WN waves owns BM rows of x and BN of w. Each step's
// chunks lie in LDS, two steps at a time: while the waves multiply one, the next
// is on its way, without a register in between (ODD: through registers, since
// the direct way takes whole aligned chunks).
//
// A fragment's 16 rows, 128 bytes apart, would fall on the same banks; so chunk c
// of row i lies at position c ^ swap(i), and neighbouring pairs of rows that are
// read together differ in it.
//
// Which of w's rows an instruction takes as its 16 is free, too: block j of a
// pair takes rows 8 t + 4 j + (0..3), t = 0..3, of the pair's 32, so that
// a lane's sums of both blocks are eight neighbours of a row of y.
static __device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// (rows r, r + 1 share one: a row is half as long as all banks together)
static __device__ __forceinline__ int swap_x(int row) { return (row >> 1) & 7; }
static __device__ __forceinline__ int swap_w(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }

template <Elt T, int BM, int BN, int WM, int WN, bool ODD>
__global__ __launch_bounds__(WM * WN * 64) void gemm_tile_kernel(GemmArgs a, int tm, int tn)
{
    constexpr int NW = WM * WN, MB = BM / WM / 16, NB = BN / WN / 16;   // waves; blocks of 16 rows a wave
    constexpr int RX = BM / 8 / NW, RW = BN / 8 / NW;                   // groups of 8 rows each wave brings
    constexpr int BUF = (BM + BN) * kStep;
    static_assert(RX * 8 * NW == BM && RW * 8 * NW == BN && NB % 2 == 0, "whole groups a wave, whole pairs");
    static_assert(NW % 4 == 0, "a wave's groups keep their place in 32 rows");
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF + 16 * (BM / 2)];   // (the sums' rows are a little longer)
    const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
    // neighbouring tiles to one XCD (workgroups go round the eight of them)
    int tile;
    {
        const int all = tm * tn, id = blockIdx.x, xcd = id & 7, q = all >> 3, rest = all & 7;
        tile = xcd * q + min(xcd, rest) + (id >> 3);
    }
    // tiles in bands of four of x's
    const int band = tile / (4 * tn), inb = tile % (4 * tn), bm = min(4, tm - band * 4);
    const int64_t m0 = (int64_t)(band * 4 + inb % bm) * BM, n0 = (int64_t)(inb / bm) * BN;

    // what this lane brings: row lane / 8 of a group, and the chunk that belongs at position lane % 8
    const int grow = lane >> 3;
    const int cx = ((lane & 7) ^ swap_x((wv & 1) * 8 + grow)) * 16, cw = ((lane & 7) ^ swap_w((wv & 3) * 8 + grow)) * 16;
    const char *px[RX], *pw[RW];
#pragma unroll
    for (int i = 0; i < RX; ++i) px[i] = (const char *)a.x + min(m0 + (i * NW + wv) * 8 + grow, a.M - 1) * a.ldx + cx;
#pragma unroll
    for (int i = 0; i < RW; ++i) pw[i] = (const char *)a.w + min(n0 + (i * NW + wv) * 8 + grow, a.N - 1) * a.ldw + cw;
    const int steps = (int)((a.kbytes + kStep - 1) / kStep);
    const int s0 = (int)((int64_t)steps * blockIdx.y / a.splits), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / a.splits);

    u4 staged[ODD ? RX + RW : 1];
    auto bring = [&](const char *p, char *to) {
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)p,
                                         (__attribute__((address_space(3))) void *)to, 16, 0, 0);
    };
    auto fetch = [&](int s, char *buf) {
        const int64_t k = (int64_t)s * kStep;
        if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < RX; ++i) staged[i] = load_chunk<T, true>(px[i] - cx, k + cx, a.kbytes);
#pragma unroll
            for (int i = 0; i < RW; ++i) staged[RX + i] = load_chunk<T, true>(pw[i] - cw, k + cw, a.kbytes);
        } else if (k + kStep <= a.kbytes) {
#pragma unroll
            for (int i = 0; i < RX; ++i) bring(px[i] + k, buf + (i * NW + wv) * 1024);
#pragma unroll
            for (int i = 0; i < RW; ++i) bring(pw[i] + k, buf + BM * kStep + (i * NW + wv) * 1024);
        } else {
            const char *zeros = (const char *)kZeros;
#pragma unroll
            for (int i = 0; i < RX; ++i) bring(k + cx < a.kbytes ? px[i] + k : zeros, buf + (i * NW + wv) * 1024);
#pragma unroll
            for (int i = 0; i < RW; ++i)
                bring(k + cw < a.kbytes ? pw[i] + k : zeros, buf + BM * kStep + (i * NW + wv) * 1024);
        }
    };
    auto settle = [&](char *buf) {
        if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < RX; ++i) *reinterpret_cast<u4 *>(buf + (i * NW + wv) * 1024 + lane * 16) = staged[i];
#pragma unroll
            for (int i = 0; i < RW; ++i)
                *reinterpret_cast<u4 *>(buf + BM * kStep + (i * NW + wv) * 1024 + lane * 16) = staged[RX + i];
        }
    };

    f4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = f4zero();
    const int wm = wv % WM, wn = wv / WM;
    // chunk g of this lane's row of a block; chunk g + 4 is at the same place ^ 64
    const int wrow = 8 * (r >> 2) + (r & 3);
    const int ox = (wm * (BM / WM) + r) * kStep + ((g ^ swap_x(r)) << 4);
    int ow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        ow[j] = (BM + wn * (BN / WN) + wrow + 4 * j) * kStep + ((g ^ swap_w(wrow + 4 * j)) << 4);

    if (s0 < s1) {
        fetch(s0, lds);
        settle(lds);
    }
    for (int s = s0; s < s1; ++s) {
        char *cur = lds + ((s - s0) & 1) * BUF, *next = lds + ((s - s0 + 1) & 1) * BUF;
        __syncthreads();   // (waits for this wave's loads into cur, and for every wave to have left next)
        if (s + 1 < s1) fetch(s + 1, next);
        u4 fw[NB][2];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                fw[j][c] = *reinterpret_cast<const u4 *>(cur + (j >> 1) * 32 * kStep + (ow[j & 1] ^ (64 * c)));
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            u4 fx[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) fx[c] = *reinterpret_cast<const u4 *>(cur + i * 16 * kStep + (ox ^ (64 * c)));
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[j][i] = Mm<T>::mma(fw[j], fx, acc[j][i]);
        }
        if (s + 1 < s1) settle(next);
    }

    // The sums go through LDS, so that lanes take whole lines of y (and of the
    // residual), eight elements each, in a short loop. kRows of each wave's rows a round.
    constexpr int PITCH = BN + 4, kRows = 16 * (MB / 2), TPR = BN / 8;
    static_assert(WM * kRows * PITCH * 4 <= (int)sizeof(lds), "the sums of a round");
    float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        __syncthreads();   // (every wave has read its last operands, or the last round's sums)
#pragma unroll
        for (int i = 0; i < MB / 2; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                *reinterpret_cast<f4 *>(&sums[(wm * kRows + i * 16 + r) * PITCH + wn * (BN / WN) + (j >> 1) * 32 + (j & 1) * 4 +
                                              g * 8]) = acc[j][q * (MB / 2) + i];
        __syncthreads();
        const int col = threadIdx.x % TPR * 8;
        const int64_t n = n0 + col;
        if (n < a.N) {
            const int cnt = (int)min((int64_t)8, a.N - n);
            for (int row = threadIdx.x / TPR; row < WM * kRows; row += NW * 64 / TPR) {
                const int64_t m = m0 + row / kRows * (BM / WM) + q * kRows + row % kRows;
                if (m >= a.M) continue;
                float v[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f4 x = *reinterpret_cast<const f4 *>(&sums[row * PITCH + col + h * 4]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[h * 4 + c] = x[c];
                }
                if (a.splits > 1) put8(a.partial + ((int64_t)blockIdx.y * a.M + m) * a.N + n, cnt, v);
                else finish8(a, m, n, cnt, v);
            }
        }
    }
}

// The parts' sums, in order, and the epilogue.
static __global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs a)
{
    const int64_t runs = (a.N + 7) / 8, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= a.M * runs) return;
    const int64_t m = e / runs, n = e % runs * 8;
    const int cnt = (int)min((int64_t)8, a.N - n);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) {
        float x[8];
        get8(a.partial + ((int64_t)s * a.M + m) * a.N + n, cnt, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += x[c];
    }
    finish8(a, m, n, cnt, v);
}

// ---- launch -------------------------------------------------------------------------

template <Elt T, bool ODD> static hipError_t launch_gemm_forms(const GemmArgs &a, hipStream_t st)
{
    auto tiles = [](int64_t rows, int b) { return (rows + b - 1) / b; };
    auto split = [&](auto mb, auto nb) {
        constexpr int MB = decltype(mb)::value, NB = decltype(nb)::value;
        const int64_t gx = tiles(a.N, NB * 16), gy = tiles(a.M, MB * 16);
        if (gy > 65535 || gx * gy > 0x7fffffLL) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((gemm_split_kernel<T, MB, NB, ODD>), dim3((unsigned)gx, (unsigned)gy), dim3(kWaves * 64), 0, st, a);
        return hipGetLastError();
    };
    auto tiled = [&](auto bm, auto bn, auto wm, auto wn) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
        const int64_t tm = tiles(a.M, BM), tn = tiles(a.N, BN);
        if (tm * tn > 0x7fffffLL) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((gemm_tile_kernel<T, BM, BN, WM, WN, ODD>), dim3((unsigned)(tm * tn), a.splits),
                           dim3(WM * WN * 64), 0, st, a, (int)tm, (int)tn);
        return hipGetLastError();
    };
    using i1 = std::integral_constant<int, 1>;
    using i2 = std::integral_constant<int, 2>;
    using i4 = std::integral_constant<int, 4>;
    using i128 = std::integral_constant<int, 128>;
    if (a.splits == 1) {
        if (a.M <= 16) return split(i1{}, i1{});
        if (a.M <= 32) return split(i2{}, i1{});
        if (a.M <= 64) return split(i4{}, i1{});
        if (tiles(a.M, 64) * tiles(a.N, 64) <= 512) return split(i4{}, i4{});
    }
    if constexpr (!ODD) {
        using i256 = std::integral_constant<int, 256>;
        if (tiles(a.M, 256) * tiles(a.N, 256) * a.splits >= 192) return tiled(i256{}, i256{}, i4{}, i2{});
    }
    return tiled(i128{}, i128{}, i2{}, i2{});
}

template <Elt T> static hipError_t launch_gemm_type(const GemmArgs &a, hipStream_t st)
{
    const bool odd = a.ldx % 16 || a.ldw % 16 || a.kbytes % 16;
    const hipError_t err = odd ? launch_gemm_forms<T, true>(a, st) : launch_gemm_forms<T, false>(a, st);
    if (err != hipSuccess || a.splits == 1) return err;
    const int64_t blocks = (a.M * ((a.N + 7) / 8) + 255) / 256;
    if (blocks > 0xffffffLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(gemm_join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn2
