// Products of rows, y = act(x w^T ...) + residual, on the matrix cores (gfx950):
// x [M][K] and w [N][K] in one type (bf16, fp32, e4m3), sums in fp32.
//
// Both operands have the contracted axis along their rows, so a step is 128 bytes
// of each row whatever the type: 64 bf16, 32 fp32 or 128 e4m3 elements, eight
// chunks of 16 bytes. Which elements of a chunk meet in which matrix
// instruction is the same for both operands, and then no matter.
//
// Products are exact and sums fp32. The matrix instructions for e4m3 do not add so: all of them first add aligned
// eights of products with 13 bits below the largest of the eight (those for bf16 keep 24 there). So
// e4m3 operands are widened to bf16, which holds them, and multiplied by bf16's instructions. Only the tiles whose y is
// rounded to bf16 take eights: they are bound by that rate, which is half with bf16 (32768 x 8192 x 2048 511 us, 845
// widened; 1000 x 2048 x 2048 9.9 and 13.5; to fp32, widened, 928 and 14.2). What is left out there is up to 2^-13 of an
// eight's largest product for each of the other seven: for random rows of 2048 2e-5 of a sum, an
// eightieth of the rounding that follows. In the blocks below widening costs at most 5 % (256 x 2048 x 2048 9.9 us and 9.4).
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

#define GDN2_INLINE __attribute__((always_inline))
static __device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

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
// Half h of a chunk of e4m3 numbers as bf16, which holds every one of them.
static __device__ __forceinline__ b8 widened(u4 q, int h)
{
    struct P { bf2 a[4]; } p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        p.a[i * 2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[h * 2 + i], 1.f, false);
        p.a[i * 2 + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[h * 2 + i], 1.f, true);
    }
    return __builtin_bit_cast(b8, p);
}
template <> struct Mm<Elt::kE4m3> {
    static constexpr int kSize = 1;
    static __device__ __forceinline__ f4 mma(const u4 (&w)[2], const u4 (&x)[2], f4 c)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widened(w[j], h), widened(x[j], h), c, 0, 0, 0);
        return c;
    }
};

// Chunk at byte `at` of a row of `bytes` that begins at any element and may end
// with a part of one; zeros behind its end.
template <Elt T> static __device__ __forceinline__ u4 load_chunk(const char *row, int64_t at, int64_t bytes)
{
    u4 r = {0u, 0u, 0u, 0u};
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
    return r;
}

// A buffer descriptor from `at` bytes into `base` to its end at `end` bytes: what is
// read beyond arrives as zeros, what is written there is dropped. Offsets are
// whole in the vector operand, which the bounds are checked against; kBeyond is
// outside always.
constexpr uint32_t kBeyond = 0xFFFFFF80u;   // (and 16 bytes on)
constexpr int kOnce = 2;   // cache policy: not to be kept (y would push x's and w's lines out of the L2)
static __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void *base, int64_t at, int64_t end)
{
    const uint32_t left = (end - at) >> 32 ? 0xFFFFFF00u : (uint32_t)(end - at);
    return __builtin_amdgcn_make_buffer_rsrc((char *)const_cast<void *>(base) + at, (short)0, (int)left, 0x00020000);
}

// ---- the epilogue ----------------------------------------------------------------

// 1 / (1 + exp(-z)); exp overflows to infinity, whose reciprocal is 0. The exponent's
// product with log2 e is rounded once, which is to z as one more rounding of its own.
static __device__ __forceinline__ float sigmoid_of(float z)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

template <int ACT> static __device__ __forceinline__ float act_of(float z)
{
    if (ACT == kActSigmoid) return sigmoid_of(z);
    if (ACT == kActSilu) return z * sigmoid_of(z);
    // gelu's tanh form, 0.5 z (1 + tanh(u / 2)) = z sigmoid(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
    if (ACT == kActGelu) return z * sigmoid_of(1.5957691216057308f * (z + 0.044715f * z * z * z));
    return z;
}

// v times a row's and a channel's scale, which may have a product that no float holds although v times both is one. So
// they are multiplied as mantissas and exponents: a sum's own range is short (e4m3 products are 2^-18 to 2^18), its
// product with two mantissas cannot leave the floats', and the power of two is exact but at their ends. (Two
// instructions an element more than v (a b), whose bits it has wherever a b is a normal number: 32768 x 8192 x 2048 to
// bf16 511 us, 501 with v (a b), 16384 x 4096 x 2048 137.7 either way. Checking the wave's scales first, to take v (a b)
// where that will do, costs as much: 512 to 515 and 140 to 143. Nor is it less with mantissas made anew for each block.)
static __device__ __forceinline__ float scaled(float v, float a, float b)
{
    return __builtin_amdgcn_ldexpf(v * (__builtin_amdgcn_frexp_mantf(a) * __builtin_amdgcn_frexp_mantf(b)),
                                   __builtin_amdgcn_frexp_expf(a) + __builtin_amdgcn_frexp_expf(b));
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

// The epilogue of eight sums of row m, columns n .. n + 7 (cnt of them in the
// row): what it reads, on its way before the sums are there, and then y.
struct Finish8 {
    float sw[8], bias[8], res[8], sx;
    __device__ __forceinline__ void load(const GemmArgs &a, int64_t m, int64_t n, int cnt)
    {
        if (a.sw) {
            sx = a.sx[m];
            get8(a.sw + n, cnt, sw);
        }
        if (a.bias) get8(a.bias + n, cnt, bias);
        if (a.residual) {
            if (a.out_bf16) get8((const uint16_t *)a.residual + m * a.N + n, cnt, res);
            else get8((const float *)a.residual + m * a.N + n, cnt, res);
        }
    }
    __device__ __forceinline__ void store(const GemmArgs &a, int64_t m, int64_t n, int cnt, float (&v)[8]) const
    {
        const int64_t at = m * a.N + n;
        if (a.sw)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = scaled(v[i], sx, sw[i]);
        if (a.bias)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += bias[i];
        if (a.preact) put8(a.preact, a.preact_bf16, at, cnt, v);
        with_act(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = act_of<decltype(act)::value>(v[i]);
        });
        if (a.residual)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += res[i];
        put8(a.y, a.out_bf16, at, cnt, v);
    }
};

// ---- few tiles: every wave a part of the contraction -----------------------------
//
// A workgroup of eight waves owns 16 MB rows of x and 16 NB of w. Wave i takes the
// steps i, i + 8, ... straight from memory into the instructions' operands
// (nothing is used twice that could be shared through LDS), D - 1 of them on their way while
// one is multiplied, and the waves' sums are added through LDS in wave order. Bound by the latency of the
// first loads and the sum where rows are few (bf16 4 x 2048 x 2048 4.7 us, e4m3 256 x 2048 x 2048 9.6), in fp32 by
// the matrix instructions (4096 x 1001 x 1024 77 us, 109 of 153 TFLOP/s).
constexpr int kWaves = 8;

template <Elt T, int MB, int NB, int D, bool ODD>
__global__ __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(MB * NB == 16 && ODD ? 4 : 1))) void
gemm_split_kernel(GemmArgs a)
{
    constexpr int PITCH = NB * 16 + 4;                   // floats a row of the sums (16-byte aligned, banks apart)
    constexpr int ROUNDS = MB * NB > 4 ? 2 : 1, MR = MB / ROUNDS;   // blocks of rows a round through LDS
    static_assert(MB % ROUNDS == 0, "whole blocks of rows a round");
    __shared__ __attribute__((aligned(16))) float sums[kWaves][MR * 16 * PITCH];
    const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * (MB * 16), n0 = (int64_t)blockIdx.x * (NB * 16);
    const auto bx = buffer_at(a.x, m0 * a.ldx, a.M * a.ldx), bw = buffer_at(a.w, n0 * a.ldw, a.N * a.ldw);
    struct Frags { u4 x[MB][2], w[NB][2]; } f[D];
    // (part: whether the step may be one that ends within 128 bytes, and is then read with more care)
    auto load = [&](Frags &q, int s, auto part) GDN2_INLINE {
        const int at = s * kStep + g * 32;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (ODD && T == Elt::kF32) {
                // (fp32 rows of any length begin at whole words; the last step's are asked for one by one)
                const bool end = decltype(part)::value && (s + 1) * kStep > (int)a.kbytes;
                auto chunk = [&](const __amdgpu_buffer_rsrc_t &b, uint32_t row) GDN2_INLINE -> u4 {
                    if (!end) return __builtin_amdgcn_raw_buffer_load_b128(b, (int)(row + (uint32_t)(at + c * 16)), 0, 0);
                    u4 v;   // (behind the row's end are the next row's first words, or the buffer's zeros)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t word = __builtin_amdgcn_raw_buffer_load_b32(b, (int)(row + (uint32_t)(at + c * 16)) + i * 4, 0, 0);
                        v[i] = at + c * 16 + i * 4 < (int)a.kbytes ? word : 0u;
                    }
                    return v;
                };
#pragma unroll
                for (int j = 0; j < NB; ++j) q.w[j][c] = chunk(bw, (uint32_t)(j * 16 + r) * (uint32_t)a.ldw);
                if constexpr (decltype(part)::value) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < MB; ++i) q.x[i][c] = chunk(bx, (uint32_t)(i * 16 + r) * (uint32_t)a.ldx);
                if constexpr (decltype(part)::value) __builtin_amdgcn_sched_barrier(0);
            } else if constexpr (ODD) {
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    q.w[j][c] = load_chunk<T>((const char *)a.w + min(n0 + j * 16 + r, a.N - 1) * a.ldw, at + c * 16, a.kbytes);
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    q.x[i][c] = load_chunk<T>((const char *)a.x + min(m0 + i * 16 + r, a.M - 1) * a.ldx, at + c * 16, a.kbytes);
            } else {
                const bool in = at + c * 16 < (int)a.kbytes;
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    q.w[j][c] = __builtin_amdgcn_raw_buffer_load_b128(
                        bw, (int)(in ? (uint32_t)(j * 16 + r) * (uint32_t)a.ldw + (uint32_t)(at + c * 16) : kBeyond), 0, 0);
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    q.x[i][c] = __builtin_amdgcn_raw_buffer_load_b128(
                        bx, (int)(in ? (uint32_t)(i * 16 + r) * (uint32_t)a.ldx + (uint32_t)(at + c * 16) : kBeyond), 0, 0);
            }
        }
    };
    f4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = f4zero();
    auto multiply = [&](const Frags &q) GDN2_INLINE {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int k = 0; k < MB; ++k) acc[j][k] = Mm<T>::mma(q.w[j], q.x[k], acc[j][k]);
    };
    const int steps = (int)((a.kbytes + kStep - 1) / kStep), mine = (steps - wv + kWaves - 1) / kWaves;
    if constexpr (D == 1 && ODD && T == Elt::kF32) {
        // (a last step apart: in the loop its care would take the registers of a second workgroup a compute
        // unit. 8192 x 1001 x 1001 175 us, 211 with one.)
        const int whole = (int)(a.kbytes / kStep);
        for (int s = wv; s < whole; s += kWaves) {
            load(f[0], s, std::false_type{});
            multiply(f[0]);
        }
        if (whole < steps && whole % kWaves == wv) {
            load(f[0], whole, std::true_type{});
            multiply(f[0]);
        }
    } else {
        auto step = [&](int i) GDN2_INLINE { return wv + i * kWaves; };
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            if (d < mine) load(f[d], step(d), std::true_type{});
        for (int i = 0; i < mine; i += D)
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i + d >= mine) break;
                if (i + d + D - 1 < mine) load(f[(d + D - 1) % D], step(i + d + D - 1), std::true_type{});
                multiply(f[d]);
            }
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
                const int cnt = (int)min((int64_t)8, a.N - n);
                Finish8 fin;
                fin.load(a, m, n, cnt);
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kWaves; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f4 s = *reinterpret_cast<const f4 *>(&sums[i][row * PITCH + col + h * 4]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[h * 4 + c] += s[c];
                    }
                fin.store(a, m, n, cnt, v);
            }
        }
    }
}

// ---- many tiles -------------------------------------------------------------------

typedef float f16v __attribute__((ext_vector_type(16)));

// Products of two chunks of 32 w rows with two of 32 x rows (32 x 32 sums). Lane
// l has row l % 32 and, of 64 bytes, chunks l / 32 and 2 + l / 32.
template <Elt T> static __device__ __forceinline__ f16v mma32(const u4 (&w)[2], const u4 (&x)[2], f16v c)
{
    if constexpr (T == Elt::kBf16) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, w[j]), __builtin_bit_cast(b8, x[j]), c, 0, 0, 0);
    } else if constexpr (T == Elt::kF32) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w[j][i]), __uint_as_float(x[j][i]), c, 0, 0, 0);
    } else if constexpr (T == Elt::kE4m3Wide) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widened(w[j], h), widened(x[j], h), c, 0, 0, 0);
    } else {
        struct P { u4 a[2]; };
        const P pw = {{w[0], w[1]}}, px = {{x[0], x[1]}};
        // both e4m3, block scales 2^0
        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_bit_cast(i8v, pw), __builtin_bit_cast(i8v, px), c, 0, 0, 0,
                                                            0x7f7f7f7f, 0, 0x7f7f7f7f);
    }
    return c;
}

// Rows of 128 bytes in LDS: a fragment's rows would fall on the same banks, so
// chunk c of row r lies at position c ^ swap(r). (Rows 2 i, 2 i + 1 share one: a row is
// half as long as all banks together.)
static __device__ __forceinline__ int swap_of(int row) { return (row >> 1) & 7; }

// A workgroup of WM x WN waves owns BM rows of x and BN of w at a time, a wave 32
// MB x 32 NB sums. Each step's chunks lie in LDS, two steps' at a time, brought
// there without a register in between.
//
// A step is two halves of 64 bytes. A wave multiplies the first while it reads the
// second into registers; then (every wave has read all of the step, and its
// own part of the next one has landed) a barrier, after which the step's LDS takes the one after
// next, and the wave multiplies the second half while it reads the first of
// the next. So the matrix cores wait neither at the barrier nor for LDS, and a
// step's loads have a whole step to land.
//
// TR: the contracted axis goes down the operands' columns (a gradient's sum over rows,
// bf16 alone). A step is 64 of its rows, BM elements of each of x's and BN of w's; the bytes are the
// same. Chunk c of row k lies at position c ^ 4 (k % 4), and LDS is read by the instruction that
// hands 16 lanes the columns of 4 x 16 elements, so nothing has to be turned in memory
// before. (32 lanes read 64 bytes of each of four rows, which fall on
// different banks.)
//
// Workgroups stay and go through the tiles; the last two steps of a tile bring
// the first two of the next, so the sums' way to memory overlaps with them.
//
// 65536 x 2048 x 2048 bf16 490 us, with residual 528 (1.04 PFLOP/s); 32768 x 8192 x 2048 e4m3 to bf16 511 to 522 (2.1); by
// columns 2048 x 2048 x 32768 bf16 298 (0.92). A tile of 256 x 256 and 2048 bf16 takes 60 us of its compute unit, 37 in matrix
// instructions alone, 49 with the reads of LDS, and 49 in fetches alone (33 where the L2 has all): x comes from memory
// behind the bursts in which y leaves.

// The kernel's first argument, where it lies in memory.
static __device__ __forceinline__ GemmArgs arguments()
{
    auto p = (const __attribute__((address_space(4))) GemmArgs *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const GemmArgs *)p;
}

// The epilogue of a wave's blocks, from row mw and column nw of y on. Each 32 x 32
// block is turned through the wave's own piece of LDS, `mine`, so that four lanes have
// 32 neighbours of a row. What is read is asked for before the writes of the blocks
// before: both come back in order, and a read behind a write would wait for it.
// PART: the sums alone, to the partial sums that begin at element `part`.
template <Elt T, typename Out, bool PART, int MB, int NB>
static __device__ __forceinline__ void finish_blocks(const GemmArgs &e, int64_t part, int mw, int nw, int lane, char *mine,
                                                     const f16v (&acc)[NB][MB])
{
    constexpr int RS = sizeof(Out) / 2;   // 16-byte pieces of eight elements
    constexpr bool kScaled = T == Elt::kE4m3 || T == Elt::kE4m3Wide;
    asm volatile("" : "+v"(lane));
    const int er = lane & 31, eh = lane >> 5, c8 = (lane & 3) * 8, row = lane >> 2;
    const uint32_t N = (uint32_t)e.N;
    const int64_t at = (int64_t)mw * e.N + nw, end = e.M * e.N;
    void *dst = PART ? (void *)(e.partial + part) : e.y;
    const auto to = buffer_at(dst, at * (int)sizeof(Out), end * (int)sizeof(Out));
    const auto from = buffer_at(e.residual ? e.residual : dst, at * (int)sizeof(Out), end * (int)sizeof(Out));
    const uint32_t first = (uint32_t)row * N + c8;
    // element 8 c8 of row t of block (j, i), in bytes of `size` an element
    auto offset = [&](int j, int i, int t, int size) GDN2_INLINE {
        return (int)(nw + j * 32 + c8 < (int)N ? (first + ((i * 32 + t * 16) * N + j * 32)) * size : kBeyond);
    };
    struct Column { u4 s[2], b[2]; } col[2];
    u4 old[2][2][RS];   // [block % 2][t]
    float sx[MB][2];
    auto ahead = [&](int b) GDN2_INLINE {
        const int j = b / MB, i = b % MB;
        if (i == 0) {
            if (e.sw) {
                const auto p = buffer_at(e.sw, (int64_t)nw * 4, e.N * 4);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    col[j & 1].s[k] = __builtin_amdgcn_raw_buffer_load_b128(p, (j * 32 + c8 + k * 4) * 4, 0, 0);
            }
            if (e.bias) {
                const auto p = buffer_at(e.bias, (int64_t)nw * 4, e.N * 4);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    col[j & 1].b[k] = __builtin_amdgcn_raw_buffer_load_b128(p, (j * 32 + c8 + k * 4) * 4, 0, 0);
            }
        }
        if (e.residual)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int k = 0; k < RS; ++k)
                    old[b & 1][t][k] = __builtin_amdgcn_raw_buffer_load_b128(from, offset(j, i, t, sizeof(Out)) + k * 16, 0, 0);
    };
    if constexpr (!PART) {
        if (e.sw) {
            const auto p = buffer_at(e.sx, (int64_t)mw * 4, e.M * 4);
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    sx[i][t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(p, (i * 32 + t * 16 + row) * 4, 0, 0));
        }
        ahead(0);
    }
#pragma unroll
    for (int b = 0; b < NB * MB; ++b) {
        const int j = b / MB, i = b % MB;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<f4 *>(mine + er * 128 + (((c * 2 + eh) ^ swap_of(er)) << 4)) =
                (f4){acc[j][i][c * 4], acc[j][i][c * 4 + 1], acc[j][i][c * 4 + 2], acc[j][i][c * 4 + 3]};
        if (!PART && b + 1 < NB * MB) ahead(b + 1);
        __builtin_amdgcn_wave_barrier();
        float v[2][8];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f4 x = *reinterpret_cast<const f4 *>(mine + (t * 16 + row) * 128 +
                                                           ((((lane & 3) * 2 + k) ^ swap_of(t * 16 + row)) << 4));
#pragma unroll
                for (int c = 0; c < 4; ++c) v[t][k * 4 + c] = x[c];
            }
        __builtin_amdgcn_wave_barrier();
        auto store = [&](__amdgpu_buffer_rsrc_t p, auto type) GDN2_INLINE {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int o = offset(j, i, t, sizeof(type));
                if constexpr (sizeof(type) == 2) {
                    const u4 x = {bf16x2(v[t][0], v[t][1]), bf16x2(v[t][2], v[t][3]), bf16x2(v[t][4], v[t][5]), bf16x2(v[t][6], v[t][7])};
                    __builtin_amdgcn_raw_buffer_store_b128(x, p, o, 0, kOnce);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const f4 x = {v[t][k * 4], v[t][k * 4 + 1], v[t][k * 4 + 2], v[t][k * 4 + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), p, o + k * 16, 0, PART ? 0 : kOnce);
                    }
                }
            }
        };
        if constexpr (!PART) {
            const Column &q = col[j & 1];
            if (e.sw)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[t][c] = scaled(v[t][c], sx[i][t], __uint_as_float(q.s[c >> 2][c & 3]));
            if (e.bias)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[t][c] += __uint_as_float(q.b[c >> 2][c & 3]);
            if constexpr (!kScaled)
                if (e.preact) {
                    using Z = std::conditional_t<T == Elt::kBf16, uint16_t, float>;
                    store(buffer_at(e.preact, at * (int)sizeof(Z), end * (int)sizeof(Z)), Z(0));
                }
            with_act(e.act, [&](auto act) GDN2_INLINE {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[t][c] = act_of<decltype(act)::value>(v[t][c]);
            });
            if (e.residual)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const u4 (&o)[RS] = old[b & 1][t];
                        v[t][c] += sizeof(Out) == 4 ? __uint_as_float(o[(c >> 2) % RS][c & 3])
                                   : c & 1          ? __uint_as_float(o[0][c >> 1] & 0xFFFF0000u)
                                                    : __uint_as_float(o[0][c >> 1] << 16);
                    }
        }
        store(to, Out(0));
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Waits for what this wave has under way from memory to LDS (a barrier alone does not).
static __device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <Elt T, int BM, int BN, int WM, int WN, bool TR>
__global__ __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(2))) void gemm_tile_kernel(GemmArgs a, int tm,
                                                                                                       int tn)
{
    constexpr int NW = WM * WN, MB = BM / WM / 32, NB = BN / WN / 32;
    constexpr int RX = BM / 8 / NW, RW = BN / 8 / NW;                   // groups of 8 rows each wave brings
    constexpr int BUF = (BM + BN) * kStep;
    static_assert(RX * 8 * NW == BM && RW * 8 * NW == BN && NW % 2 == 0, "whole groups a wave, in one half of 16 rows");
    static_assert(!TR || (T == Elt::kBf16 && BM >= 128 && BN >= 128 && MB * 32 == 64), "rows of 16 chunks and more, read 16 bits a time");
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF + NW * 4096];
    const int lane = threadIdx.x & 63, wv = wave_id();
    const int wm = wv % WM, wn = wv / WM;
    const int steps = (int)((a.kbytes + kStep - 1) / kStep);

    // Units (tiles of each part of the contraction) in an order that gives
    // neighbouring ones to one XCD (workgroups go round the eight of them)
    const int all = tm * tn * a.splits, xcd = blockIdx.x & 7, stride = gridDim.x >> 3;
    const int first = uniform(xcd * (all >> 3) + min(xcd, all & 7)), count = (all >> 3) + (xcd < (all & 7) ? 1 : 0);
    struct Unit { int m0, n0, part, s0, s1; };
    auto unit_of = [&](int j) GDN2_INLINE {
        const int u = first + j, tiles = tm * tn, part = a.splits > 1 ? u / tiles : 0, tile = u - part * tiles;
        // bands of four tiles of x
        const int band = tile / (4 * tn), inb = tile - band * 4 * tn, bm = min(4, tm - band * 4), col = inb / bm;
        return Unit{uniform((band * 4 + inb - col * bm) * BM), uniform(col * BN), uniform(part),
                    uniform((int)((unsigned)steps * part / a.splits)), uniform((int)((unsigned)steps * (part + 1) / a.splits))};
    };

    // What a lane brings: of every NW-th group of 8 rows, row lane / 8 and the
    // chunk that belongs at position lane % 8. Reads go through buffer descriptors that
    // end with the operand, and what lies beyond an end arrives as zeros: rows behind the
    // last one, and chunks behind a row's end, whose offset is made too large.
    // TR: of every NW-th KB of 1 KB pieces, each a few of the step's rows.
    constexpr int CX = BM / 8, CW = BN / 8;   // TR: chunks of a step's row
    const uint32_t gx = (uint32_t)(NW * (TR ? 64 / CX : 8)) * (uint32_t)a.ldx, gw = (uint32_t)(NW * (TR ? 64 / CW : 8)) * (uint32_t)a.ldw;
    uint32_t vx, vw;               // bytes from the step's first
    int cof, ox, ow;               // its chunk in a row; in LDS: this lane's rows of x and w, at its chunk
    auto place = [&]() GDN2_INLINE {
        // (lane from where the compiler cannot see it, here and in the epilogue: what is made
        // of it would otherwise be kept in registers through both)
        int l = lane;
        asm volatile("" : "+v"(l));
        if constexpr (TR) {
            const int rx = wv * (64 / CX) + l / CX, rw = wv * (64 / CW) + l / CW;
            vx = (uint32_t)rx * (uint32_t)a.ldx + ((l % CX) ^ (4 * (rx & 3))) * 16;
            vw = (uint32_t)rw * (uint32_t)a.ldw + ((l % CW) ^ (4 * (rw & 3))) * 16;
            cof = 0;
            // lane t of 16 reads 8 bytes of row t / 4 and is given column t; 32 columns by the half wave, rows
            // 8 (l / 32) and on by the halves. A block's chunks differ from the first's by xor.
            const int t = l & 15, k = 8 * (l >> 5) + t / 4, c = (l >> 4 & 1) * 2 + (t & 3) / 2, b = (t & 1) * 8;
            const int cx = wm * (BM / WM / 8) + c, cw = wn * (BN / WN / 8) + c;
            ox = k * (BM * 2) + (cx ^ (4 * (t / 4))) * 16 + b;
            ow = BM * kStep + k * (BN * 2) + (cw ^ (4 * (t / 4))) * 16 + b;
            return;
        }
        const int grow = l >> 3;
        cof = ((l & 7) ^ swap_of((wv & 1) * 8 + grow)) * 16;
        vx = (uint32_t)(wv * 8 + grow) * (uint32_t)a.ldx + cof;
        vw = (uint32_t)(wv * 8 + grow) * (uint32_t)a.ldw + cof;
        // its chunks of a half: half * 4 + h and two further on; their positions differ by xor
        const int r = l & 31, pos = ((l >> 5) ^ swap_of(r)) << 4;
        ox = (wm * (BM / WM) + r) * kStep + pos;
        ow = (BM + wn * (BN / WN) + r) * kStep + pos;
    };
    int64_t atx = 0, atw = 0;      // the unit's first rows, and the step in them
    int jf = uniform(blockIdx.x >> 3), fs = 0, fs1 = 0;   // the next step to bring: unit, step, the unit's end
    auto aim = [&]() GDN2_INLINE {
        if (jf >= count) return;
        const Unit q = unit_of(jf);
        fs = q.s0;
        fs1 = q.s1;
        atx = TR ? q.m0 * 2 + (int64_t)fs * (64 * a.ldx) : q.m0 * a.ldx + (int64_t)fs * kStep;
        atw = TR ? q.n0 * 2 + (int64_t)fs * (64 * a.ldw) : q.n0 * a.ldw + (int64_t)fs * kStep;
    };
    auto fetch = [&](char *buf) GDN2_INLINE {
        if (jf >= count) return;
        const bool in = TR || fs * kStep + cof < (int)a.kbytes;
        const auto bx = buffer_at(a.x, atx, (TR ? a.kbytes / 2 : a.M) * a.ldx), bw = buffer_at(a.w, atw, (TR ? a.kbytes / 2 : a.N) * a.ldw);
        auto bring = [&](__amdgpu_buffer_rsrc_t from, uint32_t v, char *to) GDN2_INLINE {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16,
                                                     (int)(in ? v : kBeyond), 0, 0, 0);
        };
#pragma unroll
        for (int i = 0; i < RX; ++i) bring(bx, vx + i * gx, buf + (i * NW + wv) * 1024);
#pragma unroll
        for (int i = 0; i < RW; ++i) bring(bw, vw + i * gw, buf + BM * kStep + (i * NW + wv) * 1024);
        atx += TR ? 64 * a.ldx : kStep;
        atw += TR ? 64 * a.ldw : kStep;
        if (++fs == fs1) {
            jf += stride;
            aim();
        }
    };

    // A step's products in phases: half of its bytes, two of the wave's blocks of w. The
    // operands of the next phase are read while one is multiplied.
    constexpr int NP = NB / 2, PH = 2 * NP;
    u4 fw[2][2][2], fx[2][MB][2];   // [phase or half % 2][block][chunk]
    auto read = [&](const char *buf, auto phase) GDN2_INLINE {
        constexpr int P = decltype(phase)::value, H = P / NP, J = P % NP * 2;
        if constexpr (TR) {
            // 16 of the step's rows: the columns of a block of 32, four rows of a lane's eight at a time
            auto columns = [&](int at, int block, int pitch, int rows) GDN2_INLINE {
                typedef short s4 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) s4 lds4;
                struct P { s4 a[2]; } p;
                p.a[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(buf + rows * pitch + (at ^ (block * 64))));
                p.a[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(buf + (rows + 4) * pitch + (at ^ (block * 64))));
                return __builtin_bit_cast(u4, p);
            };
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int j = 0; j < 2; ++j) fw[P & 1][j][c] = columns(ow, J + j, BN * 2, H * 32 + c * 16);
                if constexpr (J == 0)
#pragma unroll
                    for (int i = 0; i < MB; ++i) fx[H][i][c] = columns(ox, i, BM * 2, H * 32 + c * 16);
            }
            return;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fw[P & 1][j][c] = *reinterpret_cast<const u4 *>(buf + (J + j) * 32 * kStep + (ow ^ (H * 64 + c * 32)));
            if constexpr (J == 0)
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    fx[H][i][c] = *reinterpret_cast<const u4 *>(buf + i * 32 * kStep + (ox ^ (H * 64 + c * 32)));
        }
    };
    f16v acc[NB][MB];
    auto multiply = [&](auto phase) GDN2_INLINE {
        constexpr int P = decltype(phase)::value, H = P / NP, J = P % NP * 2;
        __builtin_amdgcn_sched_barrier(0);   // the next phase's operands first, ...
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[J + j][i] = mma32<T>(fw[P & 1][j], fx[H][i], acc[J + j][i]);
        __builtin_amdgcn_sched_barrier(0);   // ... but not those of the one after
    };
    using p0 = std::integral_constant<int, 0>;
    using last = std::integral_constant<int, PH - 1>;

    int jc = jf, odd = 0;   // the unit in hand; which buffer its step is in
    if (jc >= count) return;
    aim();
    place();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) fetch(lds + i * BUF);
    landed();
    __syncthreads();
    for (; jc < count; jc += stride) {
        const Unit q = unit_of(jc);
        place();
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[j][i][c] = 0.f;
        read(lds + odd * BUF, p0{});
        for (int s = q.s0; s < q.s1; ++s) {
            const char *cur = lds + odd * BUF;
            if constexpr (NP == 2) {
                read(cur, std::integral_constant<int, 1>{});
                multiply(p0{});
                read(cur, std::integral_constant<int, 2>{});
                multiply(std::integral_constant<int, 1>{});
                read(cur, last{});
                multiply(std::integral_constant<int, 2>{});
            } else {
                read(cur, last{});
                multiply(p0{});
            }
            // (not to be moved behind the barrier and the branches that follow)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < MB; ++i) asm volatile("" : "+v"(acc[j][i]));
            landed();
            __syncthreads();
            fetch(lds + odd * BUF);
            odd ^= 1;
            // (behind a tile's last step: read once more below)
            read(lds + odd * BUF, p0{});
            multiply(last{});
        }

        // The epilogue, block by block. The arguments come from memory anew: kept in
        // registers they would be in the way above.
        const GemmArgs e = arguments();
        const int mw = q.m0 + wm * (BM / WM), nw = q.n0 + wn * (BN / WN);
        if (mw >= e.M || nw >= e.N) continue;
        char *mine = lds + 2 * BUF + wv * 4096;
        // (e4m3 has the type of y in its own, and no parts)
        if constexpr (T == Elt::kE4m3) {
            finish_blocks<T, uint16_t, false, MB, NB>(e, 0, mw, nw, lane, mine, acc);
        } else if constexpr (T == Elt::kE4m3Wide) {
            finish_blocks<T, float, false, MB, NB>(e, 0, mw, nw, lane, mine, acc);
        } else if (e.splits > 1) {
            finish_blocks<T, float, true, MB, NB>(e, (int64_t)q.part * e.M * e.N, mw, nw, lane, mine, acc);
        } else if (e.out_bf16) {
            finish_blocks<T, uint16_t, false, MB, NB>(e, 0, mw, nw, lane, mine, acc);
        } else {
            finish_blocks<T, float, false, MB, NB>(e, 0, mw, nw, lane, mine, acc);
        }
    }
}

// The same with rows that do not begin at whole chunks or end with them: chunks go
// through registers, tiles of 128 x 128, 16 x 16 sums an instruction. Bound by the loads, which come from any
// byte (bf16 5000 x 2001 x 2047: 105 us, 0.39 PFLOP/s; 1000 x 2001 x 2047 50 us, 115 in blocks of the waves that
// share the contraction; 256 x 2001 x 2047 38 and 44, x 501 17 and 13).
template <Elt T> __global__ __launch_bounds__(256) void gemm_odd_kernel(GemmArgs a, int tm, int tn)
{
    constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
    constexpr int NW = WM * WN, MB = BM / WM / 16, NB = BN / WN / 16;
    constexpr int RX = BM / 8 / NW, RW = BN / 8 / NW;
    constexpr int BUF = (BM + BN) * kStep;
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF + 16 * (BM / 2)];   // (the sums' rows are a little longer)
    const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
    const int band = blockIdx.x / (4 * tn), inb = blockIdx.x % (4 * tn), bm = min(4, tm - band * 4);
    const int64_t m0 = (int64_t)(band * 4 + inb % bm) * BM, n0 = (int64_t)(inb / bm) * BN;
    const int grow = lane >> 3, cof = ((lane & 7) ^ swap_of((wv & 1) * 8 + grow)) * 16;
    const char *px[RX], *pw[RW];
#pragma unroll
    for (int i = 0; i < RX; ++i) px[i] = (const char *)a.x + min(m0 + (i * NW + wv) * 8 + grow, a.M - 1) * a.ldx;
#pragma unroll
    for (int i = 0; i < RW; ++i) pw[i] = (const char *)a.w + min(n0 + (i * NW + wv) * 8 + grow, a.N - 1) * a.ldw;
    const int steps = (int)((a.kbytes + kStep - 1) / kStep);

    u4 staged[RX + RW];
    auto fetch = [&](int s) {
        const int64_t k = (int64_t)s * kStep + cof;
#pragma unroll
        for (int i = 0; i < RX; ++i) staged[i] = load_chunk<T>(px[i], k, a.kbytes);
#pragma unroll
        for (int i = 0; i < RW; ++i) staged[RX + i] = load_chunk<T>(pw[i], k, a.kbytes);
    };
    auto settle = [&](char *buf) {
#pragma unroll
        for (int i = 0; i < RX; ++i) *reinterpret_cast<u4 *>(buf + (i * NW + wv) * 1024 + lane * 16) = staged[i];
#pragma unroll
        for (int i = 0; i < RW; ++i)
            *reinterpret_cast<u4 *>(buf + BM * kStep + (i * NW + wv) * 1024 + lane * 16) = staged[RX + i];
    };
    f4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = f4zero();
    const int wm = wv % WM, wn = wv / WM;
    // chunk g of this lane's row of a block; chunk g + 4 is at the same place ^ 64
    const int pos = (g ^ swap_of(r)) << 4;
    const int ox = (wm * (BM / WM) + r) * kStep + pos, ow = (BM + wn * (BN / WN) + r) * kStep + pos;
    fetch(0);
    settle(lds);
    for (int s = 0; s < steps; ++s) {
        char *cur = lds + (s & 1) * BUF, *next = lds + ((s + 1) & 1) * BUF;
        __syncthreads();
        if (s + 1 < steps) fetch(s + 1);
        u4 fw[NB][2];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) fw[j][c] = *reinterpret_cast<const u4 *>(cur + j * 16 * kStep + (ow ^ (64 * c)));
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            u4 fx[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) fx[c] = *reinterpret_cast<const u4 *>(cur + i * 16 * kStep + (ox ^ (64 * c)));
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[j][i] = Mm<T>::mma(fw[j], fx, acc[j][i]);
        }
        if (s + 1 < steps) settle(next);
    }
    // the sums through LDS, half of each wave's rows a round, eight neighbours a lane
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
                *reinterpret_cast<f4 *>(&sums[(wm * kRows + i * 16 + r) * PITCH + wn * (BN / WN) + j * 16 + g * 4]) =
                    acc[j][q * (MB / 2) + i];
        __syncthreads();
        const int col = threadIdx.x % TPR * 8;
        const int64_t n = n0 + col;
        if (n < a.N) {
            const int cnt = (int)min((int64_t)8, a.N - n);
            for (int row = threadIdx.x / TPR; row < WM * kRows; row += NW * 64 / TPR) {
                const int64_t m = m0 + row / kRows * (BM / WM) + q * kRows + row % kRows;
                if (m >= a.M) continue;
                Finish8 fin;
                fin.load(a, m, n, cnt);
                float v[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const f4 x = *reinterpret_cast<const f4 *>(&sums[row * PITCH + col + e * 4]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[e * 4 + c] = x[c];
                }
                fin.store(a, m, n, cnt, v);
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
    Finish8 fin;
    fin.load(a, m, n, cnt);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) {
        float x[8];
        get8(a.partial + ((int64_t)s * a.M + m) * a.ldp + n, cnt, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += x[c];
    }
    fin.store(a, m, n, cnt, v);
}

// ---- launch -------------------------------------------------------------------------

template <Elt T, bool ODD> static hipError_t launch_gemm_forms(const GemmArgs &a, hipStream_t st)
{
    auto tiles = [](int64_t rows, int b) { return (rows + b - 1) / b; };
    auto split = [&](auto mb, auto nb, auto d) {
        constexpr int MB = decltype(mb)::value, NB = decltype(nb)::value, D = decltype(d)::value;
        hipLaunchKernelGGL((gemm_split_kernel<T, MB, NB, D, ODD>), dim3((unsigned)tiles(a.N, NB * 16), (unsigned)tiles(a.M, MB * 16)),
                           dim3(kWaves * 64), 0, st, a);
        return hipGetLastError();
    };
    auto tiled = [&](auto bm, auto bn, auto wm, auto wn) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
        const int64_t tm = tiles(a.M, BM), tn = tiles(a.N, BN);
        if (tm * tn > 0x7fffffLL) return hipErrorInvalidConfiguration;
        // as many workgroups as there is room for (one or two a compute unit), a multiple of the XCDs'
        const int64_t grid = std::min<int64_t>((tm * tn * a.splits + 7) / 8 * 8, WM * WN == 8 ? 256 : 512);
        auto run = [&](auto elt) {
            hipLaunchKernelGGL((gemm_tile_kernel<decltype(elt)::value, BM, BN, WM, WN, false>), dim3((unsigned)grid), dim3(WM * WN * 64), 0,
                               st, a, (int)tm, (int)tn);
        };
        if constexpr (T == Elt::kE4m3) {
            if (!a.out_bf16) {
                run(std::integral_constant<Elt, Elt::kE4m3Wide>{});
                return hipGetLastError();
            }
        }
        run(std::integral_constant<Elt, T>{});
        return hipGetLastError();
    };
    using i1 = std::integral_constant<int, 1>;
    using i2 = std::integral_constant<int, 2>;
    using i4 = std::integral_constant<int, 4>;
    using i64 = std::integral_constant<int, 64>;
    using i128 = std::integral_constant<int, 128>;
    using i256 = std::integral_constant<int, 256>;
    constexpr bool kSlow = T == Elt::kF32;
    const bool whole = !ODD && a.N % 8 == 0;
    // The smallest blocks of the waves that share the contraction, if they give no compute unit
    // a second workgroup: the chip is as full as it can be, and most loads are under way (bf16, K =
    // 2048, us in blocks of 16 x 16, 16 x 32, 32 x 32, 32 x 64: 32 x 2048 6.3, 7.7, 9.5, 14.0; 64 x 2048 9.8, 7.8,
    // 9.5, 14.0; 32 x 8192 16.8, 13.0, 9.9, 14.4; 64 x 8192 30.6, 23.4, 17.7, 14.7, and 20 in tiles). fp32
    // takes some workgroups more: half the compute units would have none of the next size.
    if (a.splits == 1) {
        auto blocks = [&](int rows, int cols) { return tiles(a.M, rows) * tiles(a.N, cols); };
        if (blocks(16, 16) <= 256) return split(i1{}, i1{}, i4{});
        if (blocks(16, 32) <= 256) return split(i1{}, i2{}, i4{});
        if (blocks(32, 32) <= 256) return split(i2{}, i2{}, i4{});
        if (blocks(32, 64) <= (kSlow ? 384 : 256)) return split(i2{}, i4{}, std::conditional_t<kSlow, i1, i2>{});
    }
    // Rows that LDS can take whole chunks of, and y in whole eights: tiles, the larger ones where they
    // fill the chip (bf16, K = N = 2048: 1024 rows 18 us in tiles of 128 x 64, 35 in blocks
    // of the waves that share the contraction; 4096 rows 35 us in 128 x 128, 46 in 128 x 64; 512 rows 16 and 18).
    if (whole && tiles(a.M, 256) * tiles(a.N, 256) * a.splits >= 192) return tiled(i256{}, i256{}, i4{}, i2{});
    if (whole && tiles(a.M, 128) * tiles(a.N, 128) * a.splits >= (kSlow ? 512 : 256)) return tiled(i128{}, i128{}, i2{}, i2{});
    if (whole && (a.splits > 1 || (!kSlow && tiles(a.M, 128) * tiles(a.N, 64) >= 128))) return tiled(i128{}, i64{}, i4{}, i1{});
    // fp32's matrix instructions take so long that one step ahead is enough, and that operands
    // from the L2 keep up with them: small blocks, which leave no compute unit idle at the end, are used far longer
    // (1024^3: 23 us, 25 with a step ahead, 39 in tiles).
    if constexpr (kSlow)
        if (tiles(a.M, 64) <= 65535 && tiles(a.M, 64) * tiles(a.N, 64) <= 0x7fffffLL) return split(i4{}, i4{}, i1{});
    const int64_t tm = tiles(a.M, 128), tn = tiles(a.N, 128);
    if (tm * tn > 0x7fffffLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(gemm_odd_kernel<T>, dim3((unsigned)(tm * tn)), dim3(256), 0, st, a, (int)tm, (int)tn);
    return hipGetLastError();
}

template <Elt T> static hipError_t launch_gemm_type(const GemmArgs &a, hipStream_t st)
{
    if (a.splits == 1) {
        const bool odd = a.ldx % 16 || a.ldw % 16 || a.kbytes % 16;
        return odd ? launch_gemm_forms<T, true>(a, st) : launch_gemm_forms<T, false>(a, st);
    }
    const int64_t blocks = (a.M * ((a.N + 7) / 8) + 255) / 256;
    if (blocks > 0xffffffLL || a.ldp % 8 || a.ldp < a.N) return hipErrorInvalidConfiguration;
    GemmArgs part = a;
    part.N = a.ldp;
    const hipError_t err = launch_gemm_forms<T, false>(part, st);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(gemm_join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn2
