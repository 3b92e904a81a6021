// Row-wise helpers of the kernels around the mixer (layer norm, prologue, the
// recurrence): packed loads and stores of consecutive elements, and sums over
// the lanes that share a row.
#pragma once

#include "gdn2_device.hpp"

namespace gdn2 {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// Eight consecutive elements as they lie in memory, kept packed until use (the
// loads of a row are issued together), NT: past the caches. AL: the address is a
// multiple of 16 bytes; otherwise it is that of any element (the memory pipe
// takes a 16-byte load at any).
typedef u4 u4_any __attribute__((aligned(2)));
typedef f4 f4_any __attribute__((aligned(4)));

template <typename In> struct Pack8;
template <> struct Pack8<uint16_t> {
    u4 r;
    template <bool AL, bool NT> __device__ __forceinline__ void load(const uint16_t *p)
    {
        if constexpr (AL && NT) r = __builtin_nontemporal_load(reinterpret_cast<const u4 *>(p));
        else if constexpr (AL) r = *reinterpret_cast<const u4 *>(p);
        else if constexpr (NT) r = __builtin_nontemporal_load(reinterpret_cast<const u4_any *>(p));
        else r = *reinterpret_cast<const u4_any *>(p);
    }
    // the first n elements, zeros behind them
    __device__ __forceinline__ void load_some(const uint16_t *p, int n)
    {
        zero();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) r[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
    __device__ __forceinline__ float get(int i) const
    {
        return __uint_as_float((i & 1) ? (r[i >> 1] & 0xFFFF0000u) : (r[i >> 1] << 16));
    }
    __device__ __forceinline__ void zero() { r = (u4){0u, 0u, 0u, 0u}; }
};
template <> struct Pack8<float> {
    f4 r[2];
    template <bool AL, bool NT> __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (AL && NT) r[i] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(p) + i);
            else if constexpr (AL) r[i] = reinterpret_cast<const f4 *>(p)[i];
            else if constexpr (NT) r[i] = __builtin_nontemporal_load(reinterpret_cast<const f4_any *>(p) + i);
            else r[i] = reinterpret_cast<const f4_any *>(p)[i];
        }
    }
    __device__ __forceinline__ void load_some(const float *p, int n)
    {
        zero();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) r[i >> 2][i & 3] = p[i];
    }
    __device__ __forceinline__ float get(int i) const { return r[i >> 2][i & 3]; }
    __device__ __forceinline__ void zero() { r[0] = r[1] = f4zero(); }
};

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

// two floats to bf16, to nearest even (one conversion instruction)
__device__ __forceinline__ uint32_t bf16x2(float a, float b)
{
    bf2 x;
    x[0] = (__bf16)a;
    x[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, x);
}

__device__ __forceinline__ uint16_t bf16_of(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

// Eight floats to memory in the output type, past the caches; AL as in
// Pack8::load.
template <bool AL> __device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    const f4 a = {x[0], x[1], x[2], x[3]}, b = {x[4], x[5], x[6], x[7]};
    if constexpr (AL) {
        __builtin_nontemporal_store(a, reinterpret_cast<f4 *>(p));
        __builtin_nontemporal_store(b, reinterpret_cast<f4 *>(p) + 1);
    } else {
        __builtin_nontemporal_store(a, reinterpret_cast<f4_any *>(p));
        __builtin_nontemporal_store(b, reinterpret_cast<f4_any *>(p) + 1);
    }
}
template <bool AL> __device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8])
{
    const u4 r = {bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7])};
    if constexpr (AL) __builtin_nontemporal_store(r, reinterpret_cast<u4 *>(p));
    else __builtin_nontemporal_store(r, reinterpret_cast<u4_any *>(p));
}
// one float
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t *p, float x) { *p = bf16_of(x); }

// Sum over the TPR threads that share a row, in each of them: TPR <= 64 lanes
// of a wave, or all TPR threads of a workgroup through `red` (TPR / 64 floats
// per value, and a barrier pair). Every thread of the workgroup calls it.
template <int TPR, int NV> __device__ __forceinline__ void row_sums(float (&x)[NV], float *red)
{
    if constexpr (TPR <= 64) {
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = lane_group_sum<TPR>(x[j]);
    } else {
        constexpr int NW = TPR / 64;
        const int wv = wave_id();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j] = lane_group_sum<64>(x[j]);
            if ((threadIdx.x & 63) == 0) red[j * NW + wv] = x[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) s += red[j * NW + i];
            x[j] = s;
        }
        __syncthreads();
    }
}

} // namespace gdn2
