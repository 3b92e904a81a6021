// Row-wise helpers of the kernels around the mixer (layer norm, prologue):
// packed loads and stores of V consecutive elements, and sums over the lanes
// that share a row.
#pragma once

#include "gdn2_device.hpp"

namespace gdn2 {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// V consecutive elements as they lie in memory, kept packed until use (the
// loads of a row are issued together). V = 8 needs 16-byte alignment.
template <typename In, int V> struct Pack;
template <> struct Pack<uint16_t, 8> {
    u4 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const u4 *>(p); }
    __device__ __forceinline__ void load_nt(const uint16_t *p) { r = __builtin_nontemporal_load(reinterpret_cast<const u4 *>(p)); }
    __device__ __forceinline__ float get(int i) const
    {
        return __uint_as_float((i & 1) ? (r[i >> 1] & 0xFFFF0000u) : (r[i >> 1] << 16));
    }
    __device__ __forceinline__ void zero() { r = (u4){0u, 0u, 0u, 0u}; }
};
template <> struct Pack<float, 8> {
    f4 r[2];
    __device__ __forceinline__ void load(const float *p)
    {
        r[0] = reinterpret_cast<const f4 *>(p)[0];
        r[1] = reinterpret_cast<const f4 *>(p)[1];
    }
    __device__ __forceinline__ void load_nt(const float *p)
    {
        r[0] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(p));
        r[1] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(p) + 1);
    }
    __device__ __forceinline__ float get(int i) const { return r[i >> 2][i & 3]; }
    __device__ __forceinline__ void zero() { r[0] = r[1] = f4zero(); }
};
template <typename In> struct Pack<In, 1> {
    In r;
    __device__ __forceinline__ void load(const In *p) { r = *p; }
    __device__ __forceinline__ void load_nt(const In *p) { r = __builtin_nontemporal_load(p); }
    __device__ __forceinline__ float get(int) const { return in2f<In>(r); }
    __device__ __forceinline__ void zero() { r = (In)0; }
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

// V floats to memory in the output type
template <int V, bool NT = false> __device__ __forceinline__ void store_row(float *p, const float *x)
{
    if constexpr (V == 8) {
        f4 a = {x[0], x[1], x[2], x[3]}, b = {x[4], x[5], x[6], x[7]};
        if constexpr (NT) {
            __builtin_nontemporal_store(a, reinterpret_cast<f4 *>(p));
            __builtin_nontemporal_store(b, reinterpret_cast<f4 *>(p) + 1);
        } else {
            reinterpret_cast<f4 *>(p)[0] = a;
            reinterpret_cast<f4 *>(p)[1] = b;
        }
    } else {
        *p = *x;
    }
}
template <int V, bool NT = false> __device__ __forceinline__ void store_row(uint16_t *p, const float *x)
{
    if constexpr (V == 8) {
        u4 r = {bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7])};
        if constexpr (NT) __builtin_nontemporal_store(r, reinterpret_cast<u4 *>(p));
        else *reinterpret_cast<u4 *>(p) = r;
    } else {
        *p = __builtin_bit_cast(uint16_t, (__bf16)*x);
    }
}

// four floats to memory in the output type
__device__ __forceinline__ void store_row4(float *p, const float *x)
{
    f4 a = {x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f4 *>(p) = a;
}
__device__ __forceinline__ void store_row4(uint16_t *p, const float *x)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}

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
