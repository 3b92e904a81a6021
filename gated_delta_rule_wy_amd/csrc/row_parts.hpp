// How the row norms (layer_norm.hip, rms_norm.hip) hold a row in registers: the
// threads that share it, the packs of eight elements each of them has, and the
// choice of both from the row's length.
#pragma once

#include "rows.hpp"

#include <algorithm>

namespace gdn2 {

// Largest of x >= 0 over the TPR threads that share a row, in each of them; `red`
// and callers as in row_sums. (NaN counts as 0.)
template <int TPR> __device__ __forceinline__ float row_max(float x, float *red)
{
    auto dpp = [](float v, auto ctrl, auto rows) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value,
                                                          decltype(rows)::value, 0xF, false));
    };
    using all = std::integral_constant<int, 0xF>;
    constexpr int G = TPR < 64 ? TPR : 64;
    // (the steps of lane_group_sum; rows that a broadcast leaves out get 0)
    x = fmaxf(x, dpp(x, std::integral_constant<int, 0xB1>{}, all{}));
    x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4E>{}, all{}));
    x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}, all{}));
    if constexpr (G >= 16) x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}, all{}));
    if constexpr (G >= 32) x = fmaxf(x, dpp(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{}));
    if constexpr (G == 32) {
        const float lo = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 31));
        const float hi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
        x = (__lane_id() < 32) ? lo : hi;
    }
    if constexpr (G == 64) {
        x = fmaxf(x, dpp(x, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{}));
        x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
    }
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[wave_id()] = x;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) x = fmaxf(x, red[i]);
        __syncthreads();
    }
    return x;
}

// Eight floats (one float) to memory as e4m3, to nearest even; |x| < 464. AL: the
// address is a multiple of 8 bytes.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef u2 u2_any __attribute__((aligned(1)));
template <bool AL> __device__ __forceinline__ void store8(uint8_t *p, const float (&x)[8])
{
    const u2 r = {e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7])};
    if constexpr (AL) __builtin_nontemporal_store(r, reinterpret_cast<u2 *>(p));
    else __builtin_nontemporal_store(r, reinterpret_cast<u2_any *>(p));
}
__device__ __forceinline__ void store1(uint8_t *p, float x) { *p = (uint8_t)e4m3x4(x, 0.f, 0.f, 0.f); }

template <int TPR> struct RowShape {
    static constexpr int NT = TPR > 256 ? TPR : 256;   // threads
    static constexpr int RPB = NT / TPR;               // rows of a workgroup
};

// How a row of `cols` elements falls into packs of eight: in whole ones; or
// the last pack reaches back over its neighbour's elements, so that no lane
// loads element by element; or the row is shorter than a pack.
enum class Packs { kWhole, kOdd, kFew };

// What a lane holds: pack e of thread p of a row, elements at(e) .. at(e) + 7.
// mine(e, i): element i counts here (a row's sums take each element once; what
// a lane holds twice it computes and stores twice, with the same bits).
template <int TPR, Packs P> struct RowPart {
    int p, cols;
    __device__ __forceinline__ int col(int e) const { return (p + e * TPR) * 8; }
    __device__ __forceinline__ bool any(int e) const { return col(e) < cols; }
    __device__ __forceinline__ int at(int e) const { return P == Packs::kOdd ? min(col(e), cols - 8) : col(e); }
    __device__ __forceinline__ bool mine(int e, int i) const
    {
        if (P == Packs::kWhole) return any(e);
        if (P == Packs::kOdd) return at(e) + i >= col(e);
        return col(e) + i < cols;
    }
    template <bool NT = true, typename T> __device__ __forceinline__ void load(Pack8<T> &x, const T *row, int e) const
    {
        if constexpr (P == Packs::kOdd) {
            x.template load<false, NT>(row + at(e));
        } else if constexpr (P == Packs::kWhole) {
            x.zero();
            if (any(e)) x.template load<true, NT>(row + col(e));
        } else {
            x.load_some(row + col(e), cols - col(e));
        }
    }
    // its own elements, zeros for others (in whole and few packs those are zeros as loaded)
    __device__ __forceinline__ float own(float v, int e, int i) const
    {
        return P == Packs::kOdd && !mine(e, i) ? 0.f : v;
    }
    template <typename T> __device__ __forceinline__ void store(T *row, const float (&x)[8], int e) const
    {
        if (!any(e)) return;
        if constexpr (P == Packs::kFew) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (mine(e, i)) store1(row + col(e) + i, x[i]);
        } else {
            store8<P == Packs::kWhole>(row + at(e), x);
        }
    }
};

// Calls f with the (packs, TPR, E) that hold a row of `cols` elements in
// registers, or returns false (the long-row kernels take it). A wave a row as
// long as its registers hold one (2048 elements; 65536 x 2048 bf16 backward:
// 137 us, 222 with a workgroup a row).
template <Packs P> using PacksOf = std::integral_constant<Packs, P>;
template <typename F> inline bool for_row_shape(int cols, F f)
{
    auto go = [&](auto t, auto e) {
        if (cols % 8 == 0) f(PacksOf<Packs::kWhole>{}, t, e);
        else f(PacksOf<Packs::kOdd>{}, t, e);
        return true;
    };
    if (cols < 8) {
        f(PacksOf<Packs::kFew>{}, std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
        return true;
    }
#define GDN2_ROW(T, E) \
    if (cols <= 8 * T * E) return go(std::integral_constant<int, T>{}, std::integral_constant<int, E>{});
    GDN2_ROW(8, 1)
    GDN2_ROW(16, 1)
    GDN2_ROW(32, 1)
    GDN2_ROW(64, 1)
    GDN2_ROW(64, 2)
    GDN2_ROW(64, 4)
    GDN2_ROW(256, 2)
    GDN2_ROW(256, 4)
    GDN2_ROW(1024, 2)
#undef GDN2_ROW
    return false;
}

inline int row_grid(int64_t rows, int rpb, int most) { return (int)std::min<int64_t>((rows + rpb - 1) / rpb, most); }

} // namespace gdn2
