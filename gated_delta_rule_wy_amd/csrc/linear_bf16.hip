// Products of rows in bf16 (linear_impl.hpp).
#include "linear_impl.hpp"

namespace gdn2 {

hipError_t launch_gemm_columns(const GemmArgs &a, hipStream_t st)
{
    auto run = [&](auto b, auto wm, auto wn) {
        constexpr int B = decltype(b)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
        const int64_t tm = (a.M + B - 1) / B, tn = (a.N + B - 1) / B;
        const int64_t grid = std::min<int64_t>((tm * tn * a.splits + 7) / 8 * 8, WM * WN == 8 ? 256 : 512);
        hipLaunchKernelGGL((gemm_tile_kernel<Elt::kBf16, B, B, WM, WN, true>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, st, a,
                           (int)tm, (int)tn);
    };
    // (the joining pass has a workgroup for 2048 elements; parts are of few tiles only, so its grid is never too large where
    // they are asked for)
    const int64_t blocks = (a.M * ((a.N + 7) / 8) + 255) / 256;
    if (a.N % 8 || a.ldx % 16 || a.ldw % 16 || (a.splits > 1 && (a.ldp != a.N || blocks > 0xffffffLL))) return hipErrorInvalidConfiguration;
    using i2 = std::integral_constant<int, 2>;
    if (((a.M + 255) / 256) * ((a.N + 255) / 256) * a.splits >= 192)
        run(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{}, i2{});
    else run(std::integral_constant<int, 128>{}, i2{}, i2{});
    if (a.splits > 1) hipLaunchKernelGGL(gemm_join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_gemm_bf16(const GemmArgs &a, hipStream_t st) { return launch_gemm_type<Elt::kBf16>(a, st); }

} // namespace gdn2
