// Products of rows in f32 (linear_impl.hpp), and of columns: a gradient's sums over rows, read as
// the operands lie.
#include "linear_impl.hpp"

namespace gdn2 {

// As gemm_split_kernel in blocks of 64 x 64, but w [kbytes / 4][N] (and x [..][M] with XT) have the contracted
// axis down their columns. A lane reads four neighbouring columns of a row at once; each of
// them belongs to another of the four blocks of 16, so element q of block j is column 4 q + j. A step
// is 16 of the contracted axis: eight waves share out parts of it more evenly than 32 at a time. None is
// asked for ahead: the registers hold a second workgroup a compute unit instead, which does more (the whole
// gradient, 1554 x 1001 x 777: 86 us, 90 with two steps ahead, 107 with operands turned in
// memory before; 2048^3 289, 317, 333). Bound by the matrix instructions, 30 us of the 86 for
// both products at the rate of a large one; the rest is workgroups of which some units have two and some one.
template <bool XT> __global__ __launch_bounds__(kWaves * 64) void gemm_split_columns_kernel(GemmArgs a)
{
    constexpr int PITCH = 64 + 4, ROWS = 32;   // rows a round through LDS
    __shared__ __attribute__((aligned(16))) float sums[kWaves][ROWS * PITCH];
    const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const uint32_t count = (uint32_t)(a.kbytes / 4), ldx = (uint32_t)a.ldx, ldw = (uint32_t)a.ldw;
    const auto bx = XT ? buffer_at(a.x, 0, (int64_t)count * a.ldx) : buffer_at(a.x, m0 * a.ldx, a.M * a.ldx);
    const auto bw = buffer_at(a.w, 0, (int64_t)count * a.ldw);
    // Columns n .. n + 3 of row k, of `cols` in a row. Beyond the last row are zeros. Those behind a row's end are the
    // next row's first, and no sum that is stored takes them; the last row's (`end`) are asked for one by one.
    auto columns = [&](const __amdgpu_buffer_rsrc_t &b, uint32_t k, int64_t n, int64_t cols, uint32_t ld, bool end) GDN2_INLINE -> u4 {
        const uint32_t at = n < cols ? k * ld + (uint32_t)n * 4 : kBeyond;
        if (!end) return __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, 0);
        u4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)(n + j < cols ? at + j * 4 : kBeyond), 0, 0);
        return v;
    };
    u4 fx[4], fw[4];
    auto load = [&](int s) GDN2_INLINE {
        const uint32_t k = s * 16 + g * 4;
        const bool end = (uint32_t)s * 16 + 16 >= count;
#pragma unroll
        for (int t = 0; t < 4; ++t) fw[t] = columns(bw, k + t, n0 + r * 4, a.N, ldw, end);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if constexpr (XT) fx[t] = columns(bx, k + t, m0 + r * 4, a.M, ldx, end);
            else fx[t] = __builtin_amdgcn_raw_buffer_load_b128(bx, (int)(k < count ? (uint32_t)(t * 16 + r) * ldx + k * 4 : kBeyond), 0, 0);
    };
    f4 acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = f4zero();
    const int steps = (int)((count + 15) / 16);
    for (int s = wv; s < steps; s += kWaves) {
        load(s);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fw[t][j]),
                                                                     __uint_as_float(XT ? fx[t][i] : fx[i][t]), acc[j][i], 0, 0, 0);
    }
    // row e of round q
    auto row_of = [](int q, int e) GDN2_INLINE { return XT ? e / 2 * 4 + q * 2 + e % 2 : q * 32 + e; };
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (q) __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<f4 *>(&sums[wv][(XT ? r * 2 + i : i * 16 + r) * PITCH + g * 16 + c * 4]) =
                    (f4){acc[0][q * 2 + i][c], acc[1][q * 2 + i][c], acc[2][q * 2 + i][c], acc[3][q * 2 + i][c]};
        __syncthreads();
        if (threadIdx.x < ROWS * 8) {
            const int e = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
            const int64_t m = m0 + row_of(q, e), n = n0 + col;
            if (m < a.M && n < a.N) {
                const int cnt = (int)min((int64_t)8, a.N - n);
                Finish8 fin;
                fin.load(a, m, n, cnt);
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kWaves; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f4 s = *reinterpret_cast<const f4 *>(&sums[i][e * PITCH + col + h * 4]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[h * 4 + c] += s[c];
                    }
                fin.store(a, m, n, cnt, v);
            }
        }
    }
}

hipError_t launch_gemm_columns_f32(const GemmArgs &a, bool turned_x, hipStream_t st)
{
    const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64));
    if (turned_x) hipLaunchKernelGGL(gemm_split_columns_kernel<true>, grid, dim3(kWaves * 64), 0, st, a);
    else hipLaunchKernelGGL(gemm_split_columns_kernel<false>, grid, dim3(kWaves * 64), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_gemm_f32(const GemmArgs &a, hipStream_t st) { return launch_gemm_type<Elt::kF32>(a, st); }

} // namespace gdn2
