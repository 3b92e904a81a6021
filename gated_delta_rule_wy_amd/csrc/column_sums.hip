// Sums of partial rows (gradients of weights): out[c] = sum over rows of part[row][c].
//
// A workgroup of 16 waves owns 64 columns; each wave adds every 16th row (256
// contiguous bytes a row), then one wave adds the 16 sums in order. The order
// is fixed, so the same partial rows give the same bits. Bound by latency: each
// wave's rows come in a few rounds of eight loads (128 rows of 30720 sums 6 us,
// 512 of 4096 5 us, most of it the launch's own).
#include "gdn2_device.hpp"
#include "operators_launch.hpp"

#include <algorithm>

namespace gdn2 {

__global__ __launch_bounds__(1024) void column_sums_kernel(ColumnSums cs)
{
    __shared__ float acc[16][64];
    const int job = blockIdx.y, l = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int n0 = cs.n0[job], n = n0 + cs.n1[job], c = blockIdx.x * 64 + l;
    const float *part = cs.part[job];
    float s = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int i = wv; i < cs.parts; i += 16) s += part[(size_t)i * n + c];
    }
    acc[wv][l] = s;
    __syncthreads();
    if (wv == 0 && c < n) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += acc[i][l];
        if (c < n0) cs.out0[job][c] = t;
        else if (cs.out1[job]) cs.out1[job][c - n0] = t;
    }
}

hipError_t launch_column_sums(const ColumnSums &c, const char *name, hipStream_t st)
{
    int n = 0;
    for (int j = 0; j < c.jobs; ++j) n = std::max(n, c.n0[j] + c.n1[j]);
    prof_before(name, st);
    hipLaunchKernelGGL(column_sums_kernel, dim3((n + 63) / 64, c.jobs), dim3(1024), 0, st, c);
    prof_after(st);
    return hipGetLastError();
}

} // namespace gdn2
