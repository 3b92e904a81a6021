// The norm over many tensors and their scaling to a largest norm:
//
//   norm = sqrt(sum over all elements of g^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// Up to kTensors tensors are one launch, their addresses in the kernel's
// arguments (nothing is copied to the device, so a call can be captured). Every
// workgroup takes every gridDim-th piece of kPiece elements, whichever tensor it
// lies in; further launches add to the same partial sums. Squares and sums are
// fp64 (half the fp32 vector rate, and the loads take longer): no square of a
// float overflows or vanishes there. The scaling kernel's workgroups
// each add the partial sums themselves, in one order, so the norm costs no
// launch of its own and its bits do not depend on timing. The scaling goes from the
// last piece to the first: what the norm read last is still in the cache.
// Bound by memory.
#include "dense_launch.hpp"
#include "rows.hpp"

#include <algorithm>

namespace gdn2 {

constexpr int kTensors = 64, kThreads = 256, kRounds = 8, kPiece = kThreads * 8 * kRounds;

// Most workgroups of the scaling: many short ones keep reads and writes even (206 M bf16 to fp32,
// both kernels: 358 us with 1024 of them and two rounds of loads each under way, 285 with 16384). Up to
// kCached bytes in all what the norm read is in the caches, and read from there; more of it
// is read past them (7 M floats 20 us instead of 27, 206 M bf16 to fp32 285 instead of 317).
constexpr int kScaleGrid = 16 * kClipGrid;
constexpr int64_t kCached = 128 << 20;

struct ClipBatch {
    const void *in[kTensors];
    void *out[kTensors];
    int64_t n[kTensors];
    int32_t first[kTensors];     // its first piece
    uint64_t in_bf16, out_bf16;  // bits
    int count, pieces;
};

// Tensor that piece p lies in: the last one that begins at or before it
// (tensors without elements are not in a batch).
static __device__ __forceinline__ int tensor_of(const ClipBatch &b, int p)
{
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.first[mid] <= p) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Sum over the workgroup, in every thread, always in the same order.
static __device__ __forceinline__ double block_sum(double s, double *red)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) s += red[i];
    __syncthreads();
    return s;
}

template <typename In> static __device__ __forceinline__ double piece_squares(const In *p, int64_t n)
{
    double s = 0.;
    Pack8<In> x[kRounds];
    if (n >= kPiece) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) x[r].template load<false, false>(p + (r * kThreads + (int)threadIdx.x) * 8);
    } else {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int at = (r * kThreads + (int)threadIdx.x) * 8;
            if (at + 8 <= n) x[r].template load<false, false>(p + at);
            else x[r].load_some(p + at, (int)n - at);
        }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double v = (double)x[r].get(i);
            s += v * v;
        }
    return s;
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(ClipBatch b, double *partial, int further)
{
    __shared__ double red[kThreads / 64];
    double s = 0.;
    for (int p = blockIdx.x; p < b.pieces; p += gridDim.x) {
        const int t = tensor_of(b, p);
        const int64_t at = (int64_t)(p - b.first[t]) * kPiece, n = b.n[t] - at;
        s += (b.in_bf16 >> t) & 1 ? piece_squares((const uint16_t *)b.in[t] + at, n)
                                  : piece_squares((const float *)b.in[t] + at, n);
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = (further ? partial[blockIdx.x] : 0.) + s;
}

static __device__ __forceinline__ double norm_of(const double *partial, int parts, double *red)
{
    double s = 0.;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    return sqrt(block_sum(s, red));
}

__global__ __launch_bounds__(kThreads) void clip_finish_kernel(const double *partial, int parts, float *norm)
{
    __shared__ double red[kThreads / 64];
    const double x = norm_of(partial, parts, red);
    if (threadIdx.x == 0) *norm = (float)x;
}

// What the gradients are multiplied by, as a normal number and a power of two (2^0 but for quotients below those:
// a large gradient times such a one is an ordinary float). Beside a plain product: 206 M bf16 to fp32 286.2 us and
// 285.8, 7 M floats 20.9 and 20.5.
struct Factor {
    float m;
    int e;
    __device__ __forceinline__ explicit Factor(double q)   // (NaN stays)
    {
        const bool small = q < 0x1p-126;
        m = q >= 1. ? 1.f : (float)(small ? __builtin_amdgcn_frexp_mant(q) : q);
        e = small ? __builtin_amdgcn_frexp_exp(q) : 0;
    }
    __device__ __forceinline__ float operator()(float x) const { return __builtin_amdgcn_ldexpf(x * m, e); }
    __device__ __forceinline__ bool one() const { return m == 1.f && e == 0; }
};

// n elements of p (kPiece at most) to o, times c. A lane takes eight neighbours at a time, or four where one
// side is fp32, so that a wave's loads and stores are each in one piece.
template <bool CACHED, typename In, typename Out>
static __device__ __forceinline__ void piece_scale(const In *p, Out *o, int64_t n, Factor c)
{
    constexpr int V = sizeof(In) + sizeof(Out) > 4 ? 4 : 8, R = 2;   // rounds whose loads are under way at once
    typedef uint32_t vin __attribute__((ext_vector_type(V * sizeof(In) / 4)));
    typedef uint32_t vout __attribute__((ext_vector_type(V * sizeof(Out) / 4)));
    typedef vin vin_any __attribute__((aligned(sizeof(In))));
    typedef vout vout_any __attribute__((aligned(sizeof(Out))));
    auto get = [](const vin &x, int i) {
        if constexpr (sizeof(In) == 4) return __uint_as_float(x[i]);
        else return __uint_as_float((i & 1) ? (x[i >> 1] & 0xFFFF0000u) : (x[i >> 1] << 16));
    };
#pragma unroll 1
    for (int first = 0; first < kPiece; first += R * kThreads * V) {
        vin x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int at = first + (r * kThreads + (int)threadIdx.x) * V;
            if (at + V <= n) {
                const vin_any *q = reinterpret_cast<const vin_any *>(p + at);
                if constexpr (CACHED) x[r] = *q;
                else x[r] = __builtin_nontemporal_load(q);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int at = first + (r * kThreads + (int)threadIdx.x) * V;
            if (at + V <= n) {
                vout y;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if constexpr (sizeof(Out) == 4) y[i] = __float_as_uint(c(get(x[r], i)));
                    else if (i % 2 == 0) y[i / 2] = bf16x2(c(get(x[r], i)), c(get(x[r], i + 1)));
                }
                __builtin_nontemporal_store(y, reinterpret_cast<vout_any *>(o + at));
            } else {
                for (int i = at; i < n && i < at + V; ++i) store1(o + i, c(in2f<In>(p[i])));
            }
        }
    }
}

template <bool CACHED>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipBatch b, const double *partial, int parts,
                                                              const float *norm_in, float *norm_out, float max_norm)
{
    __shared__ double red[kThreads / 64];
    // (a norm beyond the largest float still scales by what it is)
    const double norm = norm_in ? (double)*norm_in : norm_of(partial, parts, red);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    const Factor c((double)max_norm / (norm + 1e-6));
    for (int i = blockIdx.x; i < b.pieces; i += gridDim.x) {
        const int p = b.pieces - 1 - i, t = tensor_of(b, p);
        const int64_t at = (int64_t)(p - b.first[t]) * kPiece, n = b.n[t] - at;
        if (c.one() && b.in[t] == b.out[t]) continue;   // nothing to change
        const bool ib = (b.in_bf16 >> t) & 1, ob = (b.out_bf16 >> t) & 1;
        if (ib) {
            const uint16_t *x = (const uint16_t *)b.in[t] + at;
            if (ob) piece_scale<CACHED>(x, (uint16_t *)b.out[t] + at, n, c);
            else piece_scale<CACHED>(x, (float *)b.out[t] + at, n, c);
        } else {
            const float *x = (const float *)b.in[t] + at;
            if (ob) piece_scale<CACHED>(x, (uint16_t *)b.out[t] + at, n, c);
            else piece_scale<CACHED>(x, (float *)b.out[t] + at, n, c);
        }
    }
}

// Calls f with each batch of tensors that hold anything, in order or from the last.
// The pieces of a batch stay below 2^31 (the caller bounds a tensor's size).
template <typename F> static void for_batches(const ClipArgs &a, bool backwards, F f)
{
    ClipBatch b;
    auto reset = [&] { b.count = b.pieces = 0; b.in_bf16 = b.out_bf16 = 0; };
    reset();
    for (int k = 0; k < a.count; ++k) {
        const int i = backwards ? a.count - 1 - k : k;
        if (a.sizes[i] == 0) continue;
        const int64_t pieces = (a.sizes[i] + kPiece - 1) / kPiece;
        if (b.count == kTensors || b.pieces + pieces > 0x7fff0000LL) {
            f(b);
            reset();
        }
        b.in[b.count] = a.in[i];
        b.out[b.count] = a.out ? a.out[i] : nullptr;
        b.n[b.count] = a.sizes[i];
        b.first[b.count] = b.pieces;
        if (a.in_types[i] == 1) b.in_bf16 |= 1ull << b.count;
        if (a.out && a.out_types[i] == 1) b.out_bf16 |= 1ull << b.count;
        b.pieces += (int)pieces;
        ++b.count;
    }
    if (b.count) f(b);
}

hipError_t launch_clip(const ClipArgs &a, hipStream_t st)
{
    int64_t most = 0;
    for_batches(a, false, [&](const ClipBatch &b) { most = std::max<int64_t>(most, b.pieces); });
    // (no elements: one workgroup adds no parts)
    const int parts = (int)std::min<int64_t>(most, kClipGrid);
    if (!a.norm_in) {
        prof_before("gdn2_grad_norm", st);
        int further = 0;
        for_batches(a, false, [&](const ClipBatch &b) {
            hipLaunchKernelGGL(clip_norm_kernel, dim3(parts), dim3(kThreads), 0, st, b, a.partial, further);
            further = 1;
        });
        prof_after(st);
    }
    if (!a.out || parts == 0) {
        if (!a.norm_in) hipLaunchKernelGGL(clip_finish_kernel, dim3(1), dim3(kThreads), 0, st, a.partial, parts, a.norm_out);
        return hipGetLastError();
    }
    int64_t bytes = 0;
    for (int i = 0; i < a.count; ++i) bytes += a.sizes[i] * ((a.in_types[i] == 1 ? 2 : 4) + (a.out_types[i] == 1 ? 2 : 4));
    prof_before("gdn2_clip_grads", st);
    float *norm_out = a.norm_out;
    for_batches(a, true, [&](const ClipBatch &b) {
        const auto kernel = bytes <= kCached ? clip_scale_kernel<true> : clip_scale_kernel<false>;
        hipLaunchKernelGGL(kernel, dim3(std::min(b.pieces, kScaleGrid)), dim3(kThreads), 0, st, b, a.partial, parts, a.norm_in,
                           norm_out, a.max_norm);
        norm_out = nullptr;
    });
    prof_after(st);
    return hipGetLastError();
}

} // namespace gdn2
