// Host-side launch interface between the C ABI (dense_api.hip) and the kernels of
// a layer's dense half: its projections (linear_*.hip), the norm before them
// (rms_norm.hip) and the clipping of their gradients (grad_clip.hip).
#pragma once

#include "gdn2_launch.hpp"

namespace gdn2 {

// RMS norm of x + residual over rows (rms_norm.hip).
struct RmsNormArgs {
    const void *x, *residual;    // residual, sum: or null
    const float *weight;
    void *y, *sum;
    float *scale;                // [rows]: y is e4m3; null: bf16 or fp32
    int64_t rows;
    int cols;
    float eps;
    bool in_bf16, out_bf16;      // x, residual, sum; y
};
struct RmsNormBwdArgs {
    const void *dy, *h;
    const float *weight;
    const void *dsum;            // or null
    void *dh;                    // dsum, dh: the type of h
    float *dweight;
    int64_t rows;
    int cols;
    float eps;
    bool in_bf16, out_bf16;      // h; dy
    void *workspace;
};
size_t rms_bwd_workspace(int64_t rows, int cols);
hipError_t launch_rms_norm_fwd(const RmsNormArgs &a, hipStream_t st);
hipError_t launch_rms_norm_bwd(const RmsNormBwdArgs &a, hipStream_t st);

// The norm over many tensors, and their scaling (grad_clip.hip). Arrays of the host.
struct ClipArgs {
    const void *const *in;
    void *const *out;            // null: the norm alone
    const int64_t *sizes;
    const int32_t *in_types, *out_types;
    int count;
    float max_norm;
    const float *norm_in;        // or null: it is computed
    float *norm_out;             // or null
    double *partial;             // [kClipGrid]
};
constexpr int kClipGrid = 1024;  // most workgroups of the norm, and partial sums
hipError_t launch_clip(const ClipArgs &a, hipStream_t st);

// Products with both operands' contracted axis along their rows (linear_impl.hpp).
// (kE4m3Wide: e4m3 operands that are widened to bf16 in registers; launches name kE4m3)
enum class Elt { kBf16, kF32, kE4m3, kE4m3Wide };
enum Act { kActNone = 0, kActSigmoid = 1, kActSilu = 2, kActGelu = 3 };
inline int elt_size(Elt e) { return e == Elt::kBf16 ? 2 : e == Elt::kF32 ? 4 : 1; }

// y[m][n] = act(sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
struct GemmArgs {
    const void *x, *w;
    int64_t ldx, ldw;            // bytes from a row to the next
    int64_t kbytes;              // bytes of a row that count
    int64_t M, N;
    const float *sx, *sw;        // or null
    const float *bias;           // or null
    const void *residual;        // [M][N], type of y; or null
    void *y, *preact;            // [M][N]; preact (bf16 where y's operands are, else fp32): or null
    int act;
    bool out_bf16, preact_bf16;
    // splits > 1 (rows at whole 16 bytes only): partial [splits][M][ldp]; ldp: N rounded up to eight, and
    // so many rows of w can be read
    float *partial;
    int64_t ldp;
    int splits;
};
// parts that the contraction is split into, for a product whose partial sums may be kept in a workspace
int gemm_splits(int64_t M, int64_t N, int64_t kbytes);
int gemm_columns_splits(int64_t M, int64_t N, int64_t kbytes);
hipError_t launch_gemm(Elt e, const GemmArgs &a, const char *name, hipStream_t st);
// The contracted axis down the columns, bf16: x [kbytes / 2][ldx], w [kbytes / 2][ldw], rows at whole 16
// bytes, N in eights.
hipError_t launch_gemm_columns(const GemmArgs &a, hipStream_t st);
// Whether a product in fp32 takes w (and, with turned_x, x) [count][N] ([count][M]) as they lie, and that product: a.kbytes
// is 4 count then, the rows of an x that is not turned are whole chunks.
bool gemm_columns_f32(int64_t M, int64_t N, int64_t count, bool turned_x);
hipError_t launch_gemm_columns_f32(const GemmArgs &a, bool turned_x, hipStream_t st);
hipError_t launch_gemm_bf16(const GemmArgs &a, hipStream_t st);
hipError_t launch_gemm_f32(const GemmArgs &a, hipStream_t st);
hipError_t launch_gemm_e4m3(const GemmArgs &a, hipStream_t st);

// Gradient of a linear layer (linear_bwd.hip).
struct LinearBwdArgs {
    const void *dy, *x, *w, *preact;
    void *dx, *dweight;          // either may be null
    float *dbias;                // or null
    int64_t M;
    int N, K;
    int act;
    bool bf16, dy_bf16;          // x, w, preact, dx, dweight; dy
    void *workspace;
};
size_t linear_bwd_workspace(int64_t M, int N, int K, int act, bool bf16, bool dy_bf16, bool need_dx, bool need_dw,
                            bool need_db);
hipError_t launch_linear_bwd(const LinearBwdArgs &a, hipStream_t st);

} // namespace gdn2
