// Host-side launch interface between the C ABI (operators_api.hip) and the kernels
// of the operators around the mixer. (Apart from gdn2_launch.hpp, which the
// mixer's kernels include: the counters taken on those hold as long as their
// sources are unchanged.)
#pragma once

#include "gdn2_launch.hpp"

namespace gdn2 {

// The recurrence over short runs of tokens, states in a pool (recurrent_impl.hpp).
struct RecurrentArgs {
    const void *q, *k, *v, *b, *w;
    const float *log_alpha;
    float *state;                // [slots][H][dk][dv]
    const int32_t *slot_in;      // [N] or null (sequence i reads slot i)
    const int32_t *slot_out;     // [N] or null (= slot_in)
    const int32_t *commit;       // [N] or null (every token)
    void *o;
    const int32_t *cu_seqlens;
    int T, N, H, HK, slots, dk, dv;   // T: tokens per sequence, or in all with cu_seqlens
    int gates;
    bool bf16, out_bf16;
};
hipError_t launch_recurrent(const RecurrentArgs &a, hipStream_t st);
hipError_t launch_recurrent_bf16(const RecurrentArgs &a, hipStream_t st);
hipError_t launch_recurrent_f32(const RecurrentArgs &a, hipStream_t st);

// The prologue on its own (prologue.hip): tensors 0, 1, 2 are q, k, v.
struct PrologueArgs {
    const void *x[3];            // raw, [tokens][heads][d]
    const float *weight[3], *bias[3];
    const void *hist_in[3];      // [slots][heads][3][d], or null
    void *hist_out[3];           // or null; may equal hist_in
    const int32_t *slot_in, *slot_out;   // [N], or null (sequence i: slot i; slot_out: = slot_in)
    const int32_t *commit;       // [N] or null (every token)
    void *y[3];
    const void *logit[2];        // b, w: [tokens][nlogit]
    void *gate[2];
    const int32_t *cu_seqlens;
    int T, N, slots;
    int heads[3], d[3];
    int nlogit[2];
    bool bf16;
};
hipError_t launch_prologue_fwd(const PrologueArgs &a, hipStream_t st);

struct PrologueBwdArgs {
    PrologueArgs f;              // x, weight, bias, hist_in, slot_in, logit, sizes
    const float *dy[3], *dgate[2];
    void *dx[3], *dlogit[2];     // input type or, with out_bf16 = false, float
    bool out_bf16;
    float *dweight[3], *dbias[3];
    void *workspace;
};
// tokens each thread of the backward passes over, and its workspace
int prologue_bwd_tile(long long tokens, long long channels);
size_t prologue_bwd_workspace(long long tokens, long long channels);
hipError_t launch_prologue_bwd(const PrologueBwdArgs &a, hipStream_t st);

// LayerNorm(x + residual) over rows (layer_norm.hip).
struct LayerNormArgs {
    const void *x, *residual;    // residual, bias, sum: or null
    const float *weight, *bias;
    void *y, *sum;
    int64_t rows;
    int cols;
    float eps;
    bool in_bf16, out_bf16;      // x, residual, sum; y
};
struct LayerNormBwdArgs {
    const void *dy, *h;          // dy in the output type of the forward
    const float *weight;
    const void *dsum;            // or null
    void *dh;                    // dsum, dh: the type of h
    float *dweight, *dbias;      // dbias: or null
    int64_t rows;
    int cols;
    float eps;
    bool in_bf16, out_bf16;      // h; dy
    void *workspace;             // [ln_bwd_parts][2][cols] floats
};
// most workgroups of the two kernels (each takes every gridDim-th set of rows)
constexpr int kLnFwdGrid = 2048, kLnBwdGrid = 512;
int ln_bwd_parts(int64_t rows, int cols);
hipError_t launch_layer_norm_fwd(const LayerNormArgs &a, hipStream_t st);
hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs &a, hipStream_t st);

// Column sums of partial rows: for each job, out0[c] (c < n0) and out1[c - n0]
// (c < n0 + n1) are the sums over `parts` rows of n0 + n1 floats, added in
// row order within 16 strided classes and then over the classes.
struct ColumnSums {
    const float *part[3];
    float *out0[3], *out1[3];    // out1: or null (not written)
    int n0[3], n1[3];
    int parts, jobs;
};
hipError_t launch_column_sums(const ColumnSums &c, const char *name, hipStream_t st);

} // namespace gdn2
