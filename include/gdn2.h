/*
 * gdn2.h - C ABI of libgdn2, the MI355X (gfx950) Gated DeltaNet-2 token mixer.
 *
 * The operation (snilld.dk, "Gated DeltaNet-2 fra NVIDIA ...", section "Hvad
 * Gated DeltaNet-2 ændrer", compact update equation), per sequence and head:
 *
 *     S_t = (I - k_t (b_t * k_t)^T) Diag(alpha_t) S_{t-1} + k_t (w_t * v_t)^T
 *     o_t = S_t^T q_t
 *
 * with state S in R^{dk x dv} (rows are key channels), channel-wise decay
 * alpha_t = exp(log_alpha_t) in (0, 1]^{dk} applied before the edit, erase
 * gate b_t in [0, 1]^{dk} and write gate w_t in [0, 1]^{dv} (both already
 * passed through their sigmoid), and readout after the update (aifetchly-
 * blog.pages.dev, "Gated DeltaNet-2 Guide", layer workflow step 4). No query
 * scale is applied. A missing initial state means zeros, and the final state
 * is returned, as in that guide's "End-to-End PyTorch Implementation".
 *
 * Conventions for every entry point:
 *  - All pointers are DEVICE pointers except where stated. The caller owns
 *    every buffer; the library allocates no device memory and keeps no pointer
 *    after a call returns.
 *  - Layouts are dense row-major. Token tensors are [tokens, H, d], where
 *    tokens = B*T (equal-length rows back to back) or the packed total.
 *  - Work is enqueued on the calling thread's stream (gdn2_set_stream) and the
 *    call returns without synchronising. Device-side faults surface at the
 *    caller's next synchronisation, like any other stream work.
 *  - Arguments are validated on the host before anything is enqueued. On any
 *    non-OK status nothing has been launched. GDN2_ERR_HIP reports a launch
 *    error from the HIP runtime.
 *  - Preconditions that are not checked on the host: contiguity; finite
 *    log_alpha <= 0; cu_seqlens starting at 0, non-decreasing and ending at T.
 *  - Device pointers must be 16-byte aligned.
 */
#ifndef GDN2_H
#define GDN2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN2_OK = 0,
    GDN2_ERR_INVALID = 1,     /* null/misaligned pointer, bad size or dims    */
    GDN2_ERR_UNSUPPORTED = 2, /* valid but not implemented (head dims, dtype) */
    GDN2_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required   */
    GDN2_ERR_HIP = 4          /* the HIP runtime reported an error            */
} gdn2_status;

/* Values of the in_dtype / out_dtype arguments. Those arguments are plain
 * ints, so that any value a caller passes is well defined on the library's
 * side; a value that is not one of these gives GDN2_ERR_INVALID. */
typedef enum {
    GDN2_F32 = 0,
    GDN2_BF16 = 1,
    GDN2_E4M3 = 2             /* 8 bits, only where an entry point names it   */
} gdn2_dtype;

/*
 * Gate layouts for the *_gates entry points. A set bit means that gate holds
 * one value per token and head ([tokens, H], or [N, H] for a decode step)
 * instead of one per channel; the value applies to every channel. Kimi Delta
 * Attention is the erase and write gates collapsed to one scalar beta per
 * token-head (pass GDN2_GATE_B_PER_HEAD | GDN2_GATE_W_PER_HEAD with b == w),
 * and Gated DeltaNet additionally has a scalar decay (also set
 * GDN2_GATE_ALPHA_PER_HEAD): the special cases that Gated DeltaNet-2 reduces
 * to (snilld.dk, section "Hvad Gated DeltaNet-2 ændrer").
 */
typedef enum {
    GDN2_GATES_PER_CHANNEL = 0,
    GDN2_GATE_B_PER_HEAD = 1,
    GDN2_GATE_W_PER_HEAD = 2,
    GDN2_GATE_ALPHA_PER_HEAD = 4
} gdn2_gate_layout;

/* Set the HIP stream (a hipStream_t) used by this thread's later calls.
 * NULL selects the default stream. Always returns GDN2_OK. */
int gdn2_set_stream(void *hip_stream);

/* The stream set by this thread (NULL = default stream). */
void *gdn2_get_stream(void);

/* Human-readable name of a status code (static storage; never NULL). */
const char *gdn2_status_string(int status);

/*
 * Bytes of device workspace that gdn2_chunk_fwd needs for these sizes, or 0
 * if the arguments are invalid or unsupported. `varlen` is 1 when the call
 * will pass cu_seqlens (then B must be 1 and T is the total token count).
 */
size_t gdn2_chunk_fwd_workspace_bytes(int B, int T, int N, int H, int dk, int dv,
                                      int in_dtype, int varlen);

/*
 * Prefill forward over a batch, chunkwise (64-token chunks, WY form: the
 * chunk's rank-one erase factors with the cumulative decay folded in are
 * applied as one block per chunk, snilld.dk, section "Hvad betyder det for
 * træning og inferens").
 *
 *   q, k, b    [tokens, H, dk]  in_dtype (GDN2_BF16 or GDN2_F32)
 *   v, w       [tokens, H, dv]  in_dtype
 *   log_alpha  [tokens, H, dk]  float, finite, <= 0
 *   S0         [N, H, dk, dv]   float, or NULL for zeros
 *   o          [tokens, H, dv]  out_dtype (GDN2_F32 only)
 *   ST         [N, H, dk, dv]   float, or NULL; may alias S0
 *   cu_seqlens [N + 1]          int32 device array, or NULL
 *
 * Without cu_seqlens the batch is B sequences of T tokens each and N must
 * equal B. With cu_seqlens, B must be 1, T is the total token count and
 * sequence i is tokens [cu_seqlens[i], cu_seqlens[i+1]); sequences may be
 * empty (then ST[i] = S0[i]). Outputs must not alias the token inputs.
 * Supported head dims: dk in {32, 64, 128} for bf16 inputs and
 * {16, 32, 64, 128} for f32 inputs; dv in {16, 32, 64, 128}.
 * workspace: device memory of at least gdn2_chunk_fwd_workspace_bytes(...).
 *
 * Value range (bf16 inputs, whose products run on f16 matrix cores): q_t
 * and k_t must have at most unit L2 norm per token and head, as the layer's
 * L2 normalisation gives them (bf16 rounding aside; "Gated DeltaNet-2 Guide",
 * section "2. Normalization and Short Convolutions"). v, w, S0 and the state
 * have no bound: every value column of the state, of w * v and of the
 * corrected writes is carried through the f16 products with its own power of
 * two scale, chosen each chunk, so large states stay finite and small ones
 * keep full precision. fp32 inputs run on fp32 matrix cores.
 */
int gdn2_chunk_fwd(const void *q, const void *k, const void *v, const float *log_alpha,
                   const void *b, const void *w, const float *S0, void *o, float *ST,
                   const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                   int in_dtype, int out_dtype, void *workspace,
                   size_t workspace_bytes);

/*
 * gdn2_chunk_fwd for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same arguments without the workspace, which instead lives in a fixed
 * device array of GDN2_NOALLOC_WORKSPACE_MAX bytes inside the library, one
 * per device, held until the process ends. Nothing is allocated or freed
 * during the call. Sizes whose workspace (gdn2_chunk_fwd_workspace_bytes)
 * exceeds GDN2_NOALLOC_WORKSPACE_MAX give GDN2_ERR_WORKSPACE, with nothing
 * launched; e.g. 4 x 4096 tokens x 16 heads at d = 128 fit (254 MB). Every
 * call on one device shares that device's array: calls that can overlap on
 * one device (other streams, other host threads) race and must be
 * serialised by the caller. Results are those of gdn2_chunk_fwd.
 */
#define GDN2_NOALLOC_WORKSPACE_MAX (256u << 20)
int gdn2_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const float *log_alpha,
                           const void *b, const void *w, const float *S0, void *o, float *ST,
                           const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                           int in_dtype, int out_dtype);

/*
 * gdn2_chunk_fwd with the gate layouts given by `gates` (gdn2_gate_layout
 * bits): b is [tokens, H] when GDN2_GATE_B_PER_HEAD is set, w is [tokens, H]
 * with GDN2_GATE_W_PER_HEAD and log_alpha is [tokens, H] with
 * GDN2_GATE_ALPHA_PER_HEAD; the other arguments, the workspace size and the
 * errors are those of gdn2_chunk_fwd. Unknown bits give GDN2_ERR_INVALID.
 * gdn2_chunk_fwd is this call with gates = GDN2_GATES_PER_CHANNEL.
 */
int gdn2_chunk_fwd_gates(const void *q, const void *k, const void *v, const float *log_alpha,
                         const void *b, const void *w, int gates, const float *S0, void *o, float *ST,
                         const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                         int in_dtype, int out_dtype, void *workspace,
                         size_t workspace_bytes);

/*
 * Chunk-size variants of the prefill forward: gdn2_chunk_fwd with chunks of
 * `chunk` tokens, 32, 64 or 128 (snilld.dk, section "POC-matrix der dækker
 * de hårde hjørner": latency, throughput and peak memory at C = 32 and 128
 * besides the C = 64 of the implementation). The result is the same
 * recurrence; a longer chunk halves the serial chain over chunks and
 * doubles the triangular work per token. chunk = 64 is gdn2_chunk_fwd.
 *
 * Arguments, layouts, ownership and errors as gdn2_chunk_fwd (per-channel
 * gates), with the workspace size from gdn2_chunk_fwd_sized_workspace_bytes
 * for the same chunk. A chunk other than 32, 64 or 128 gives
 * GDN2_ERR_INVALID; f32 inputs with dk = 128 and chunk = 128 give
 * GDN2_ERR_UNSUPPORTED (the preparation kernel's tiles would not fit one
 * compute unit's 160 KB of LDS).
 */
size_t gdn2_chunk_fwd_sized_workspace_bytes(int B, int T, int N, int H, int dk, int dv,
                                            int in_dtype, int varlen, int chunk);
int gdn2_chunk_fwd_sized(const void *q, const void *k, const void *v, const float *log_alpha,
                         const void *b, const void *w, const float *S0, void *o, float *ST,
                         const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                         int in_dtype, int out_dtype, int chunk, void *workspace,
                         size_t workspace_bytes);

/*
 * One recurrent decode step for N independent sequences (the same update
 * and readout for a single token; constant-size state, aifetchly, "Gated
 * DeltaNet-2 Guide", section "3. Chunkwise Parallel Algorithm ...": O(1)
 * memory during token generation).
 *
 *   q, k, b    [N, H, dk]       in_dtype
 *   v, w       [N, H, dv]       in_dtype
 *   log_alpha  [N, H, dk]       float, finite, <= 0
 *   S          [N, H, dk, dv]   float, read and updated in place
 *   o          [N, H, dv]       out_dtype (GDN2_F32 only)
 *
 * dk, dv in {16, 32, 64, 128}. S is read once and written once. Successive
 * calls from one thread on the same S visit the (sequence, head) chains in
 * alternating order (the chains written last, still in the last-level cache,
 * are read first); the results do not depend on the order.
 */
int gdn2_decode_step(const void *q, const void *k, const void *v, const float *log_alpha,
                     const void *b, const void *w, float *S, void *o, int N, int H, int dk,
                     int dv, int in_dtype, int out_dtype);

/*
 * gdn2_decode_step with the gate layouts given by `gates`: b, w and
 * log_alpha are [N, H] where their bit is set. Unknown bits give
 * GDN2_ERR_INVALID.
 */
int gdn2_decode_step_gates(const void *q, const void *k, const void *v, const float *log_alpha,
                           const void *b, const void *w, int gates, float *S, void *o, int N, int H, int dk,
                           int dv, int in_dtype, int out_dtype);

/*
 * Fused input prologue. The layer computes the mixer's inputs from its
 * projections as q = L2Norm(ShortConv(q_raw)), k = L2Norm(ShortConv(k_raw)),
 * v = ShortConv(v_raw), b = sigmoid(b_logit), w = sigmoid(w_logit)
 * (aifetchly-blog.pages.dev, "Gated DeltaNet-2 Guide", the "Architectural
 * Workflow" diagram, steps 1 and 2, and section "2. Normalization and Short
 * Convolutions"). The *_prologue entry points take the raw tensors and do
 * these steps inside the mixer's own kernels, so q, k, v, b and w never
 * travel through memory.
 *
 * ShortConv is a causal depthwise convolution of kernel 4 along the tokens
 * of each sequence: for channel c of head h (row h*d + c of the weights),
 *     y_t = bias[c] + sum_{j=0..3} weight[c][j] * x_{t-3+j}
 * so weight[c][3] multiplies the current token; no activation follows (the
 * construction in that guide's "End-to-End PyTorch Implementation"). L2Norm
 * divides by max(||y||_2, 1e-12) over the head's channels.
 *
 * All pointers in the struct are device pointers; the struct itself is
 * read on the host during the call.
 *   weight_q, weight_k  [H*dk, 4] float   required
 *   weight_v            [H*dv, 4] float   required
 *   bias_q, bias_k      [H*dk] float, or NULL for no bias
 *   bias_v              [H*dv] float, or NULL
 *   state_in_q/k/v      [N, H, 3, d] in_dtype: the three raw inputs before
 *                       each sequence's first token, oldest first; all three
 *                       NULL means zeros (sequences that start here)
 *   state_out_q/k/v     [N, H, 3, d] in_dtype: receives the last three raw
 *                       inputs of each sequence (reaching back into
 *                       state_in when a sequence is shorter than three
 *                       tokens), or all three NULL; may alias state_in
 * Only all-or-none of the three state_in (and of the three state_out)
 * pointers may be NULL, else GDN2_ERR_INVALID.
 */
typedef struct gdn2_short_conv {
    const float *weight_q, *weight_k, *weight_v;
    const float *bias_q, *bias_k, *bias_v;
    const void *state_in_q, *state_in_k, *state_in_v;
    void *state_out_q, *state_out_k, *state_out_v;
} gdn2_short_conv;

/*
 * gdn2_chunk_fwd on the raw tensors, with the prologue above fused in.
 *   q_raw, k_raw, b_logit  [tokens, H, dk]  in_dtype
 *   v_raw, w_logit         [tokens, H, dv]  in_dtype
 *   conv                   host pointer to the convolution parameters
 * log_alpha, S0, o, ST, cu_seqlens, sizes, dtypes, workspace (the size from
 * gdn2_chunk_fwd_workspace_bytes) and errors are those of gdn2_chunk_fwd.
 * Gates are per channel. The state_out tensors are written after every
 * read of state_in, so the two may alias.
 */
int gdn2_chunk_fwd_prologue(const void *q_raw, const void *k_raw, const void *v_raw, const float *log_alpha,
                            const void *b_logit, const void *w_logit, const gdn2_short_conv *conv,
                            const float *S0, void *o, float *ST, const int32_t *cu_seqlens, int B, int T,
                            int N, int H, int dk, int dv, int in_dtype, int out_dtype,
                            void *workspace, size_t workspace_bytes);

/*
 * gdn2_decode_step on the raw inputs of one token per sequence
 * (q_raw, k_raw, b_logit [N, H, dk]; v_raw, w_logit [N, H, dv]), with the
 * prologue fused in. conv->state_in_* is the convolution history (NULL:
 * zeros, the sequence's first token); conv->state_out_* receives the history
 * shifted by this token and may alias state_in_* (the usual in-place cache).
 */
int gdn2_decode_step_prologue(const void *q_raw, const void *k_raw, const void *v_raw, const float *log_alpha,
                              const void *b_logit, const void *w_logit, const gdn2_short_conv *conv, float *S,
                              void *o, int N, int H, int dk, int dv, int in_dtype, int out_dtype);

/*
 * Backward of gdn2_chunk_fwd: the gradients of a scalar loss L with respect
 * to every input, given dL/do and dL/dS_T. The chunkwise form runs the
 * forward again (keeping each chunk's start state and corrected writes),
 * passes the state gradient from the last chunk to the first, then forms
 * the per-chunk gradients in parallel (the pages name a fused chunkwise WY
 * backward for training: snilld.dk, section "Hvad betyder det for træning og
 * inferens"; aifetchly, "Gated DeltaNet-2 Guide", section "3. Chunkwise
 * Parallel Algorithm for GPU Training").
 *
 *   q, k, v, log_alpha, b, w, S0, cu_seqlens, B, T, N, H, dk, dv, in_dtype
 *                    as in gdn2_chunk_fwd (gates per channel)
 *   dO               [tokens, H, dv] float: dL/do
 *   dST              [N, H, dk, dv] float, or NULL for zero
 *   dq, dk_, db, dlog_alpha   [tokens, H, dk] float (written)
 *   dv_, dw          [tokens, H, dv] float (written)
 *   dS0              [N, H, dk, dv] float, or NULL (not written)
 *   workspace        device memory of at least
 *                    gdn2_chunk_bwd_workspace_bytes(...) bytes
 * Gradient outputs must not alias any input. Errors as in gdn2_chunk_fwd.
 * Any log_alpha <= 0 is handled (16-token blocks whose decay is too wide for
 * the factored form take exact pairwise exponents). Value range: with bf16
 * inputs the chunk start states, corrected writes and end-state gradients
 * that the backward keeps between its kernels are f16 without scales, so
 * their entries must stay below 65504 in magnitude (the forward alone has no
 * such bound).
 */
size_t gdn2_chunk_bwd_workspace_bytes(int B, int T, int N, int H, int dk, int dv,
                                      int in_dtype, int varlen);

int gdn2_chunk_bwd(const void *q, const void *k, const void *v, const float *log_alpha,
                   const void *b, const void *w, const float *S0, const float *dO, const float *dST,
                   const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                   int in_dtype, float *dq, float *dk_, float *dv_, float *dlog_alpha,
                   float *db, float *dw, float *dS0, void *workspace, size_t workspace_bytes);

/*
 * The training pair: gdn2_chunk_fwd_keep is gdn2_chunk_fwd (per-channel
 * gates) that also leaves in `workspace` what the backward would otherwise
 * recompute (each chunk's operand block, start state S_c and corrected
 * writes), and gdn2_chunk_bwd_kept is gdn2_chunk_bwd without its own run of
 * the forward, starting from what a gdn2_chunk_fwd_keep left there. A
 * training step thus runs the forward once (the chunkwise form for GPU
 * training: aifetchly, "Gated DeltaNet-2 Guide", section "3. Chunkwise
 * Parallel Algorithm for GPU Training"; snilld.dk, section "Hvad betyder det
 * for træning og inferens").
 *
 * gdn2_chunk_fwd_keep: arguments as gdn2_chunk_fwd, except that `workspace`
 *   holds at least gdn2_chunk_bwd_workspace_bytes(...) bytes. o and S_T are
 *   those gdn2_chunk_fwd returns for the same inputs, bit for bit.
 * gdn2_chunk_bwd_kept: arguments as gdn2_chunk_bwd. The workspace, q, k, v,
 *   log_alpha, b, w, S0, cu_seqlens and sizes must be those of the last
 *   gdn2_chunk_fwd_keep on this workspace, with the workspace untouched since
 *   (on the same stream, or ordered after it); then the gradients equal those
 *   of gdn2_chunk_bwd bit for bit. Nothing checks this pairing on the device:
 *   a workspace that another call overwrote gives meaningless gradients.
 * Errors as in gdn2_chunk_fwd / gdn2_chunk_bwd; nothing is launched on an
 * error.
 */
int gdn2_chunk_fwd_keep(const void *q, const void *k, const void *v, const float *log_alpha,
                        const void *b, const void *w, const float *S0, void *o, float *ST,
                        const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                        int in_dtype, int out_dtype, void *workspace, size_t workspace_bytes);

int gdn2_chunk_bwd_kept(const void *q, const void *k, const void *v, const float *log_alpha,
                        const void *b, const void *w, const float *S0, const float *dO, const float *dST,
                        const int32_t *cu_seqlens, int B, int T, int N, int H, int dk, int dv,
                        int in_dtype, float *dq, float *dk_, float *dv_, float *dlog_alpha,
                        float *db, float *dw, float *dS0, void *workspace, size_t workspace_bytes);

/*
 * ---- The recurrence over short runs of tokens, states in a pool -------------
 *
 * gdn2_recurrent_fwd applies the update and readout to the tokens of N
 * sequences one after the other, on states that live in a pool of slots: the
 * serving form between gdn2_decode_step (one token, dense states in order) and
 * gdn2_chunk_fwd (64-token chunks). It serves continuous batching (one token
 * a sequence, any slots), draft tokens whose effect must not stay (`commit`;
 * snilld.dk names state versioning and rollback as what a stateful server
 * needs) and short prompts. Everything is computed in fp32.
 *
 *   q, k       [tokens, HK, dk]     in_dtype; head h of H uses q/k head
 *                                   h / (H / HK); HK divides H
 *   v          [tokens, H, dv]      in_dtype
 *   b, w, log_alpha                 [tokens, H, dk], [tokens, H, dv] (in_dtype)
 *                                   and [tokens, H, dk] (float), or [tokens, H]
 *                                   where `gates` has their bit
 *   state      [slots, H, dk, dv]   float, updated in place
 *   slot_in    [N] int32, or NULL   the slot sequence i starts from (NULL: i)
 *   slot_out   [N] int32, or NULL   the slot its kept state goes to (NULL: slot_in)
 *   commit     [N] int32, or NULL   tokens of sequence i whose effect is kept
 *                                   (NULL: all of them)
 *   o          [tokens, H, dv]      out_dtype (GDN2_F32 or GDN2_BF16)
 *   cu_seqlens [N + 1] int32, or NULL: as in gdn2_chunk_fwd
 *
 * slot_in, slot_out, commit and cu_seqlens are device arrays. A slot number
 * outside [0, slots) means none: the sequence starts from zeros, or its state
 * is not kept. commit is taken within [0, length]: every token is read out
 * with all tokens before it applied, and the kept state is the one after the
 * first commit[i] tokens; an empty sequence, or commit 0, copies slot_in to
 * slot_out. Several sequences may start from one slot; no slot may be written
 * by two sequences of a call, nor written by one and read by another. Slots
 * that no sequence writes, and rows of o behind the last sequence, are left as
 * they were. o and state overlap neither each other nor an input. Unlike
 * elsewhere, log_alpha may be -infinity (a full forget).
 * A NaN or infinity in a token reaches that token and later ones of its
 * sequence, never an earlier token or a prefix kept without it.
 *
 * dk, dv in {16, 32, 64, 128}. GDN2_ERR_INVALID also for HK not dividing H,
 * slots < 1, slot_in NULL with slots < N, or an output's pointer that is also
 * an input's or the other output's (partial overlaps are not checked), and
 * GDN2_ERR_UNSUPPORTED for N * H * dv / 16 >= 2^26 (one launch).
 */
int gdn2_recurrent_fwd(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                       const void *w, int gates, float *state, const int32_t *slot_in, const int32_t *slot_out,
                       const int32_t *commit, void *o, const int32_t *cu_seqlens, int B, int T, int N, int H, int HK,
                       int slots, int dk, int dv, int in_dtype, int out_dtype);

/*
 * ---- The prologue on its own, and its gradient -------------------------------
 *
 * gdn2_prologue_fwd computes what the *_prologue entry points fuse (the
 * formulas above: short convolutions of q, k, v, unit norm of q and k,
 * sigmoids of the gate logits) and writes the mixer's inputs, for the entry
 * points that take those: gdn2_recurrent_fwd, gdn2_chunk_fwd_keep.
 *
 *   q_raw, k_raw [tokens, HK, dk], v_raw [tokens, H, dv]   in_dtype
 *   b_logit [tokens, H, dk], w_logit [tokens, H, dv]       in_dtype, or
 *                        [tokens, H] where `gates` has GDN2_GATE_B_PER_HEAD /
 *                        GDN2_GATE_W_PER_HEAD (no other bit)
 *   conv                 as above, with HK heads for q and k (weight_q
 *                        [HK*dk, 4]); its histories are pools:
 *                        state_in / state_out_q [slots, HK, 3, dk] and so on
 *   slot_in, slot_out, commit   as in gdn2_recurrent_fwd, for the histories:
 *                        the three raw inputs before the sequence come from
 *                        slot_in (none: zeros), the last three up to its first
 *                        commit[i] tokens go to slot_out. state_out_* may be
 *                        state_in_* (the pools updated in place).
 *   q, k, v, b, w        shaped like the raw tensors, in_dtype
 *
 * b may be b_logit and w w_logit, each of state_out_* the state_in_* of the same
 * tensor; otherwise no output may overlap an input, a weight, a history or
 * another output (GDN2_ERR_INVALID where two pointers are one; partial overlaps
 * are not checked).
 *
 * Sizes, cu_seqlens and errors as in gdn2_recurrent_fwd (slots counts only
 * where a history is given); rows behind the last sequence are left as they
 * were. The squares of a head's convolved channels are added in fp32: above
 * about 1e19 their sum is infinite and the unit vector zero. Sizes that would
 * take 2^32 threads or more in one launch give GDN2_ERR_UNSUPPORTED.
 */
int gdn2_prologue_fwd(const void *q_raw, const void *k_raw, const void *v_raw, const void *b_logit,
                      const void *w_logit, int gates, const gdn2_short_conv *conv, const int32_t *slot_in,
                      const int32_t *slot_out, const int32_t *commit, void *q, void *k, void *v, void *b, void *w,
                      const int32_t *cu_seqlens, int B, int T, int N, int H, int HK, int slots, int dk, int dv,
                      int in_dtype);

/*
 * Gradient of gdn2_prologue_fwd: from dq, dk_, dv_, db, dw (float, shaped like
 * q, k, v, b, w, as gdn2_chunk_bwd returns them) those of the raw tensors and
 * logits (grad_dtype: GDN2_F32 or GDN2_BF16) and of taps and biases (float,
 * [heads*d, 4] and [heads*d]; the three dbias pointers may each be NULL).
 * conv: weights, biases and state_in as in the forward (state_out is not
 * used); histories are taken as constants. No output, nor the workspace, may
 * overlap an input or another output (GDN2_ERR_INVALID where two pointers are
 * one).
 * workspace: gdn2_prologue_bwd_workspace_bytes(...) of device memory. The
 * taps' sums run in a fixed order: the same inputs give the same bits. Rows of
 * the raw gradients behind the last sequence are left as they were.
 */
size_t gdn2_prologue_bwd_workspace_bytes(int B, int T, int N, int H, int HK, int dk, int dv, int varlen);
int gdn2_prologue_bwd(const void *q_raw, const void *k_raw, const void *v_raw, const void *b_logit,
                      const void *w_logit, int gates, const gdn2_short_conv *conv, const int32_t *slot_in,
                      const float *dq, const float *dk_, const float *dv_, const float *db, const float *dw,
                      void *dq_raw, void *dk_raw, void *dv_raw, void *db_logit, void *dw_logit, float *dweight_q,
                      float *dweight_k, float *dweight_v, float *dbias_q, float *dbias_k, float *dbias_v,
                      const int32_t *cu_seqlens, int B, int T, int N, int H, int HK, int slots, int dk, int dv,
                      int in_dtype, int grad_dtype, void *workspace, size_t workspace_bytes);

/*
 * ---- LayerNorm(x + residual) and its gradient ---------------------------------
 *
 * The layer's closing step, LayerNorm(x + out_proj(y)) (aifetchly, "Gated
 * DeltaNet-2 Guide", "End-to-End PyTorch Implementation"), over rows of `cols`
 * elements:
 *   h = x + residual, y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias
 *
 *   x, residual  [rows, cols] in_dtype; residual may be NULL (h = x)
 *   weight, bias [cols] float; bias may be NULL (none)
 *   y            [rows, cols] out_dtype
 *   sum          [rows, cols] in_dtype, or NULL: receives h, rounded
 * y and sum may each be x or residual itself (same type), but must not overlap
 * an input otherwise, nor each other (GDN2_ERR_INVALID where they are one).
 * mean and variance are those of the unrounded h, in fp32.
 *
 * gdn2_layer_norm_bwd: from dy = dL/dy (out_dtype of the forward) and h (the
 * sum the forward wrote, or its x; in_dtype), dh = dL/dh (in_dtype; the
 * gradient of x and of residual alike), plus dsum (in_dtype) where not NULL:
 * what else depends on h. dweight, dbias [cols] float are summed over the rows
 * in a fixed order; dbias may be NULL. dh may be dy, h or dsum itself (same
 * type); otherwise no output, nor the workspace, may overlap an input or another
 * output (GDN2_ERR_INVALID where two pointers are one).
 * workspace: gdn2_layer_norm_bwd_workspace_bytes(...) of device memory.
 *
 * rows >= 0, 1 <= cols <= GDN2_LAYER_NORM_MAX_COLS, eps > 0, each finite.
 * Pointers are 16-byte aligned; cols may be any number (a multiple of 8 is
 * faster).
 */
#define GDN2_LAYER_NORM_MAX_COLS (1 << 20)
int gdn2_layer_norm_fwd(const void *x, const void *residual, const float *weight, const float *bias, void *y, void *sum,
                        int64_t rows, int cols, float eps, int in_dtype, int out_dtype);
size_t gdn2_layer_norm_bwd_workspace_bytes(int64_t rows, int cols);
int gdn2_layer_norm_bwd(const void *dy, const void *h, const float *weight, const void *dsum, void *dh, float *dweight,
                        float *dbias, int64_t rows, int cols, float eps, int in_dtype, int out_dtype, void *workspace,
                        size_t workspace_bytes);

/*
 * ---- The layer's projections, and their gradient ------------------------------
 *
 * A linear layer with what follows it (the projections to q, k, v, the gate
 * logits with their sigmoid, out_proj with the residual's addition; aifetchly,
 * "Gated DeltaNet-2 Guide", "End-to-End PyTorch Implementation"):
 *   z = x_scale[row] weight_scale[n] sum_k x[row, k] weight[n, k] + bias[n]
 *   y = act(z) + residual
 *
 *   x            [rows, in_features] in_dtype (GDN2_F32, GDN2_BF16 or GDN2_E4M3)
 *   weight       [out_features, in_features] in_dtype
 *   x_scale      [rows] float, weight_scale [out_features] float: with
 *                GDN2_E4M3, and only then (gdn2_rms_norm_fwd writes such rows)
 *   bias         [out_features] float, or NULL (none)
 *   residual     [rows, out_features] out_dtype, or NULL (none); y may be it
 *   y            [rows, out_features] out_dtype (GDN2_F32 or GDN2_BF16)
 *   preact       [rows, out_features] in_dtype, or NULL: receives z, rounded
 *                (not with GDN2_E4M3): what the gradient of an activation takes
 * act: none, sigmoid, silu z sigmoid(z), or gelu in its tanh form
 *   0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))).
 * e4m3 is the 8-bit float with 4 exponent and 3 mantissa bits, no infinities
 * and largest value 448. Products are exact and sums fp32, in a fixed order. Of
 * e4m3 products whose y is bf16, large ones (about 2^20 elements of y and more)
 * are added in aligned eights along k, with 13 bits below the largest of the eight
 * (the matrix instruction's way at its full rate: an error of up to 2^-13 of it
 * for each of the others); with y in fp32 all sums are fp32, at half the rate.
 * Otherwise no output overlaps an input or another output (GDN2_ERR_INVALID
 * where two pointers are one; partial overlaps are not checked).
 *
 * gdn2_linear_bwd: from dy = dL/dy (dy_dtype: the forward's out_dtype) the
 * gradients dx, dweight (in_dtype, shaped like x and weight) and dbias (float);
 * each may be NULL, not all of them. The residual's gradient is dy itself.
 * preact: the z that the forward wrote (NULL without an activation). dz =
 * dy act'(z) is rounded to in_dtype for the products; dbias sums it unrounded.
 * x may be NULL without dweight, weight without dx. in_dtype: GDN2_F32 or
 * GDN2_BF16. No output, nor the workspace, may overlap an input or another
 * output. workspace: gdn2_linear_bwd_workspace_bytes(...) of device memory.
 *
 * rows >= 0 (the gradient: up to GDN2_LINEAR_BWD_MAX_ROWS);
 * 1 <= in_features, out_features <= GDN2_LINEAR_MAX_FEATURES.
 * GDN2_ERR_UNSUPPORTED, before anything is enqueued, where two of the three
 * sizes, each rounded up to 128s, have a product of 2^37 or more. Pointers are
 * 16-byte aligned; the sizes may be any number (in_features in whole 16 bytes
 * and out_features in whole eights are faster).
 */
typedef enum {
    GDN2_ACT_NONE = 0,
    GDN2_ACT_SIGMOID = 1,
    GDN2_ACT_SILU = 2,
    GDN2_ACT_GELU_TANH = 3
} gdn2_activation;
#define GDN2_LINEAR_MAX_FEATURES (1 << 20)
#define GDN2_LINEAR_BWD_MAX_ROWS (1 << 22)
int gdn2_linear_fwd(const void *x, const void *weight, const float *bias, const void *residual, const float *x_scale,
                    const float *weight_scale, void *y, void *preact, int64_t rows, int in_features, int out_features,
                    int activation, int in_dtype, int out_dtype);
size_t gdn2_linear_bwd_workspace_bytes(int64_t rows, int in_features, int out_features, int activation, int in_dtype,
                                       int dy_dtype, int need_dx, int need_dweight, int need_dbias);
int gdn2_linear_bwd(const void *dy, const void *x, const void *weight, const void *preact, void *dx, void *dweight,
                    float *dbias, int64_t rows, int in_features, int out_features, int activation, int in_dtype,
                    int dy_dtype, void *workspace, size_t workspace_bytes);

/*
 * ---- RMS norm of x + residual, and its gradient --------------------------------
 *
 * The norm before a layer's projections, over rows of `cols` elements:
 *   h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight
 *
 *   x, residual, sum, weight   as in gdn2_layer_norm_fwd
 *   y            [rows, cols] out_dtype: GDN2_F32, GDN2_BF16, or GDN2_E4M3 with
 *   scale        [rows] float (NULL otherwise): max |y| / 448 of the row, at
 *                least 2^-126; y then holds y / scale, to nearest even, which
 *                gdn2_linear_fwd takes with this x_scale
 * y (same type) and sum may each be x or residual itself, but must not overlap
 * an input otherwise, nor each other (GDN2_ERR_INVALID where they are one). The
 * squares of a row are added in fp32: above about 1e19 their sum is infinite. A
 * NaN in h makes its row NaN; scale is then that of a row of zeros.
 *
 * gdn2_rms_norm_bwd: as gdn2_layer_norm_bwd, without a bias; dy is dL/dy in
 * out_dtype, GDN2_F32 or GDN2_BF16.
 * workspace: gdn2_rms_norm_bwd_workspace_bytes(...) of device memory.
 * Sizes, alignment and errors as in gdn2_layer_norm_fwd.
 */
int gdn2_rms_norm_fwd(const void *x, const void *residual, const float *weight, void *y, float *scale, void *sum,
                      int64_t rows, int cols, float eps, int in_dtype, int out_dtype);
size_t gdn2_rms_norm_bwd_workspace_bytes(int64_t rows, int cols);
int gdn2_rms_norm_bwd(const void *dy, const void *h, const float *weight, const void *dsum, void *dh, float *dweight,
                      int64_t rows, int cols, float eps, int in_dtype, int out_dtype, void *workspace,
                      size_t workspace_bytes);

/*
 * ---- The norm over many gradients, and their clipping ---------------------------
 *
 *   norm = sqrt(sum of g^2 over all elements of all tensors)
 *   out[i] = grads[i] * min(1, max_norm / (norm + 1e-6))
 *
 *   grads, out   host arrays of `count` device pointers; sizes: host array of
 *                element counts (0 is allowed, its pointers are then unused);
 *                dtypes, out_dtypes: host arrays of GDN2_F32 / GDN2_BF16. All are
 *                read before the call returns.
 *   norm         [1] float on the device: written, or, where norm_given is not
 *                0, read (a norm over several devices' parts, say)
 *   workspace    gdn2_clip_grads_workspace_bytes() of device memory (NULL is
 *                allowed with norm_given)
 * out[i] may be grads[i] itself with the same dtype (nothing is written there when nothing
 * is to be scaled); otherwise no out[i] may overlap any grads[j], out[j] or the
 * norm, and a norm that is written and the workspace no tensor and not each other
 * (GDN2_ERR_INVALID; checked over their whole length). Tensors lie at any
 * multiple of their element's size. Squares and their sums are fp64, in a fixed
 * order; a norm beyond the largest float is written as infinity, and scales by what
 * it is. Infinite gradients make finite ones 0 and themselves NaN; a NaN makes all
 * of them NaN. 0 <= max_norm, finite.
 */
size_t gdn2_clip_grads_workspace_bytes(void);
int gdn2_grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes, int count, float *norm,
                   void *workspace, size_t workspace_bytes);
int gdn2_clip_grads(const void *const *grads, void *const *out, const int64_t *sizes, const int32_t *dtypes,
                    const int32_t *out_dtypes, int count, float max_norm, float *norm, int norm_given, void *workspace,
                    size_t workspace_bytes);

/*
 * Per-kernel timing, for measurement tools (not needed for computing).
 * gdn2_profile_begin(max_calls) makes this thread's next gdn2_chunk_fwd /
 * gdn2_decode_step calls (up to max_calls of them, 1..4096) record a HIP
 * event before and after each kernel they launch, on the call's stream.
 * Events are created here, on the current device. gdn2_profile_end() stops
 * recording and returns the number of calls recorded (or a negative status).
 * gdn2_profile_kernel(idx, ...) then reports, for the idx-th distinct kernel
 * name in launch order, its launch count and summed duration in ms; it waits
 * for the recorded events and returns GDN2_ERR_INVALID when idx is past the
 * last kernel. `name` points to static storage.
 */
int gdn2_profile_begin(int max_calls);
int gdn2_profile_end(void);
int gdn2_profile_kernel(int idx, const char **name, int *launches, double *total_ms);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H */
