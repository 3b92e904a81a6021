// The input prologue on its own and its gradient: short causal depthwise
// convolution of 4 taps on q, k, v, unit norm of q and k over a head's
// channels, sigmoid of the gate logits (aifetchly-blog.pages.dev, "Gated
// DeltaNet-2 Guide", the "Architectural Workflow" diagram, steps 1 and 2).
//
//   y_t = bias + sum_j w_j x_{t-3+j},   q = y r,  r = 1 / max(|y|, 1e-12)
//   gate = 1 / (1 + exp(-logit))
//   backward: dy = dq (v), dy = r dq - y r^3 (y.dq) (q, k; r dq where |y| <= 1e-12)
//     dx_t = sum_j w_j dy_{t+3-j},  dw_j = sum_t dy_t x_{t-3+j},  dbias = sum_t dy_t
//     dlogit = dgate s (1 - s) = dgate e / (1 + e)^2,  e = exp(-|logit|)
//
// Bound by memory: every element is read once and written once. A thread owns
// a few neighbouring channels of one tensor (the lanes of a head are
// neighbours, and its norm a sum over them) and walks along the tokens with the
// last three inputs in registers, eight rows of loads ahead. Few channels a
// thread, so that many waves fit: forward over 32 packed sequences of up to
// 2048 tokens, 16 heads of 128, bf16: 274 us with four, 296 with eight, and 267
// (5.6 TB/s) since the histories no longer take a launch of their own; backward
// over 8 of up to 4096: 368 us with two (5.4 TB/s), 379 with four. All sums are
// fp32; outputs are rounded once.
#include "operators_launch.hpp"
#include "rows.hpp"

#include <algorithm>

namespace gdn2 {

constexpr int kNT = 256;
constexpr int kFwdV = 4, kBwdV = 2;   // channels of a thread

// Sum over aligned groups of G lanes (a power of two up to 64), in each of
// them: swaps within rows of 16 lanes, each adding the halves that hold their
// sums, and gfx950's swaps of rows beyond. All lanes of a group are active
// together; G is the same for the workgroup.
__device__ __forceinline__ float head_sum(float x, int G)
{
    auto add = [](float v, auto ctrl) {
        return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    x = add(x, std::integral_constant<int, 0xB1>{});                  // quad_perm [1,0,3,2]
    if (G >= 4) x = add(x, std::integral_constant<int, 0x4E>{});      // quad_perm [2,3,0,1]
    if (G >= 8) x = add(x, std::integral_constant<int, 0x141>{});     // row_half_mirror
    if (G >= 16) x = add(x, std::integral_constant<int, 0x140>{});    // row_mirror
    if (G >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    if (G >= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    return x;
}

// 1 / max(|y|, 1e-12) from the sum of squares, NaN where that is NaN (which a
// maximum would replace by the floor).
__device__ __forceinline__ float unit_scale(float ss) { return rsqrtf(ss < 1e-24f ? 1e-24f : ss); }

struct SeqTable {
    const int32_t *cu;   // or null: sequences of T tokens
    int T, N;            // T: tokens of a sequence, or in all
    __device__ __forceinline__ int total() const { return cu ? min(max(cu[N], 0), T) : N * T; }
    // (bounds of a table that is not what it has to be still lie within [0, T])
    __device__ __forceinline__ int start(int i) const { return cu ? (i > 0 ? min(max(cu[i], 0), T) : 0) : i * T; }
    __device__ __forceinline__ int end(int i) const { return cu ? min(max(cu[i + 1], start(i)), T) : (i + 1) * T; }
    // the first sequence behind i that ends behind token t
    __device__ __forceinline__ int next(int i, int t) const
    {
        while (i < N - 1)
            if (end(++i) > t) break;
        return i;
    }
    // the last sequence that starts at or before token t (eighths of what is
    // left at a time: the loads of a step are under way together)
    __device__ __forceinline__ int of(int t) const
    {
        if (!cu) return min(t / T, N - 1);
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int step = (hi - lo) / 8 + 1;
            int at = lo;
#pragma unroll
            for (int j = 1; j < 8; ++j) {
                const int m = min(lo + j * step, hi);
                if (cu[m] <= t) at = max(at, m);
            }
            lo = at;
            hi = min(hi, at + step - 1);
        }
        return lo;
    }
};

// V channels of one tensor and token, packed.
template <typename In, int V> struct PackV {
    In e[V] __attribute__((aligned(V * sizeof(In) > 16 ? 16 : V * sizeof(In))));
    __device__ __forceinline__ void load(const In *p)
    {
        constexpr int B = V * sizeof(In);
        if constexpr (B == 4) *reinterpret_cast<uint32_t *>(e) = *reinterpret_cast<const uint32_t *>(p);
        else if constexpr (B == 8) *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(p);
        else
#pragma unroll
            for (int i = 0; i < B / 16; ++i) reinterpret_cast<u4 *>(e)[i] = reinterpret_cast<const u4 *>(p)[i];
    }
    __device__ __forceinline__ void store(In *p) const
    {
        constexpr int B = V * sizeof(In);
        if constexpr (B == 4) *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(e);
        else if constexpr (B == 8) *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(e);
        else
#pragma unroll
            for (int i = 0; i < B / 16; ++i) reinterpret_cast<u4 *>(p)[i] = reinterpret_cast<const u4 *>(e)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = (In)0;
    }
    __device__ __forceinline__ float get(int i) const { return in2f<In>(e[i]); }
};
template <typename T> __device__ __forceinline__ T from_f(float x)
{
    if constexpr (sizeof(T) == 4) return x;
    else return (uint16_t)bf16x2(x, 0.f);
}

// One tensor's part of a launch.
struct ProTensor {
    const void *x;
    const float *w, *bias;
    const void *hin;
    void *hout;
    void *y;
    int heads, d;        // channels a token: heads * d
    int ld;              // log2 d
    // its workgroups: `per` of them pass over a tile's vectors of channels, or
    // (per = 0) one over `rows` tiles
    int block0, blocks, per, rows;
};
struct ProGate {
    const void *x;
    void *y;
    const float *dy;
    int n;               // values a token
    int block0, blocks;
};
struct ProParams {
    ProTensor t[3];
    ProGate g[2];
    SeqTable sq;
    const int32_t *slot_in, *slot_out, *commit;
    int slots, tile;     // tokens a thread walks over
    int empty0;          // first of the workgroups for sequences without tokens
};

// This thread's tile and first channel, V of them: false where it has none
// (a head's lanes always agree).
template <int V> __device__ __forceinline__ bool my_part(const ProTensor &t, int block, int64_t &tile, int &ch)
{
    const int nvec = t.heads * t.d / V;
    if (t.per > 0) {
        const int v = block % t.per * kNT + threadIdx.x;
        tile = block / t.per;
        ch = v * V;
        return v < nvec;
    }
    const int r = threadIdx.x / (unsigned)nvec;
    tile = (int64_t)block * t.rows + r;
    ch = (threadIdx.x - r * nvec) * V;
    return r < t.rows;
}

// History element j (0..2, oldest first) of sequence i for the V channels at
// ch (head ch / d), or zeros.
template <typename In, int V>
__device__ __forceinline__ void load_history(PackV<In, V> &r, const ProTensor &t, const ProParams &p, int i, int j, int ch)
{
    const int slot = p.slot_in ? p.slot_in[i] : i;
    if (t.hin && (unsigned)slot < (unsigned)p.slots)
        r.load((const In *)t.hin + ((((size_t)slot * t.heads + (ch >> t.ld)) * 3 + j) << t.ld) + (ch & (t.d - 1)));
    else r.zero();
}

// x rows p0 + 0 .. 2 (positions in the sequence, negative ones from the
// history) into win[0..2].
template <typename In, int V>
__device__ __forceinline__ void load_window(PackV<In, V> (&win)[3], const ProTensor &t, const ProParams &p, int i, int s0,
                                            int pos, int ch)
{
    const size_t W = (size_t)t.heads * t.d;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int q = pos + j;
        if (q >= 0) win[j].load((const In *)t.x + (size_t)(s0 + q) * W + ch);
        else load_history<In, V>(win[j], t, p, i, 3 + q, ch);
    }
}

// ---- forward -------------------------------------------------------------------

template <typename In>
__device__ void gate_fwd(const ProGate &gt, int64_t total, int block)
{
    const int64_t n = total * gt.n, at = ((int64_t)block * kNT + threadIdx.x) * 8;
    if (at >= n) return;
    const In *x = (const In *)gt.x + at;
    In *y = (In *)gt.y + at;
    auto one = [](float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); };
    if (at + 8 <= n) {
        PackV<In, 8> r;
        r.load(x);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = one(r.get(i));
        store8<true>(y, o);
    } else {
        for (int i = 0; i < (int)(n - at); ++i) y[i] = from_f<In>(one(in2f<In>(x[i])));
    }
}

template <typename In, int V>
__device__ __forceinline__ void store_history(const PackV<In, V> (&r)[3], const ProTensor &t, int slot, int ch)
{
#pragma unroll
    for (int j = 0; j < 3; ++j)
        r[j].store((In *)t.hout + ((((size_t)slot * t.heads + (ch >> t.ld)) * 3 + j) << t.ld) + (ch & (t.d - 1)));
}

// The history that sequence i (tokens s0 .. s0 + len - 1) leaves: the three raw
// inputs up to its last kept token, read before any is written.
template <typename In, int V>
__device__ __forceinline__ void put_history(const ProTensor &t, const ProParams &p, int i, int s0, int len, int ch)
{
    const int slot = p.slot_out ? p.slot_out[i] : (p.slot_in ? p.slot_in[i] : i);
    if ((unsigned)slot >= (unsigned)p.slots) return;
    const int keep = p.commit ? min(max(p.commit[i], 0), len) : len;
    PackV<In, V> r[3];
    load_window<In, V>(r, t, p, i, s0, keep - 3, ch);
    store_history<In, V>(r, t, slot, ch);
}

// A sequence without tokens: its history goes from slot to slot. One workgroup
// a sequence, 8 elements a thread.
template <typename In> __device__ void empty_history(const ProParams &p, int i)
{
    if (p.sq.end(i) != p.sq.start(i)) return;
    const int in = p.slot_in ? p.slot_in[i] : i, out = p.slot_out ? p.slot_out[i] : in;
    if ((unsigned)out >= (unsigned)p.slots) return;
    for (int z = 0; z < 3; ++z) {
        const ProTensor &t = p.t[z];
        const size_t n = (size_t)t.heads * t.d * 3;
        if (t.hin == t.hout && in == out) continue;
        for (size_t c = threadIdx.x * 8; c < n; c += kNT * 8) {
            PackV<In, 8> r;
            r.zero();
            if (t.hin && (unsigned)in < (unsigned)p.slots) r.load((const In *)t.hin + in * n + c);
            r.store((In *)t.hout + out * n + c);
        }
    }
}

// OWN: the thread's tile is one whole sequence (short ones), and it also
// writes the sequence's new history, after reading the old one. Otherwise
// tiles cut sequences, and the thread in whose tile a sequence begins takes its
// first three tokens whole, so that it alone reads the history, and writes the
// new one (which may take the old one's place).
template <typename In, bool OWN>
__global__ __launch_bounds__(kNT) void prologue_fwd_kernel(ProParams p)
{
    constexpr int V = kFwdV, U = OWN ? 4 : 8;   // U: rows of loads ahead
    const int total = p.sq.total();
    const int bid = blockIdx.x;
#pragma unroll
    for (int z = 0; z < 2; ++z)
        if (bid >= p.g[z].block0 && bid < p.g[z].block0 + p.g[z].blocks) {
            gate_fwd<In>(p.g[z], total, bid - p.g[z].block0);
            return;
        }
    if (!OWN && bid >= p.empty0) {
        empty_history<In>(p, bid - p.empty0);
        return;
    }
    const int z = bid >= p.t[2].block0 ? 2 : (bid >= p.t[1].block0 ? 1 : 0);
    const ProTensor &t = p.t[z];
    const size_t W = (size_t)t.heads * t.d;
    const int G = t.d / V;
    int64_t tl;
    int ch;
    if (!my_part<V>(t, bid - t.block0, tl, ch)) return;
    int i, tb, te, s0, s1, first = 0, bound = 0;   // sequences from `first` that begin before `bound` begin here
    if (OWN) {
        if (tl >= p.sq.N) return;   // (a head's lanes leave together)
        i = (int)tl;
        s0 = tb = p.sq.start(i);
        s1 = te = p.sq.end(i);
    } else {
        if (tl * p.tile >= total) return;
        tb = (int)(tl * p.tile);
        te = min(tb + p.tile, total);
        i = p.sq.of(tb);
        s0 = p.sq.start(i);
        s1 = p.sq.end(i);
        first = s0 < tb ? i + 1 : i;
        bound = te;
        if (s0 < tb) tb = max(tb, min(s0 + 3, s1));
        if (tb >= te) return;
        const int il = te <= s1 ? i : p.sq.next(i, te - 1), sl = p.sq.start(il);
        if (sl >= tb) te = max(te, min(sl + 3, p.sq.end(il)));
    }
    const In *x = (const In *)t.x;
    In *y = (In *)t.y;
    f4 tap[V];
    float bias[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        tap[c] = *reinterpret_cast<const f4 *>(t.w + 4 * (size_t)(ch + c));
        bias[c] = t.bias ? t.bias[ch + c] : 0.f;
    }
    PackV<In, V> win[3];
    float old[3][V];   // win as numbers
    auto numbers = [&]() {
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) old[j][c] = win[j].get(c);
    };
    if (OWN) {
        load_window<In, V>(win, t, p, i, s0, -3, ch);
    } else if (s0 < tb && tb < s1) {   // in the midst of a sequence: behind its first three tokens
#pragma unroll
        for (int j = 0; j < 3; ++j) win[j].load(x + (size_t)(tb - 3 + j) * W + ch);
    } else {                           // a sequence begins, this or a later one: the loop opens it
#pragma unroll
        for (int j = 0; j < 3; ++j) win[j].zero();
        if (s0 == tb) --i;
        s1 = tb;
    }
    numbers();
    PackV<In, V> nxt[U];
    if (tb < te)
#pragma unroll
        for (int u = 0; u < U; ++u) nxt[u].load(x + (size_t)min(tb + u, te - 1) * W + ch);
    for (int tok = tb; tok < te; tok += U) {
        PackV<In, V> cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = nxt[u];
#pragma unroll
        for (int u = 0; u < U; ++u) nxt[u].load(x + (size_t)min(tok + U + u, te - 1) * W + ch);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = tok + u;
            if (at < te) {
                if (!OWN && at >= s1) {   // the next sequence with tokens
                    i = p.sq.next(i, at);
                    s0 = p.sq.start(i);
                    s1 = p.sq.end(i);
                    load_window<In, V>(win, t, p, i, s0, -3, ch);
                    numbers();
                }
                float o[V], ss = 0.f;
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const float now = cur[u].get(c);
                    o[c] = bias[c] + tap[c][0] * old[0][c] + tap[c][1] * old[1][c] + tap[c][2] * old[2][c] +
                           tap[c][3] * now;
                    ss += o[c] * o[c];
                    old[0][c] = old[1][c];
                    old[1][c] = old[2][c];
                    old[2][c] = now;
                }
                if (z < 2) {
                    const float r = unit_scale(head_sum(ss, G));
#pragma unroll
                    for (int c = 0; c < V; ++c) o[c] *= r;
                }
                PackV<In, V> out;
#pragma unroll
                for (int c = 0; c < V; ++c) out.e[c] = from_f<In>(o[c]);
                out.store(y + (size_t)at * W + ch);
                if (OWN) {
                    win[0] = win[1];
                    win[1] = win[2];
                    win[2] = cur[u];
                }
            }
        }
    }
    if (OWN && t.hout) {
        const int slot = p.slot_out ? p.slot_out[i] : (p.slot_in ? p.slot_in[i] : i);
        if ((unsigned)slot >= (unsigned)p.slots) return;
        const int keep = p.commit ? min(max(p.commit[i], 0), te - tb) : te - tb;
        // (win holds the last three inputs, or the old history's)
        if (keep < te - tb) load_window<In, V>(win, t, p, i, tb, keep - 3, ch);
        store_history<In, V>(win, t, slot, ch);
    } else if (t.hout) {
        for (int j = first; j < p.sq.N && p.sq.start(j) < bound; ++j) {
            const int b = p.sq.start(j), len = p.sq.end(j) - b;
            if (len > 0) put_history<In, V>(t, p, j, b, len, ch);
        }
    }
}

// ---- backward ------------------------------------------------------------------

struct ProBwdParams {
    ProParams f;
    const float *dy[3];
    void *dx[3];
    float *part[3];      // [tiles][5 * channels]: 4 tap sums a channel, then the bias sums
};

template <typename In, typename Out>
__device__ void gate_bwd(const ProGate &gt, int64_t total, int block)
{
    const int64_t n = total * gt.n, at = ((int64_t)block * kNT + threadIdx.x) * 8;
    if (at >= n) return;
    const In *x = (const In *)gt.x + at;
    const float *dy = gt.dy + at;
    Out *dx = (Out *)gt.y + at;
    // s (1 - s), with no difference of s from one to take: exact to a few units
    // also where s rounds to one
    auto one = [](float z, float d) {
        const float e = __expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.f + e);
        return d * e * (r * r);
    };
    if (at + 8 <= n) {
        PackV<In, 8> r;
        PackV<float, 8> d;
        r.load(x);
        d.load(dy);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = one(r.get(i), d.e[i]);
        store8<true>(dx, o);
    } else {
        for (int i = 0; i < (int)(n - at); ++i) dx[i] = from_f<Out>(one(in2f<In>(x[i]), dy[i]));
    }
}

template <typename In, typename Out>
__global__ __launch_bounds__(kNT) void prologue_bwd_kernel(ProBwdParams p)
{
    constexpr int V = kBwdV, U = 8;
    const int total = p.f.sq.total();
    const int bid = blockIdx.x;
#pragma unroll
    for (int z = 0; z < 2; ++z)
        if (bid >= p.f.g[z].block0 && bid < p.f.g[z].block0 + p.f.g[z].blocks) {
            gate_bwd<In, Out>(p.f.g[z], total, bid - p.f.g[z].block0);
            return;
        }
    const int z = bid >= p.f.t[2].block0 ? 2 : (bid >= p.f.t[1].block0 ? 1 : 0);
    const ProTensor &t = p.f.t[z];
    const size_t W = (size_t)t.heads * t.d;
    const int G = t.d / V;
    int64_t tl;
    int ch;
    if (!my_part<V>(t, bid - t.block0, tl, ch)) return;
    // every tile up to the last token the sizes allow has its partial row;
    // those behind the last sequence write zeros
    if (tl * p.f.tile >= (p.f.sq.cu ? (int64_t)p.f.sq.T : (int64_t)p.f.sq.N * p.f.sq.T)) return;
    f4 dw[V];
    float db[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        dw[c] = f4zero();
        db[c] = 0.f;
    }
    if (tl * p.f.tile < total) {
        const int tb = (int)(tl * p.f.tile), te = min(tb + p.f.tile, total);
        const In *x = (const In *)t.x;
        const float *dy = p.dy[z];
        Out *dx = (Out *)p.dx[z];
        f4 tap[V];
        float bias[V], a[3][V];   // a[j]: what is known of dx of the token j + 1 back
#pragma unroll
        for (int c = 0; c < V; ++c) {
            tap[c] = *reinterpret_cast<const f4 *>(t.w + 4 * (size_t)(ch + c));
            bias[c] = t.bias ? t.bias[ch + c] : 0.f;
            a[0][c] = a[1][c] = a[2][c] = 0.f;
        }
        int i = p.f.sq.of(tb), s0 = p.f.sq.start(i), s1 = p.f.sq.end(i);
        float old[3][V];   // the three inputs before a token
        auto window = [&](int pos) {
            PackV<In, V> win[3];
            load_window<In, V>(win, t, p.f, i, s0, pos, ch);
#pragma unroll
            for (int j = 0; j < 3; ++j)
#pragma unroll
                for (int c = 0; c < V; ++c) old[j][c] = win[j].get(c);
        };
        window(tb - s0 - 3);
        // up to three tokens past the tile, of the sequence of its last one
        const int il = p.f.sq.of(te - 1);
        const int th = max(te, min(te + 3, p.f.sq.end(il)));
        PackV<In, V> nx[U];
        PackV<float, V> nd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            nx[u].load(x + (size_t)min(tb + u, th - 1) * W + ch);
            nd[u].load(dy + (size_t)min(tb + u, th - 1) * W + ch);
        }
        for (int tok = tb; tok < th; tok += U) {
            PackV<In, V> cx[U];
            PackV<float, V> cd[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                cx[u] = nx[u];
                cd[u] = nd[u];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                nx[u].load(x + (size_t)min(tok + U + u, th - 1) * W + ch);
                nd[u].load(dy + (size_t)min(tok + U + u, th - 1) * W + ch);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = tok + u;
                if (at < th) {
                    if (at >= s1) {
                        i = p.f.sq.next(i, at);
                        s0 = p.f.sq.start(i);
                        s1 = p.f.sq.end(i);
                        window(-3);
                    }
                    float d[V], now[V];
#pragma unroll
                    for (int c = 0; c < V; ++c) {
                        d[c] = cd[u].e[c];
                        now[c] = cx[u].get(c);
                    }
                    if (z < 2) {
                        float y[V], ss = 0.f, yd = 0.f;
#pragma unroll
                        for (int c = 0; c < V; ++c) {
                            y[c] = bias[c] + tap[c][0] * old[0][c] + tap[c][1] * old[1][c] + tap[c][2] * old[2][c] +
                                   tap[c][3] * now[c];
                            ss += y[c] * y[c];
                            yd += y[c] * d[c];
                        }
                        ss = head_sum(ss, G);
                        yd = head_sum(yd, G);
                        const float r = unit_scale(ss);
                        // (r y).dq along the unit vector; none where the norm is at its floor
                        const float m = ss <= 1e-24f ? 0.f : r * yd * r;
#pragma unroll
                        for (int c = 0; c < V; ++c) d[c] = r * (d[c] - m * y[c]);
                    }
                    if (at < te) {
#pragma unroll
                        for (int c = 0; c < V; ++c) {
                            dw[c][0] += d[c] * old[0][c];
                            dw[c][1] += d[c] * old[1][c];
                            dw[c][2] += d[c] * old[2][c];
                            dw[c][3] += d[c] * now[c];
                            db[c] += d[c];
                        }
                    }
                    // dx of the token three back is complete; the others move up
                    float o[V];
#pragma unroll
                    for (int c = 0; c < V; ++c) {
                        o[c] = a[2][c] + tap[c][0] * d[c];
                        a[2][c] = a[1][c] + tap[c][1] * d[c];
                        a[1][c] = a[0][c] + tap[c][2] * d[c];
                        a[0][c] = tap[c][3] * d[c];
                    }
                    const int low = max(tb, s0);
                    auto put = [&](int to, const float *v) {
                        if (to >= low && to < te) {
                            PackV<Out, V> r;
#pragma unroll
                            for (int c = 0; c < V; ++c) r.e[c] = from_f<Out>(v[c]);
                            r.store(dx + (size_t)to * W + ch);
                        }
                    };
                    put(at - 3, o);
                    if (at == s1 - 1) {   // the sequence's last token: nothing follows
                        put(at - 2, a[2]);
                        put(at - 1, a[1]);
                        put(at, a[0]);
#pragma unroll
                        for (int c = 0; c < V; ++c) a[0][c] = a[1][c] = a[2][c] = 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < V; ++c) {
                        old[0][c] = old[1][c];
                        old[1][c] = old[2][c];
                        old[2][c] = now[c];
                    }
                }
            }
        }
    }
    float *part = p.part[z] + (size_t)tl * 5 * W;
#pragma unroll
    for (int c = 0; c < V; ++c) *reinterpret_cast<f4 *>(part + 4 * (size_t)(ch + c)) = dw[c];
    PackV<float, V> b;
#pragma unroll
    for (int c = 0; c < V; ++c) b.e[c] = db[c];
    b.store(part + 4 * W + ch);
}

// ---- launch --------------------------------------------------------------------

static int64_t tokens_of(const PrologueArgs &a) { return a.cu_seqlens ? (int64_t)a.T : (int64_t)a.N * a.T; }

// A launch takes fewer than 2^32 threads.
constexpr int64_t kMostBlocks = 0xFFFFFFFFLL / kNT;

// blocks: how many workgroups these take (the parameters hold their numbers
// where it is at most kMostBlocks)
static ProParams pro_params(const PrologueArgs &a, int V, int64_t tiles, int tile, int64_t *blocks)
{
    ProParams p = {};
    int64_t at = 0;
    for (int z = 0; z < 3; ++z) {
        ProTensor &t = p.t[z];
        t.x = a.x[z];
        t.w = a.weight[z];
        t.bias = a.bias[z];
        t.hin = a.hist_in[z];
        t.hout = a.hist_out[z];
        t.y = a.y[z];
        t.heads = a.heads[z];
        t.d = a.d[z];
        t.ld = __builtin_ctz(t.d);
        const int nvec = t.heads * t.d / V;
        t.per = nvec >= kNT ? (nvec + kNT - 1) / kNT : 0;
        t.rows = nvec >= kNT ? 0 : kNT / nvec;
        const int64_t n = t.per ? tiles * t.per : (tiles + t.rows - 1) / t.rows;
        t.block0 = (int)at;
        t.blocks = (int)n;
        at += n;
    }
    for (int z = 0; z < 2; ++z) {
        ProGate &g = p.g[z];
        g.x = a.logit[z];
        g.y = a.gate[z];
        g.n = a.nlogit[z];
        const int64_t n = (tokens_of(a) * g.n + 8 * kNT - 1) / (8 * kNT);
        g.block0 = (int)at;
        g.blocks = (int)n;
        at += n;
    }
    p.sq = {a.cu_seqlens, a.T, a.N};
    p.slot_in = a.slot_in;
    p.slot_out = a.slot_out;
    p.commit = a.commit;
    p.slots = a.slots;
    p.tile = tile;
    *blocks = at;
    return p;
}

// Tokens a thread of V channels walks over: as many as leave 12 waves a compute
// unit, between `least` and `most` (a tile reads three rows before its own,
// backward also three after it). Backward, 4 x 2048 tokens, 16 heads of 128,
// fp32: 199 us so, 248 with 8 waves, 210 with 16; 300 bf16 tokens: 16.6 us with
// 8 tokens a tile, 18.9 with 16. Forward, 300 bf16 tokens of one sequence: 10 us,
// 22 with tiles of 64.
static int tile_of(long long tokens, long long channels, int V, long long least, long long most)
{
    const long long t = tokens * (channels / V) / (256LL * 12 * 64);
    return (int)std::max(std::max(1LL, least), std::min(most, t));
}
int prologue_bwd_tile(long long tokens, long long channels) { return tile_of(tokens, channels, kBwdV, 8, 256); }

// Sequences of at most this many tokens are walked by one thread a channel
// group each, which then also writes their histories (one launch).
constexpr int kOwnTokens = 16;

template <typename In> static hipError_t prologue_fwd_t(const PrologueArgs &a, hipStream_t st)
{
    const bool own = a.T <= kOwnTokens, hist = a.hist_out[0] != nullptr;
    const int64_t tokens = tokens_of(a);
    int64_t channels = 0;
    for (int z = 0; z < 3; ++z) channels += a.heads[z] * a.d[z];
    // (a tile's sequences come one after the other, so no more than two of them on
    // average: 256 packed sequences of one token 16 us, 21 with tiles of 8 tokens,
    // and 19 with a tile each)
    const int tile = tile_of(tokens, channels, kFwdV, std::min<long long>(4, tokens / a.N),
                             std::min<long long>(64, 2 * tokens / a.N));
    int64_t blocks = 0;
    ProParams p = pro_params(a, kFwdV, own ? a.N : (tokens + tile - 1) / tile, tile, &blocks);
    p.empty0 = (int)blocks;
    if (!own && hist && a.cu_seqlens) blocks += a.N;
    if (blocks == 0 || (tokens == 0 && !hist)) return hipSuccess;
    if (blocks > kMostBlocks) return hipErrorInvalidConfiguration;
    prof_before("gdn2_prologue_fwd", st);
    if (own) hipLaunchKernelGGL((prologue_fwd_kernel<In, true>), dim3((unsigned)blocks), dim3(kNT), 0, st, p);
    else hipLaunchKernelGGL((prologue_fwd_kernel<In, false>), dim3((unsigned)blocks), dim3(kNT), 0, st, p);
    prof_after(st);
    return hipGetLastError();
}

hipError_t launch_prologue_fwd(const PrologueArgs &a, hipStream_t st)
{
    return a.bf16 ? prologue_fwd_t<uint16_t>(a, st) : prologue_fwd_t<float>(a, st);
}

size_t prologue_bwd_workspace(long long tokens, long long channels)
{
    const long long tile = prologue_bwd_tile(tokens, channels);
    return (size_t)((tokens + tile - 1) / tile) * 5 * channels * sizeof(float);
}

template <typename In, typename Out> static hipError_t prologue_bwd_t(const PrologueBwdArgs &a, hipStream_t st)
{
    const int64_t tokens = tokens_of(a.f);
    int64_t channels = 0;
    for (int z = 0; z < 3; ++z) channels += a.f.heads[z] * a.f.d[z];
    const int tile = prologue_bwd_tile(tokens, channels);
    const int64_t tiles = (tokens + tile - 1) / tile;
    int64_t blocks = 0;
    ProBwdParams p = {};
    p.f = pro_params(a.f, kBwdV, tiles, tile, &blocks);
    if (blocks > kMostBlocks) return hipErrorInvalidConfiguration;
    float *part = (float *)a.workspace;
    ColumnSums cs = {};
    for (int z = 0; z < 3; ++z) {
        const int W = a.f.heads[z] * a.f.d[z];
        p.dy[z] = a.dy[z];
        p.dx[z] = a.dx[z];
        p.part[z] = part;
        cs.part[z] = part;
        cs.out0[z] = a.dweight[z];
        cs.out1[z] = a.dbias[z];
        cs.n0[z] = 4 * W;
        cs.n1[z] = W;
        part += (size_t)tiles * 5 * W;
    }
    for (int z = 0; z < 2; ++z) {
        p.f.g[z].y = a.dlogit[z];
        p.f.g[z].dy = a.dgate[z];
    }
    if (blocks > 0) {
        prof_before("gdn2_prologue_bwd", st);
        hipLaunchKernelGGL((prologue_bwd_kernel<In, Out>), dim3((unsigned)blocks), dim3(kNT), 0, st, p);
        prof_after(st);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    cs.parts = (int)tiles;
    cs.jobs = 3;
    return launch_column_sums(cs, "gdn2_prologue_reduce", st);
}

hipError_t launch_prologue_bwd(const PrologueBwdArgs &a, hipStream_t st)
{
    if (a.f.bf16) return a.out_bf16 ? prologue_bwd_t<uint16_t, uint16_t>(a, st) : prologue_bwd_t<uint16_t, float>(a, st);
    return a.out_bf16 ? prologue_bwd_t<float, uint16_t>(a, st) : prologue_bwd_t<float, float>(a, st);
}

} // namespace gdn2
