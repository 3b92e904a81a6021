// The gated delta rule over short runs of tokens (one token a sequence up to
// a few dozen), states in a pool of slots: the serving form of the recurrence
// (snilld.dk, "Hvad Gated DeltaNet-2 ændrer", update equation) between the
// single-token step on a dense state array and the 64-token chunks.
//
//   S~ = Diag(alpha_t) S,  delta_t = w_t*v_t - S~^T (b_t*k_t),
//   S = S~ + k_t delta_t^T,  o_t = S^T q_t
//
// Tokens go through in blocks of up to 8. With D_t the product of the
// block's alphas up to t, a block of start state S0 is
//   A_ts = (b_t k_t D_t) . (k_s / D_s)  (t > s),  P_ts = (q_t D_t) . (k_s / D_s)  (t >= s)
//   R_E = (b k D) S0, R_Q = (q D) S0, X = (I + A)^-1
//   Delta = X (U - R_E),  O = R_Q + P Delta
//   S = D_8 S0 + (k_t D_8 / D_t)^T Delta
// Decays are running products of alphas, so log alpha may be anything down to
// -inf (a full forget); the quotients need D_s >= 2^-60 (the
// products then stay far from the smallest floats), and a block with less is
// cut in half, down to a single token, which has none. All of it is
// fp32, the products on the fp32 matrix instruction. Products with the zeros
// above a triangle are harmless but for values that are not finite: blocks
// with such tokens are cut, and products that overflow are formed anew, a
// token at a time.
//
// A workgroup of dv/16 waves (or half as many) owns the state of one (sequence,
// head), or half its columns, a wave 16 of them in registers: tile r, lane n +
// 16g holds rows 16r + 4g + j of column n, which is the accumulator layout, and
// with element j of a 16-deep fragment on row 4g + j also the right operand's.
// The block's 16 left rows are
// ordered so that rows 4g .. 4g+3 are the erase rows of tokens g and g+4 and
// their query rows: the first product leaves in each lane just what the second
// one (by X, then P,) takes as its right operand, which leaves Delta where the
// third one (by the decayed keys) takes it. The state thus never moves between
// lanes and is read and written once however many tokens follow, which is what
// the operator is bound by: 8 bytes a state element.
//
// Measured at 128 x 128 heads (bf16 inputs): 256 sequences x 16 heads, one
// token, 110 us (4.9 TB/s; the same bytes multiplied in place by a library
// kernel 91 us); 128 sequences x 32 heads of 0 to 8 tokens, part committed,
// 90 us (5.4 TB/s). With more tokens a sequence the blocks come one after the
// other: about 2.6 us a block of one chain alone, some 6500 cycles, of which
// a quarter prepares the rows, an eighth forms X in one wave, and the matrix
// products need 1900; 256 x 16 chains of 64 tokens 418 us; 48 sequences x 16
// heads of up to 64 fp32 tokens (128 x 64) 42 us, a third of them at the matrix
// cores' rate.
// A block that is cut leaves no longer blocks to the rest of its sequence: 48 x
// 16 chains of 64 fp32 tokens (128 x 64) 55 us, 92 with four channels at e^-8 a
// token, 317 with one channel forgotten at the fifth token.
#pragma once

#include "operators_launch.hpp"
#include "rows.hpp"

#include <type_traits>

namespace gdn2 {

constexpr int kRecTokens = 8;   // tokens of a block

__device__ __forceinline__ f4 mfma4(float a, float b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Left row of token t's erase row; its query row is two further.
__device__ __forceinline__ constexpr int rec_row(int t) { return t < 4 ? 4 * t : 4 * (t - 4) + 1; }

struct RecParams {
    const void *q, *k, *v, *b, *w;
    const float *la;
    float *state;
    const int32_t *slot_in, *slot_out, *commit, *cu;
    void *o;
    int T, H, HK, slots, gates, out_bf16;
};

// Four elements as they lie in memory.
template <typename In> struct Raw4;
template <> struct Raw4<uint16_t> {
    uint2 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ f4 get() const
    {
        f4 x = {__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                __uint_as_float(r.y & 0xFFFF0000u)};
        return x;
    }
};
template <> struct Raw4<float> {
    f4 r;
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const f4 *>(p); }
    __device__ __forceinline__ f4 get() const { return r; }
};

template <typename In, int DK, int DV, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW == 1 ? 1 : NW < 4 ? 3 : 4))) void recurrent_kernel(RecParams a)
{
    constexpr int C = kRecTokens, NT = 64 * NW, NR = DK / 16, WGC = DV / (16 * NW);   // WGC: workgroups of a chain
    constexpr int XS = DK + 4;    // row stride of the fragment tiles (16-byte rows)
    // A lane takes four channels of a token, a wave 8 tokens of 32 channels
    constexpr int C4 = DK / 4, NCH = (DK + 31) / 32, IPT = (NCH + NW - 1) / NW;
    constexpr int NAP = NW < NR ? NW : NR;   // waves that share the products for A and P
    __shared__ __align__(16) float sX[16][XS], sKi[C][XS], sKh[2][C][XS], sG[2][DK], sPart[NAP][4][C][4];
    __shared__ float sM[16][C + 1];
    __shared__ int2 sFlag[2];   // of even and odd blocks: x: a value is not finite, y: a wide decay

    const int chain = blockIdx.x / WGC, i = chain / a.H, h = chain % a.H;
    const int col0 = blockIdx.x % WGC * 16 * NW;
    const int hk = h / (a.H / a.HK);
    const int tid = threadIdx.x, lane = tid & 63, wv = wave_id();
    const int n = lane & 15, g = lane >> 4;
    const int col = col0 + 16 * wv + n;

    int t0, t1;
    if (a.cu) {
        t0 = min(max(a.cu[i], 0), a.T);
        t1 = min(max(a.cu[i + 1], t0), a.T);
    } else {
        t0 = i * a.T;
        t1 = t0 + a.T;
    }
    // (one value for the workgroup, kept in scalar registers)
    t0 = __builtin_amdgcn_readfirstlane(t0);
    t1 = __builtin_amdgcn_readfirstlane(t1);
    const int len = t1 - t0;
    const int commit = __builtin_amdgcn_readfirstlane(a.commit ? min(max(a.commit[i], 0), len) : len);
    const int sin = __builtin_amdgcn_readfirstlane(a.slot_in ? a.slot_in[i] : i);
    const int sout = __builtin_amdgcn_readfirstlane(a.slot_out ? a.slot_out[i] : sin);
    const bool has_in = (unsigned)sin < (unsigned)a.slots, has_out = (unsigned)sout < (unsigned)a.slots;
    // nothing to say and nothing to move
    if (len == 0 && (!has_out || sin == sout)) return;

    const In *q = (const In *)a.q, *k = (const In *)a.k, *v = (const In *)a.v, *b = (const In *)a.b,
             *w = (const In *)a.w;
    const bool asc = a.gates & kGateAlpha, bsc = a.gates & kGateB, wsc = a.gates & kGateW;
    // Raw rows: loads only, so that all of a block's are under way together;
    // what they hold is made of them afterwards.
    struct Item {
        Raw4<In> k, q, b;
        f4 la;
        In b1;       // gates of one value a head
        float la1;
    };
    // A token's rows lie a scalar base and a small lane offset away: `off`
    // tokens behind token tok (the same for the workgroup).
    const int wk = a.HK * DK, wh = a.H * DK, wvw = a.H * DV;
    // (in bytes: 32 of them are enough for a block)
    auto at = [](auto *p, unsigned n) {
        using T = std::remove_reference_t<decltype(*p)>;
        using B = std::conditional_t<std::is_const_v<T>, const char, char>;
        return reinterpret_cast<T *>(reinterpret_cast<B *>(p) + n * (unsigned)sizeof(T));
    };
    // the four channels at c. Both forms of a gate are loaded, the one that is
    // not there from rows that are: a branch around a load would make the
    // wave wait for it there.
    auto load_item = [&](int tok, int off, int c, Item &x) {
        const size_t ih = (size_t)tok * a.H + h, ik = ((size_t)tok * a.HK + hk) * DK;
        const unsigned ok = off * wk + c, oh = off * wh + c, o1 = off * a.H;
        x.k.load(at(k + ik, ok));
        x.q.load(at(q + ik, ok));
        x.b.load(at(bsc ? k + ik : b + ih * DK, bsc ? ok : oh));
        x.b1 = *at(bsc ? b + ih : k + ik, bsc ? o1 : 0);
        x.la = *reinterpret_cast<const f4 *>(at(asc ? a.state : a.la + ih * DK, asc ? 0 : oh));
        x.la1 = *at(a.la + (asc ? ih : ih * DK), asc ? o1 : 0);
    };
    // k, q, b*k and alpha
    auto make_item = [&](const Item &x, f4 &kk, f4 &qq, f4 &bb, f4 &dd) {
        kk = x.k.get();
        qq = x.q.get();
        const f4 bw = x.b.get();
        const float b1 = in2f<In>(x.b1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bb[e] = (bsc ? b1 : bw[e]) * kk[e];
            dd[e] = __expf(asc ? x.la1 : x.la[e]);
        }
    };
    // v and w of this lane's column
    struct Col {
        In v, w;
    };
    auto load_u = [&](int tok, int off, int col, Col &x) {
        const size_t ih = (size_t)tok * a.H + h;
        x.v = *at(v + ih * DV, off * wvw + col);
        x.w = *at(w + (wsc ? ih : ih * DV), wsc ? off * a.H : off * wvw + col);
    };
    auto make_u = [&](const Col &x) { return in2f<In>(x.v) * in2f<In>(x.w); };
    auto put_o = [&](int tok, int off, int col, float x) {
        const size_t io = ((size_t)tok * a.H + h) * DV;
        const unsigned to = off * wvw + col;
        if (a.out_bf16) *at((uint16_t *)a.o + io, to) = (uint16_t)bf16x2(x, 0.f);
        else *at((float *)a.o + io, to) = x;
    };

    const size_t own = (size_t)h * DK * DV, slot_sz = (size_t)a.H * DK * DV;
    f4 S[NR];
    if (has_in) {
        const float *sp = a.state + sin * slot_sz + own + 4 * g * DV + col;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[r][j] = sp[(16 * r + j) * DV];
    } else {
#pragma unroll
        for (int r = 0; r < NR; ++r) S[r] = f4zero();
    }
    auto keep = [&]() {
        if (!has_out) return;
        // (formed here: as loop invariants the rows' addresses would fill 64 registers)
        int at = 4 * g * DV + col;
        asm volatile("" : "+v"(at));
        float *sp = a.state + sout * slot_sz + own + at;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) sp[(16 * r + j) * DV] = S[r][j];
    };
    // sum over the four rows of 16 lanes
    auto across = [](float v) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return __uint_as_float(b[0]) + __uint_as_float(b[1]);
    };
    // row `row` (of lane n) of sX times the state, in two chains of products
    auto left_product = [&](int row) {
        f4 R[2] = {f4zero(), f4zero()};
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            R[r & 1] = Mma<float>::mma(*reinterpret_cast<const f4 *>(&sX[row][16 * r + 4 * g]), S[r], R[r & 1]);
        }
        return R[0] + R[1];
    };
    if (commit == 0 && sin != sout) keep();
    if (len == 0) return;   // (no token to load)

    if (len == 1) {
        // ---- a single token: Delta = U - R_E, O = R_Q + (q.k) Delta
        Col cu;
        load_u(t0, 0, col, cu);
        if (tid < C4) {
            Item x;
            f4 kk, qq, bb, dd;
            load_item(t0, 0, 4 * tid, x);
            make_item(x, kk, qq, bb, dd);
            *reinterpret_cast<f4 *>(&sX[0][4 * tid]) = bb * dd;
            *reinterpret_cast<f4 *>(&sX[2][4 * tid]) = qq * dd;
            *reinterpret_cast<f4 *>(&sKh[0][0][4 * tid]) = kk;
            *reinterpret_cast<f4 *>(&sKi[0][4 * tid]) = qq;
            *reinterpret_cast<f4 *>(&sG[0][4 * tid]) = dd;
        }
        __syncthreads();
        float kq = 0.f;
#pragma unroll
        for (int c = 0; c < DK; c += 64)
            if (DK >= 64 || lane < DK) kq += sKh[0][0][c + lane] * sKi[0][c + lane];
        kq = lane_group_sum<64>(kq);
        // rows 0 and 2 are the token's; all others repeat one of them
        const f4 R = left_product(n & 2);
        const float d = make_u(cu) - R[0];
        if (commit == 1 && has_out) {
            const float dg = g == 0 ? d : 0.f;
#pragma unroll
            for (int r = 0; r < NR; ++r)
                S[r] = mfma4(sKh[0][0][16 * r + n], dg, S[r] * *reinterpret_cast<const f4 *>(&sG[0][16 * r + 4 * g]));
            keep();
        }
        if (g == 0) put_o(t0, 0, col, R[2] + kq * d);
        return;
    }

    // Tokens of a block. A block is done again with fewer tokens where
    //  - a token holds a NaN or an infinity: the products multiply what comes
    //    after a token by zeros, which hides any other number. First without a
    //    draft's end (its committed part stays one block), then token by token;
    //  - a channel decays by more than 2^60 within it: A and P are formed as
    //    products of rows decayed from the block's start and keys divided by
    //    that decay (nor may a key overflow by it). Half the tokens, down to
    //    one, which needs neither.
    int most = C, L = 0, par = 0;
    // A block ends at the committed prefix, whose state is kept, but for the
    // last one, whose later tokens then leave the state alone. (Also one that
    // was cut: it may no longer be the last.)
    auto length = [&](int done) {
        const int rem = len - done;
        return rem <= most ? rem : min(most, done < commit ? commit - done : rem);
    };
    Item x[IPT];
    Col cu[2];
    auto load_block = [&](int tb, int L, int lane) {
#pragma unroll
        for (int m = 0; m < IPT; ++m) {
            const int c = (wv + m * NW) * 32 + (lane & 7) * 4;
            if (NCH % NW == 0 || wv + m * NW < NCH) load_item(tb, min(lane >> 3, L - 1), DK < 32 ? c % DK : c, x[m]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) load_u(tb, min((lane >> 4) + 4 * j, L - 1), col0 + 16 * wv + (lane & 15), cu[j]);
    };
    // Of the products of d over a channel's 8 tokens (lanes 8 apart): up to the
    // lane's token, and of all. Each step joins the groups of tokens that
    // differ in one bit.
    auto scan = [&](const f4 &d, f4 &up, f4 &all, int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float p = d[e], t = d[e];
            const float o8 = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(t), 0x128, 0xF, 0xF, false));   // row_ror:8
            p *= lane & 8 ? o8 : 1.f;
            t *= o8;
            const auto a16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(t), __float_as_uint(t), false, false);
            const float e16 = __uint_as_float(a16[0]), f16 = __uint_as_float(a16[1]);   // of the even row, of the odd one
            p *= lane & 16 ? e16 : 1.f;
            t = e16 * f16;
            const auto a32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(t), __float_as_uint(t), false, false);
            const float e32 = __uint_as_float(a32[0]), f32 = __uint_as_float(a32[1]);
            p *= lane & 32 ? e32 : 1.f;
            up[e] = p;
            all[e] = e32 * f32;
        }
    };
    if (tid < 2) sFlag[tid] = make_int2(0, 0);
    L = length(0);
    load_block(t0, L, lane);
    __syncthreads();
    for (int done = 0; done < len; par ^= 1) {
        int lane = tid & 63;
        // (the lane's addresses are formed anew in each block: kept over the
        // loop they would take a third of the registers)
        asm volatile("" : "+v"(lane));
        const int n = lane & 15, g = lane >> 4, col = col0 + 16 * wv + n;
        const int tb = t0 + done;
        // ---- the block's rows; tokens past it are zeros that decay nothing
        // (those whose effect stays: all but those of a draft's end)
        const int stay = done + L < len ? L : min(max(commit - done, 0), L);
        float bad = 0.f;
        bool wide = false;
#pragma unroll
        for (int m = 0; m < IPT; ++m) {
            const int t = lane >> 3, c = (wv + m * NW) * 32 + (lane & 7) * 4;
            if (NCH % NW != 0 && wv + m * NW >= NCH) break;
            f4 kk, qq, bb, dd, up, on, all;
            make_item(x[m], kk, qq, bb, dd);
            // (a token alone: its query, undecayed, in the next one's row too, for q.k)
            const bool alone = L == 1 && t == 1;
            if (L < C)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    kk[e] = t < L ? kk[e] : 0.f;
                    qq[e] = t < L || alone ? qq[e] : 0.f;
                    bb[e] = t < L ? bb[e] : 0.f;
                    dd[e] = t < L ? dd[e] : 1.f;
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) bad += 0.f * (kk[e] + qq[e] + bb[e] + dd[e]);
            scan(dd, up, all, lane);
            f4 ki;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float r = __builtin_amdgcn_rcpf(up[e]);
                ki[e] = L > 1 ? kk[e] * r : kk[e];
                on[e] = L > 1 ? all[e] * r : 1.f;   // what decays behind the token
            }
            wide = wide || !(fminf(fminf(up[0], up[1]), fminf(up[2], up[3])) >= 0x1p-60f) ||
                   !(fabsf(ki[0]) + fabsf(ki[1]) + fabsf(ki[2]) + fabsf(ki[3]) < __builtin_inff());
            if (stay < L) {
                f4 part;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    kk[e] = t < stay ? kk[e] : 0.f;
                    dd[e] = t < stay ? dd[e] : 1.f;
                }
                scan(dd, part, all, lane);
#pragma unroll
                for (int e = 0; e < 4; ++e) on[e] = L > 1 ? all[e] * __builtin_amdgcn_rcpf(part[e]) : 1.f;
            }
            if (DK >= 32 || c < DK) {
                *reinterpret_cast<f4 *>(&sX[rec_row(t)][c]) = bb * up;
                *reinterpret_cast<f4 *>(&sX[rec_row(t) + 2][c]) = alone ? qq : qq * up;
                *reinterpret_cast<f4 *>(&sKi[t][c]) = ki;
                *reinterpret_cast<f4 *>(&sKh[par][t][c]) = kk * on;
                if (t == 0) *reinterpret_cast<f4 *>(&sG[par][c]) = all;
            }
        }
        // U = w*v of this lane's column, tokens g and g + 4
        float U[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            U[j] = g + 4 * j < L ? make_u(cu[j]) : 0.f;
            bad += 0.f * U[j];
        }
        if (bad != 0.f) sFlag[par].x = 1;   // (0 x: NaN unless x is finite)
        if (wide) sFlag[par].y = 1;
        __syncthreads();
        // ---- A and P: the decayed rows by the keys over their decays (their
        // fragments first: what follows takes as long as they do to arrive)
        constexpr int NT_AP = (NR + NAP - 1) / NAP;
        f4 fx[NT_AP], fk[NT_AP];
        if (NAP == NW || wv < NAP) {
#pragma unroll
            for (int m = 0; m < NT_AP; ++m) {
                const int at = 16 * (m * NAP + wv) + 4 * g;
                fx[m] = *reinterpret_cast<const f4 *>(&sX[n][at]);
                fk[m] = *reinterpret_cast<const f4 *>(&sKi[n & 7][at]);
            }
        }
        // (one value for all: the block's bounds stay in scalar registers)
        const int bads = __builtin_amdgcn_readfirstlane(sFlag[par].x), wides = __builtin_amdgcn_readfirstlane(sFlag[par].y);
        if (L > 1 && (bads | wides)) {
            if (!bads) {
                most = L / 2;
                L = length(done);
            } else if (done < commit && commit < done + L) {
                L = commit - done;
            } else {
                most = L = 1;
            }
            load_block(tb, L, lane);
            if (tid == 0) sFlag[par ^ 1] = make_int2(0, 0);
            __syncthreads();
            continue;
        }
        if (tid == 0) sFlag[par ^ 1] = make_int2(0, 0);
        // lane n (of 8) + 16 g has A and P of tokens g and g + 4 with token n
        f4 ap = f4zero();
        if (NAP == NW || wv < NAP) {
#pragma unroll
            for (int m = 0; m < NT_AP; ++m) ap = Mma<float>::mma(fx[m], fk[m], ap);
        }
        // the next block's loads, under way during this one's products
        const int next = done + L, Lb = L;
        if (next < len) {
            L = length(next);
            load_block(t0 + next, L, lane);
        }
        if ((NAP == NW || wv < NAP) && n < C) *reinterpret_cast<f4 *>(&sPart[wv][g][n][0]) = ap;
        __syncthreads();

        // ---- X and P by wave 0 (X a column a lane, the entries of A as
        // scalars), R = [b k D; q D] S0 by all
        if (wv == 0) {
            f4 ap = f4zero();
#pragma unroll
            for (int z = 0; z < NAP; ++z) ap += *reinterpret_cast<const f4 *>(&sPart[z][g][n & 7][0]);
            const int j = lane & 7;
            if (n < C) {
                sM[rec_row(g) + 2][j] = j <= g ? ap[2] : 0.f;
                sM[rec_row(g + 4) + 2][j] = j <= g + 4 ? ap[3] : 0.f;
            }
            auto entry = [&](int t, int s) {
                return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ap[t >> 2]), 16 * (t & 3) + s));
            };
            float y[C];
#pragma unroll
            for (int t = 0; t < C; ++t) {
                y[t] = t == j ? 1.f : 0.f;
#pragma unroll
                for (int s = 0; s < t; ++s) y[t] -= entry(t, s) * y[s];
                sM[rec_row(t)][j] = y[t];   // (eight lanes write the same)
            }
            if (Lb == 1) sM[rec_row(0) + 2][0] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ap[2]), 16));
        }
        f4 R = left_product(n);
        // the state's decay, while wave 0 works (by one where nothing stays)
#pragma unroll
        for (int r = 0; r < NR; ++r) S[r] *= *reinterpret_cast<const f4 *>(&sG[par][16 * r + 4 * g]);
        __syncthreads();

        // ---- Delta = X (U - R_E), O = R_Q + P Delta, then the state
        {
            const float m0 = sM[n][g], m1 = sM[n][g + 4];
            const bool query = n & 2;
            const float x0 = query ? 0.f : m0, x1 = query ? 0.f : m1, p0 = query ? m0 : 0.f, p1 = query ? m1 : 0.f;
            const float u0 = U[0] - R[0], u1 = U[1] - R[1];
            const f4 rq = {0.f, 0.f, R[2], R[3]};
            const f4 z = mfma4(x1, u1, mfma4(x0, u0, rq));
            R = mfma4(p1, z[1], mfma4(p0, z[0], z));
            if (__builtin_amdgcn_ballot_w64(!(fabsf(z[0]) + fabsf(z[1]) < __builtin_inff()))) {
                // Finite tokens whose product with the state, or whose X, is
                // not: the zeros above a triangle must not meet it. One token
                // after the other, from those up to it: as above, and by A
                // itself where X fails.
                float d0 = 0.f, d1 = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll 1
                for (int t = 0; t < C; ++t) {
                    float a0 = 0.f, a1 = 0.f;   // A of token t with tokens g and g + 4
#pragma unroll 1
                    for (int z = 0; z < NAP; ++z) {
                        a0 += sPart[z][t & 3][g][t >> 2];
                        a1 += sPart[z][t & 3][g + 4][t >> 2];
                    }
                    const float e = across((g < t ? a0 * d0 : 0.f) + (g + 4 < t ? a1 * d1 : 0.f));
                    const f4 y = mfma4(x1, g + 4 <= t ? u1 : 0.f, mfma4(x0, g <= t ? u0 : 0.f, rq));
                    d0 = g == t ? (fabsf(y[0]) < __builtin_inff() ? y[0] : u0 - e) : d0;
                    d1 = g + 4 == t ? (fabsf(y[1]) < __builtin_inff() ? y[1] : u1 - e) : d1;
                    const f4 o = mfma4(p1, g + 4 <= t ? d1 : 0.f, mfma4(p0, g <= t ? d0 : 0.f, rq));
                    o0 = g == t ? o[2] : o0;
                    o1 = g + 4 == t ? o[3] : o1;
                }
                R = (f4){g < stay ? d0 : 0.f, g + 4 < stay ? d1 : 0.f, o0, o1};
            }
        }
        if (stay > 0)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                S[r] = mfma4(sKh[par][g + 4][16 * r + n], R[1], mfma4(sKh[par][g][16 * r + n], R[0], S[r]));
            }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (g + 4 * j < Lb) put_o(tb, g + 4 * j, col, R[2 + j]);
        if (stay > 0 && done + stay == commit) keep();
        done = next;
        // No barrier: what the products here read (sKh, sG: one of two) is
        // written again two blocks on, the rest after this block's last barrier.
    }
}

template <typename In, int DK, int DV, int NW> static void rec_go(const RecurrentArgs &a, hipStream_t st)
{
    RecParams p = {a.q, a.k, a.v, a.b, a.w, a.log_alpha, a.state, a.slot_in, a.slot_out, a.commit, a.cu_seqlens, a.o,
                   a.T, a.H, a.HK, a.slots, a.gates, a.out_bf16};
    hipLaunchKernelGGL((recurrent_kernel<In, DK, DV, NW>), dim3(a.N * a.H * (DV / (16 * NW))), dim3(64 * NW), 0, st, p);
}

// A workgroup a chain, unless two workgroups a chain still leave every compute
// unit at most one: then a chain of eight waves is cut in two, so that each
// wave has a matrix core to itself (one chain, 64 tokens, 128 x 128: 34 -> 28
// us; 128 chains: 37 -> 33; 256 chains: 41 either way; 256 x 16 chains of one
// token: 111 us whole, 113 in two, 126 in four).
template <typename In, int DK, int DV> static void rec_split(const RecurrentArgs &a, hipStream_t st)
{
    constexpr int ALL = DV / 16, CUS = 256;
    if (ALL > 4 && (long long)a.N * a.H * 2 <= CUS) rec_go<In, DK, DV, (ALL < 4 ? ALL : 4)>(a, st);
    else rec_go<In, DK, DV, ALL>(a, st);
}

template <typename In, int DK> static hipError_t rec_dv(const RecurrentArgs &a, hipStream_t st)
{
    prof_before("gdn2_recurrent", st);
    switch (a.dv) {
    case 16: rec_split<In, DK, 16>(a, st); break;
    case 32: rec_split<In, DK, 32>(a, st); break;
    case 64: rec_split<In, DK, 64>(a, st); break;
    case 128: rec_split<In, DK, 128>(a, st); break;
    default: return hipErrorInvalidValue;
    }
    prof_after(st);
    return hipGetLastError();
}

template <typename In> static hipError_t rec_dk(const RecurrentArgs &a, hipStream_t st)
{
    switch (a.dk) {
    case 16: return rec_dv<In, 16>(a, st);
    case 32: return rec_dv<In, 32>(a, st);
    case 64: return rec_dv<In, 64>(a, st);
    case 128: return rec_dv<In, 128>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace gdn2
