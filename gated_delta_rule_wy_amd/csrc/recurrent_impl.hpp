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
//   A_ts = sum_c (b_t k_t)_c (alpha_{s+1} .. alpha_t)_c (k_s)_c      (t > s)
//   P_ts = sum_c (q_t)_c (alpha_{s+1} .. alpha_t)_c (k_s)_c          (t >= s)
//   R_E = (b k D) S0,  R_Q = (q D) S0,  X = (I + A)^-1
//   Delta = X (U - R_E),  O = R_Q + P X (U - R_E)
//   S = D_8 S0 + (k alpha_{t+1} .. alpha_8)^T Delta
// Every decay is a running product of alphas (never a quotient or a
// difference of logarithms), so any log alpha <= 0 is exact to a few units of
// the last place, log alpha = -inf (a full forget) among them. All of it is
// fp32, on the fp32 matrix instruction.
//
// A workgroup owns 16*NC*NW columns of one (sequence, head) state, a wave
// 16*NC of them in registers: tile r, lane n + 16g holds rows 16r + 4g + j of
// columns NC*n .. NC*n + NC - 1, which is the accumulator layout, and with
// element j of a 16-deep fragment on row 4g + j also the right operand's. The
// block's 16 left rows are ordered so that rows 4g .. 4g+3 are the erase rows
// of tokens g and g+4 and their query rows: the first product leaves in each
// lane just what the second one (by [X; P X]) takes as its right operand,
// which leaves Delta where the third one (by the decayed keys) takes it. The
// state thus never moves between lanes and is read and written once however
// many tokens follow, which is what the operator is bound by: 8 bytes a state
// element.
#pragma once

#include "gdn2_launch.hpp"
#include "rows.hpp"

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

// Four elements as they lie in memory (or the first of them alone).
template <typename In> struct Raw4;
template <> struct Raw4<uint16_t> {
    uint2 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void load1(const uint16_t *p) { r.x = *p; }
    __device__ __forceinline__ f4 get() const
    {
        f4 x = {__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                __uint_as_float(r.y & 0xFFFF0000u)};
        return x;
    }
    __device__ __forceinline__ float get1() const { return __uint_as_float(r.x << 16); }
};
template <> struct Raw4<float> {
    f4 r;
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const f4 *>(p); }
    __device__ __forceinline__ void load1(const float *p) { r[0] = *p; }
    __device__ __forceinline__ f4 get() const { return r; }
    __device__ __forceinline__ float get1() const { return r[0]; }
};
// Keeps the LDS reads behind it from being issued before it, where that would
// take more registers than there are.
__device__ __forceinline__ void hold_reads() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ f4 splat4(float x) { f4 r = {x, x, x, x}; return r; }

template <typename In, int DK, int NW>
__global__ __launch_bounds__(64 * NW, 4) void recurrent_kernel(RecParams a)
{
    constexpr int C = kRecTokens, NT = 64 * NW, NR = DK / 16, DV = 16 * NW;
    constexpr int XS = DK + 4;    // row stride of the fragment tiles (16-byte rows)
    constexpr int RS = DK + 16;   // row stride of the raw rows: four of them apart in the banks
    // one thread takes four channels of a token
    constexpr int C4 = DK / 4, ITEMS = C * C4, IPT = (ITEMS + NT - 1) / NT;
    __shared__ __align__(16) float sX[16][XS], sKh[C][XS], sG[DK];
    __shared__ __align__(16) float sK[C][RS], sB[C][RS], sQ[C][RS], sD[C][RS];
    __shared__ float sPart[NW][4][9][2], sM[16][C + 1];
    __shared__ int sBad;   // a value of the block's tokens is not finite

    const int i = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int hk = h / (a.H / a.HK);
    const int tid = threadIdx.x, lane = tid & 63, wv = wave_id();
    const int n = lane & 15, g = lane >> 4;
    const int col = 16 * wv + n;

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
    };
    // the four channels at c of token tok
    auto load_item = [&](int tok, int c, Item &x) {
        const size_t ih = (size_t)tok * a.H + h, ik = ((size_t)tok * a.HK + hk) * DK + c, ic = ih * DK + c;
        x.k.load(k + ik);
        x.q.load(q + ik);
        if (bsc) x.b.load1(b + ih);
        else x.b.load(b + ic);
        if (asc) x.la[0] = a.la[ih];
        else x.la = *reinterpret_cast<const f4 *>(a.la + ic);
    };
    // k, q, b*k and alpha
    auto make_item = [&](const Item &x, f4 &kk, f4 &qq, f4 &bb, f4 &dd) {
        kk = x.k.get();
        qq = x.q.get();
        bb = (bsc ? splat4(x.b.get1()) : x.b.get()) * kk;
        const f4 la = asc ? splat4(x.la[0]) : x.la;
#pragma unroll
        for (int e = 0; e < 4; ++e) dd[e] = __expf(la[e]);
    };
    // v and w of this lane's column
    struct Col {
        In v, w;
    };
    auto load_u = [&](int tok, int col, Col &x) {
        const size_t ih = (size_t)tok * a.H + h;
        x.v = v[ih * DV + col];
        x.w = w[wsc ? ih : ih * DV + col];
    };
    auto make_u = [&](const Col &x) { return in2f<In>(x.v) * in2f<In>(x.w); };
    auto put_o = [&](int tok, int col, float x) {
        const size_t io = ((size_t)tok * a.H + h) * DV + col;
        if (a.out_bf16) ((uint16_t *)a.o)[io] = (uint16_t)bf16x2(x, 0.f);
        else ((float *)a.o)[io] = x;
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
            for (int j = 0; j < 4; ++j) __builtin_nontemporal_store(S[r][j], sp + (16 * r + j) * DV);
    };
    if (commit == 0 && sin != sout) keep();
    if (len == 0) return;   // (no token to load)

    if (len == 1) {
        // ---- a single token: Delta = U - R_E, O = R_Q + (q.k) Delta
        Col cu;
        load_u(t0, col, cu);
        if (tid < C4) {
            Item x;
            f4 kk, qq, bb, dd;
            load_item(t0, 4 * tid, x);
            make_item(x, kk, qq, bb, dd);
            *reinterpret_cast<f4 *>(&sX[0][4 * tid]) = bb * dd;
            *reinterpret_cast<f4 *>(&sX[2][4 * tid]) = qq * dd;
            *reinterpret_cast<f4 *>(&sKh[0][4 * tid]) = kk;
            *reinterpret_cast<f4 *>(&sQ[0][4 * tid]) = qq;
            *reinterpret_cast<f4 *>(&sG[4 * tid]) = dd;
        }
        __syncthreads();
        float kq = 0.f;
#pragma unroll
        for (int c = 0; c < DK; c += 64)
            if (DK >= 64 || lane < DK) kq += sKh[0][c + lane] * sQ[0][c + lane];
        kq = lane_group_sum<64>(kq);
        // rows 0 and 2 are the token's; all others repeat one of them
        f4 R = f4zero();
#pragma unroll
        for (int r = 0; r < NR; ++r) R = Mma<float>::mma(*reinterpret_cast<const f4 *>(&sX[n & 2][16 * r + 4 * g]), S[r], R);
        const float d = make_u(cu) - R[0];
        if (commit == 1 && has_out) {
            const float dg = g == 0 ? d : 0.f;
#pragma unroll
            for (int r = 0; r < NR; ++r)
                S[r] = mfma4(sKh[0][16 * r + n], dg, S[r] * *reinterpret_cast<const f4 *>(&sG[16 * r + 4 * g]));
            keep();
        }
        if (g == 0) put_o(t0, col, R[2] + kq * d);
        return;
    }

    // Tokens of a block. The products multiply what comes after a token by
    // zeros, which hides any number but a NaN or an infinity: a block that
    // holds one is done again without the tokens that are not committed, or,
    // where that is not it, one token at a time, with all that follow it.
    int most = C, L = 0;
    // A block ends at the committed prefix, whose state is kept, but for the
    // last one, whose later tokens then leave the state alone.
    auto length = [&](int done) {
        const int rem = len - done;
        return rem <= most ? rem : min(most, done < commit ? commit - done : rem);
    };
    if (tid == 0) sBad = 0;
    Item x[IPT];
    Col cu[2];
    auto load_block = [&](int tb, int L, int tid) {
        const int g = tid >> 4 & 3, col = 16 * wv + (tid & 15);
#pragma unroll
        for (int m = 0; m < IPT; ++m) {
            const int it = min(tid + m * NT, ITEMS - 1);
            load_item(tb + min(it / C4, L - 1), it % C4 * 4, x[m]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) load_u(tb + min(g + 4 * j, L - 1), col, cu[j]);
    };
    L = length(0);
    load_block(t0, L, tid);
    __syncthreads();
    for (int done = 0; done < len;) {
        int lane = tid & 63;
        // (the lane's addresses are formed anew in each block: kept over the
        // loop they would take a third of the registers)
        asm volatile("" : "+v"(lane));
        const int tid = wv * 64 + lane, n = lane & 15, g = lane >> 4, col = 16 * wv + n;
        const int tb = t0 + done;
        f4 kk[IPT], qq[IPT], bb[IPT];
        float U[2];
        for (;;) {
            // ---- raw rows; those past the block are zeros that decay nothing
            float bad = 0.f;
#pragma unroll
            for (int m = 0; m < IPT; ++m) {
                const int it = tid + m * NT, t = it / C4, c = it % C4 * 4;
                f4 dd;
                make_item(x[m], kk[m], qq[m], bb[m], dd);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    kk[m][e] = t < L ? kk[m][e] : 0.f;
                    qq[m][e] = t < L ? qq[m][e] : 0.f;
                    bb[m][e] = t < L ? bb[m][e] : 0.f;
                    dd[e] = t < L ? dd[e] : 1.f;
                    bad += 0.f * (kk[m][e] + qq[m][e] + bb[m][e] + dd[e]);
                }
                if (ITEMS % NT == 0 || it < ITEMS) {
                    *reinterpret_cast<f4 *>(&sK[t][c]) = kk[m];
                    *reinterpret_cast<f4 *>(&sQ[t][c]) = qq[m];
                    *reinterpret_cast<f4 *>(&sB[t][c]) = bb[m];
                    *reinterpret_cast<f4 *>(&sD[t][c]) = dd;
                }
            }
            // U = w*v of this lane's column, tokens g and g + 4
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                U[j] = g + 4 * j < L ? make_u(cu[j]) : 0.f;
                bad += 0.f * U[j];
            }
            if (L > 1 && bad != 0.f) sBad = 1;   // (0 x: NaN unless x is finite)
            __syncthreads();
            if (L == 1 || !sBad) break;
            // (first without a draft's end: its committed part stays one block)
            if (done < commit && commit < done + L) L = commit - done;
            else most = L = 1;
            load_block(tb, L, tid);
            __syncthreads();
            if (tid == 0) sBad = 0;
        }
        // the block's tokens whose effect stays: all but those of a draft's end
        const int stay = done + L < len ? L : min(max(commit - done, 0), L);
        // the next block's loads, under way during this one's products
        const int next = done + L;
        const int Lb = L;
        if (next < len) {
            L = length(next);
            load_block(t0 + next, L, tid);
        }

        // ---- the decayed rows: products of alphas up to a token and behind it
#pragma unroll
        for (int m = 0; m < IPT; ++m) {
            const int it = tid + m * NT, t = it / C4, c = it % C4 * 4;
            if (ITEMS % NT != 0 && it >= ITEMS) break;
            f4 up = splat4(1.f), on = splat4(1.f), all = splat4(1.f);
#pragma unroll
            for (int s = 0; s < C; ++s) {
                const f4 d = *reinterpret_cast<const f4 *>(&sD[s][c]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    up[e] *= s <= t ? d[e] : 1.f;
                    on[e] *= s > t && s < stay ? d[e] : 1.f;
                    all[e] *= s < stay ? d[e] : 1.f;
                }
                if (s == 3) hold_reads();
            }
            *reinterpret_cast<f4 *>(&sX[rec_row(t)][c]) = bb[m] * up;
            *reinterpret_cast<f4 *>(&sX[rec_row(t) + 2][c]) = qq[m] * up;
            *reinterpret_cast<f4 *>(&sKh[t][c]) = t < stay ? kk[m] * on : f4zero();
            if (t == C - 1) *reinterpret_cast<f4 *>(&sG[c]) = all;
        }

        // ---- A and P: lane group p of 16 takes columns s = p and 7 - p of
        // the triangle (9 entries), its lanes and the waves share the channels
        {
            const int p = g;
            float ea[9], ep[9];
#pragma unroll
            for (int e = 0; e < 9; ++e) ea[e] = ep[e] = 0.f;
#pragma unroll
            for (int c0 = 0; c0 < DK; c0 += 16 * NW) {
                const int c = c0 + wv * 16 + n;
                if (DK % (16 * NW) != 0 && c >= DK) break;
                float kf = 0.f;
#pragma unroll
                for (int e = 0; e < 9; ++e) {
                    const int t = e < 8 - p ? p + e : e - 1;
                    // the pair's first entry is (s, s); the factor then runs on
                    const float kx = sK[t][c], dx = sD[t][c];
                    kf = e == 0 || e == 8 - p ? kx : kf * dx;
                    ea[e] += sB[t][c] * kf;
                    ep[e] += sQ[t][c] * kf;
                    if (e == 4) hold_reads();
                }
                hold_reads();
            }
#pragma unroll
            for (int e = 0; e < 9; ++e) {
                ea[e] = lane_group_sum<16>(ea[e]);
                ep[e] = lane_group_sum<16>(ep[e]);
            }
            if (n == 0)
#pragma unroll
                for (int e = 0; e < 9; ++e) {
                    sPart[wv][p][e][0] = ea[e];
                    sPart[wv][p][e][1] = ep[e];
                }
        }
        __syncthreads();

        // ---- [X; P X] by wave 0, a column a lane: lane 9 p + e has an entry
        // of A and one of P, which go to all lanes as scalars
        if (wv == 0) {
            float xa = 0.f, xp = 0.f;
            if (lane < 36) {
                const int p = lane / 9, e = lane % 9;
#pragma unroll
                for (int z = 0; z < NW; ++z) {
                    xa += sPart[z][p][e][0];
                    xp += sPart[z][p][e][1];
                }
            }
            auto entry = [](float f, int t, int s) {
                const int at = s < 4 ? 9 * s + t - s : 9 * (7 - s) + t + 1;
                return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), at));
            };
            const int j = lane & 7;
            float y[C];
#pragma unroll
            for (int t = 0; t < C; ++t) {
                float z = 0.f;
                y[t] = t == j ? 1.f : 0.f;
#pragma unroll
                for (int s = 0; s < t; ++s) y[t] -= entry(xa, t, s) * y[s];
#pragma unroll
                for (int s = 0; s <= t; ++s) z += entry(xp, t, s) * y[s];
                if (lane < C) {
                    sM[rec_row(t)][j] = y[t];
                    sM[rec_row(t) + 2][j] = z;
                }
            }
        }
        // ---- R = [b k D; q D] S0 (all waves, no wait for the above), in two
        // chains of products
        f4 R = f4zero(), R2 = f4zero();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const f4 z = *reinterpret_cast<const f4 *>(&sX[n][16 * r + 4 * g]);
            if (r % 2 == 0) R = Mma<float>::mma(z, S[r], R);
            else R2 = Mma<float>::mma(z, S[r], R2);
            if (r % 4 == 3) hold_reads();
        }
        R += R2;
        __syncthreads();

        // ---- Delta and O, then the state
        {
            f4 z = {0.f, 0.f, R[2], R[3]};
            z = mfma4(sM[n][g], U[0] - R[0], z);
            R = mfma4(sM[n][g + 4], U[1] - R[1], z);
        }
        if (stay > 0)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                S[r] = mfma4(sKh[g + 4][16 * r + n], R[1],
                             mfma4(sKh[g][16 * r + n], R[0], S[r] * *reinterpret_cast<const f4 *>(&sG[16 * r + 4 * g])));
                if (r % 4 == 3) hold_reads();
            }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (g + 4 * j < Lb) put_o(tb + g + 4 * j, col, R[2 + j]);
        if (stay > 0 && done + stay == commit) keep();
        done = next;
        // No barrier: the next block's raw rows are read last before the second
        // barrier above, and what the products here read is written after its first.
    }
}

template <typename In, int DK, int NW> static void rec_go(const RecurrentArgs &a, hipStream_t st)
{
    RecParams p = {a.q, a.k, a.v, a.b, a.w, a.log_alpha, a.state, a.slot_in, a.slot_out, a.commit, a.cu_seqlens, a.o,
                   a.T, a.H, a.HK, a.slots, a.gates, a.out_bf16};
    hipLaunchKernelGGL((recurrent_kernel<In, DK, NW>), dim3(a.N * a.H), dim3(64 * NW), 0, st, p);
}

template <typename In, int DK> static hipError_t rec_dv(const RecurrentArgs &a, hipStream_t st)
{
    prof_before("gdn2_recurrent", st);
    switch (a.dv) {
    case 16: rec_go<In, DK, 1>(a, st); break;
    case 32: rec_go<In, DK, 2>(a, st); break;
    case 64: rec_go<In, DK, 4>(a, st); break;
    case 128: rec_go<In, DK, 8>(a, st); break;
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
