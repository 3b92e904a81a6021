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
    int T, N, H, HK, slots, dv, gates, out_bf16;
};

template <int NC> struct ColVec;
template <> struct ColVec<1> {
    typedef float t;
};
template <> struct ColVec<2> {
    typedef f2 t;
};
template <int NC> __device__ __forceinline__ float col_get(const typename ColVec<NC>::t &x, int c)
{
    if constexpr (NC == 1) return x;
    else return x[c];
}
template <int NC> __device__ __forceinline__ void col_set(typename ColVec<NC>::t &x, int c, float f)
{
    if constexpr (NC == 1) x = f;
    else x[c] = f;
}

template <typename In, int DK, int NC, int NW>
__global__ __launch_bounds__(64 * NW) void recurrent_kernel(RecParams a)
{
    typedef typename ColVec<NC>::t cols_t;
    constexpr int C = kRecTokens, NT = 64 * NW, NR = DK / 16;
    constexpr int XS = DK + 4;    // row stride of the fragment tiles (16-byte rows)
    constexpr int RS = DK + 16;   // row stride of the raw rows: four of them apart in the banks
    constexpr int CPT = (DK + NT - 1) / NT;
    __shared__ __align__(16) float sX[16][XS], sKh[C][XS], sG[DK];
    __shared__ float sK[C][RS], sB[C][RS], sQ[C][RS], sD[C][RS];
    __shared__ float sPart[NW][4][9][2], sA[C][C], sP[C][C], sM[16][C + 1];
    __shared__ int sBad;   // a value of the block's tokens is not finite

    const int wgc = a.dv / (16 * NC * NW);   // workgroups of a chain
    const int chain = blockIdx.x / wgc;
    const int i = chain / a.H, h = chain % a.H;
    const int hk = h / (a.H / a.HK);
    const int tid = threadIdx.x, lane = tid & 63, wv = wave_id();
    const int n = lane & 15, g = lane >> 4;
    const int col = (blockIdx.x % wgc * NW + wv) * 16 * NC + NC * n;

    int t0, t1;
    if (a.cu) {
        t0 = min(max(a.cu[i], 0), a.T);
        t1 = min(max(a.cu[i + 1], t0), a.T);
    } else {
        t0 = i * a.T;
        t1 = t0 + a.T;
    }
    const int len = t1 - t0;
    const int commit = a.commit ? min(max(a.commit[i], 0), len) : len;
    const int sin = a.slot_in ? a.slot_in[i] : i;
    const int sout = a.slot_out ? a.slot_out[i] : sin;
    const bool has_in = (unsigned)sin < (unsigned)a.slots, has_out = (unsigned)sout < (unsigned)a.slots;
    // nothing to say and nothing to move
    if (len == 0 && (!has_out || sin == sout)) return;

    const size_t own = (size_t)h * DK * a.dv + col, slot_sz = (size_t)a.H * DK * a.dv;
    f4 S[NR][NC];
    if (has_in) {
        const float *sp = a.state + sin * slot_sz + own;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const cols_t x = *reinterpret_cast<const cols_t *>(sp + (size_t)(16 * r + 4 * g + j) * a.dv);
#pragma unroll
                for (int c = 0; c < NC; ++c) S[r][c][j] = col_get<NC>(x, c);
            }
    } else {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) S[r][c] = f4zero();
    }
    auto keep = [&]() {
        if (!has_out) return;
        float *sp = a.state + sout * slot_sz + own;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cols_t x;
#pragma unroll
                for (int c = 0; c < NC; ++c) col_set<NC>(x, c, S[r][c][j]);
                *reinterpret_cast<cols_t *>(sp + (size_t)(16 * r + 4 * g + j) * a.dv) = x;
            }
    };
    if (commit == 0 && sin != sout) keep();

    const In *q = (const In *)a.q, *k = (const In *)a.k, *v = (const In *)a.v, *b = (const In *)a.b,
             *w = (const In *)a.w;
    const bool asc = a.gates & kGateAlpha, bsc = a.gates & kGateB, wsc = a.gates & kGateW;
    // Tokens of a block. The products multiply what comes after a token by
    // zeros, which hides any number but a NaN or an infinity: a block that
    // holds one is done again, and what follows it, one token at a time.
    int most = C, L = 0;
    if (tid == 0) sBad = 0;
    __syncthreads();
    for (int done = 0; done < len; done += L) {
        // a block ends at the committed prefix, whose state is kept
        L = min(most, (done < commit ? commit : len) - done);
        const int tb = t0 + done;
        float bad = 0.f;

        // ---- the block's rows: one thread a channel
#pragma unroll
        for (int x = 0; x < CPT; ++x) {
            const int c = tid + x * NT;
            if (DK % NT == 0 || c < DK) {
                float kk[C], qq[C], bb[C], dd[C];
#pragma unroll
                for (int t = 0; t < C; ++t) {
                    const size_t tok = tb + min(t, L - 1);
                    const size_t ik = (tok * a.HK + hk) * DK + c, ih = tok * a.H + h, ic = ih * DK + c;
                    kk[t] = Ld<In>::one(k + ik);
                    qq[t] = Ld<In>::one(q + ik);
                    bb[t] = Ld<In>::one(b + (bsc ? ih : ic));
                    dd[t] = a.la[asc ? ih : ic];
                }
                float D = 1.f;
#pragma unroll
                for (int t = 0; t < C; ++t) {
                    const bool on = t < L;
                    kk[t] = on ? kk[t] : 0.f;
                    qq[t] = on ? qq[t] : 0.f;
                    bb[t] = on ? bb[t] * kk[t] : 0.f;
                    dd[t] = on ? __expf(dd[t]) : 1.f;
                    D *= dd[t];
                    bad += 0.f * (kk[t] + qq[t] + bb[t] + dd[t]);
                    sK[t][c] = kk[t];
                    sQ[t][c] = qq[t];
                    sB[t][c] = bb[t];
                    sD[t][c] = dd[t];
                    sX[rec_row(t)][c] = bb[t] * D;
                    sX[rec_row(t) + 2][c] = qq[t] * D;
                }
                sG[c] = D;
                float R = 1.f;
#pragma unroll
                for (int t = C - 1; t >= 0; --t) {
                    sKh[t][c] = kk[t] * R;
                    R *= dd[t];
                }
            }
        }
        // U = w*v of this lane's columns, tokens g and g + 4
        float U[2][NC];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = g + 4 * j;
            const size_t ih = (size_t)(tb + min(t, L - 1)) * a.H + h, iv = ih * a.dv + col;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float u = Ld<In>::one(w + (wsc ? ih : iv + c)) * Ld<In>::one(v + iv + c);
                U[j][c] = t < L ? u : 0.f;
                bad += 0.f * U[j][c];
            }
        }
        if (L > 1 && bad != 0.f) sBad = 1;   // (0 x: NaN unless x is finite)
        __syncthreads();
        if (L > 1 && sBad) {
            most = 1;
            L = 0;
            __syncthreads();
            if (tid == 0) sBad = 0;
            continue;
        }

        // ---- A and P: lane group p of 16 takes columns s = p and 7 - p of
        // the triangle (9 entries), its lanes and the waves share the channels
        {
            const int p = lane >> 4;
            float ea[9], ep[9];
#pragma unroll
            for (int e = 0; e < 9; ++e) ea[e] = ep[e] = 0.f;
            for (int c = wv * 16 + n; c < DK; c += 16 * NW) {
                float kf = 0.f;
#pragma unroll
                for (int e = 0; e < 9; ++e) {
                    const bool fst = e < 8 - p;
                    const int t = fst ? p + e : e - 1;
                    // the pair's first entry is (s, s); the factor then runs on
                    if (e == 0 || e == 8 - p) kf = sK[t][c];
                    else kf *= sD[t][c];
                    ea[e] += sB[t][c] * kf;
                    ep[e] += sQ[t][c] * kf;
                }
            }
#pragma unroll
            for (int e = 0; e < 9; ++e) {
                ea[e] = lane_group_sum<16>(ea[e]);
                ep[e] = lane_group_sum<16>(ep[e]);
                if (n == 0) {
                    sPart[wv][p][e][0] = ea[e];
                    sPart[wv][p][e][1] = ep[e];
                }
            }
        }
        __syncthreads();

        // ---- [X; P X] by wave 0, a column a lane
        if (wv == 0) {
            if (lane < 36) {
                const int p = lane / 9, e = lane % 9;
                const bool fst = e < 8 - p;
                const int t = fst ? p + e : e - 1, s = fst ? p : 7 - p;
                float xa = 0.f, xp = 0.f;
#pragma unroll
                for (int x = 0; x < NW; ++x) {
                    xa += sPart[x][p][e][0];
                    xp += sPart[x][p][e][1];
                }
                sA[t][s] = xa;
                sP[t][s] = xp;
            }
            __builtin_amdgcn_wave_barrier();
            const int j = lane & 7;
            float x[C];
#pragma unroll
            for (int t = 0; t < C; ++t) {
                float y = t == j ? 1.f : 0.f, z = 0.f;
#pragma unroll
                for (int s = 0; s < t; ++s) y -= sA[t][s] * x[s];
                x[t] = y;
#pragma unroll
                for (int s = 0; s <= t; ++s) z += sP[t][s] * x[s];
                if (lane < C) {
                    sM[rec_row(t)][j] = y;
                    sM[rec_row(t) + 2][j] = z;
                }
            }
        }
        // ---- R = [b k D; q D] S0 (all waves, no wait for the above)
        f4 R[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) R[c] = f4zero();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const f4 x = *reinterpret_cast<const f4 *>(&sX[n][16 * r + 4 * g]);
#pragma unroll
            for (int c = 0; c < NC; ++c) R[c] = Mma<float>::mma(x, S[r][c], R[c]);
        }
        __syncthreads();

        // ---- Delta and O, then the state
        const float m0 = sM[n][g], m1 = sM[n][g + 4];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            f4 x = {0.f, 0.f, R[c][2], R[c][3]};
            x = mfma4(m0, U[0][c] - R[c][0], x);
            R[c] = mfma4(m1, U[1][c] - R[c][1], x);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const f4 gm = *reinterpret_cast<const f4 *>(&sG[16 * r + 4 * g]);
            const float k0 = sKh[g][16 * r + n], k1 = sKh[g + 4][16 * r + n];
#pragma unroll
            for (int c = 0; c < NC; ++c) S[r][c] = mfma4(k1, R[c][1], mfma4(k0, R[c][0], S[r][c] * gm));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = g + 4 * j;
            if (t < L) {
                const size_t io = ((size_t)(tb + t) * a.H + h) * a.dv + col;
                if (a.out_bf16) {
                    uint16_t *o = (uint16_t *)a.o + io;
                    if constexpr (NC == 2) *reinterpret_cast<uint32_t *>(o) = bf16x2(R[0][2 + j], R[1][2 + j]);
                    else *o = (uint16_t)bf16x2(R[0][2 + j], 0.f);
                } else {
                    cols_t x;
#pragma unroll
                    for (int c = 0; c < NC; ++c) col_set<NC>(x, c, R[c][2 + j]);
                    *reinterpret_cast<cols_t *>((float *)a.o + io) = x;
                }
            }
        }
        if (done + L == commit) keep();
        __syncthreads();
    }
}

template <typename In, int DK, int NC, int NW> static void rec_go(const RecurrentArgs &a, hipStream_t st)
{
    RecParams p = {a.q, a.k, a.v, a.b, a.w, a.log_alpha, a.state, a.slot_in, a.slot_out, a.commit, a.cu_seqlens, a.o,
                   a.T, a.N, a.H, a.HK, a.slots, a.dv, a.gates, a.out_bf16};
    hipLaunchKernelGGL((recurrent_kernel<In, DK, NC, NW>), dim3(a.N * a.H * (a.dv / (16 * NC * NW))), dim3(64 * NW), 0,
                       st, p);
}

template <typename In, int DK> static hipError_t rec_dv(const RecurrentArgs &a, hipStream_t st)
{
    prof_before("gdn2_recurrent", st);
    switch (a.dv) {
    case 16: rec_go<In, DK, 1, 1>(a, st); break;
    case 32: rec_go<In, DK, 1, 2>(a, st); break;
    case 64: rec_go<In, DK, 2, 2>(a, st); break;
    case 128: rec_go<In, DK, 2, 4>(a, st); break;
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
