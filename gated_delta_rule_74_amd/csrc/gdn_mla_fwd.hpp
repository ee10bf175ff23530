// Causal attention of expanded latent-attention heads, forward.
//
//   z_ij = scale (q_i[:dn] . k_j + q_i[dn:] . kr_j),  o_i = sum_j softmax(z_i)_j v_j,
//   lse_i = log sum_j exp z_ij   over the keys j <= i + Tk - Tq, j < len_b
//
// in one pass over the keys with the running maximum and sum of the softmax.
// A workgroup takes NW * QT * 16 queries of one head and walks the keys in
// tiles of 64 that all its waves share in LDS; a wave holds its QT * 16
// queries in registers for the whole walk. The products are formed
// transposed, S^T = K Q^T and O^T = V^T P^T: then a lane owns one query
// (column), the maximum and the rescaling are per-lane scalars, and the
// probabilities leave the first product in exactly the lanes and K order that
// the second one wants its operand in, so they never pass through LDS; V is
// read from its row-major tile by transposing LDS reads.
// The running maximum is only moved when a score exceeds it by more than
// RAISE (in powers of two): until then the probabilities are merely up to
// 2^RAISE too large, in P, in the sum and in O alike, which fp32 holds without
// loss; this keeps the cross-lane maximum and the rescaling of O out of almost
// every tile.
#pragma once

#include "gdn_mla.hpp"

namespace gdn {

constexpr int MLA_KT = 64;      // keys per tile
constexpr float MLA_RAISE = 8.f; // see above

template <bool BF, int DP, int DVP, int NW, int QT> struct MlaFwdShape {
    using S = typename Op<BF>::S;
    static constexpr int LDK = DP + Op<BF>::PAD, LDV = DVP + Op<BF>::PAD, QB = NW * QT * 16;
    // two tiles where a second workgroup still fits the CU's 160 KB beside them
    static constexpr int NB = 2 * MLA_KT * (LDK + LDV) * (int)sizeof(S) <= 80 * 1024 ? 2 : 1;
};

// Block qb of the queries of head bh.
template <bool BF, int DP, int DVP, int NW, int QT, class S>
__device__ __forceinline__ void mla_fwd_block(const MlaFwdArgs a, int bh, int qb, S *Kst, S *Vst) {
    using H = MlaFwdShape<BF, DP, DVP, NW, QT>;
    constexpr int LDK = H::LDK, LDV = H::LDV, NB = H::NB, NT = NW * 64, KS = DP / 32, MV = DVP / 16;
    const MlaArgs s = a.s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    constexpr int QB = H::QB;
    const int b = bh / s.H, h = bh % s.H, hk = h / (s.H / s.Hk);
    const int hr = s.Hr > 0 ? h / (s.H / s.Hr) : 0;
    const int D = s.dn + s.dr, off = s.Tk - s.Tq;
    const int n = s.lens ? min(max(s.lens[b], 0), s.Tk) : s.Tk;
    const int q0 = qb * QB + wave * QT * 16; // first query of this wave
    const size_t rq = (size_t)s.H * D, rk = (size_t)s.Hk * s.dn, rr = (size_t)s.Hr * s.dr, rv = (size_t)s.Hk * s.dv;
    const S *kp = (const S *)s.k + (size_t)b * s.Tk * rk + (size_t)hk * s.dn;
    const S *krp = s.dr > 0 ? (const S *)s.kr + (size_t)b * s.Tk * rr + (size_t)hr * s.dr : kp;
    const S *vp = (const S *)s.v + (size_t)b * s.Tk * rv + (size_t)hk * s.dv;

    // keys the workgroup has to see: those of its last query that is not padding
    const int last = min(min(qb * QB + QB, s.Tq) - 1 + off, n - 1);
    const int first = qb * QB + off; // position of its first query
    const int nt = first < n ? last / MLA_KT + 1 : 0;

    RowTile<BF, DP, MLA_KT, NT> kt;
    RowTile<BF, DVP, MLA_KT, NT> vt;
    kt.init(kp, rk, s.dn, krp, rr, s.dr, tid);
    vt.init(vp, rv, s.dv, vp, 0, 0, tid);
    if (nt > 0) {
        kt.fetch(0, n);
        vt.fetch(0, n);
    }
    // queries as operand columns; rows past the sequence read as zero
    Frag<BF> Q[QT][KS];
    const S *qp = (const S *)s.q + (size_t)b * s.Tq * rq + (size_t)h * D;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = q0 + 16 * t + r;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int c = 32 * k + 8 * g;
            Q[t][k] = (i < s.Tq && c < D) ? row8(qp + (size_t)i * rq + c) : zero8<BF>();
        }
    }
    f32x4 O[QT][MV];
    float m[QT], l[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.f;
#pragma unroll
        for (int v = 0; v < MV; ++v) O[t][v] = zero4();
    }
    const float c2 = s.scale * (float)LOG2E;
    if (nt > 0) {
        kt.stash(Kst, LDK, 0, n);
        vt.stash(Vst, LDV, 0, n);
        lds_barrier();
    }
    wait_vmem(); // (Q is there: else its first use in the loop waits for the tile in flight)
    const int wlast = min(q0 + QT * 16 - 1 + off, n - 1), wfirst = q0 + off;
    for (int kb = 0; kb < nt; ++kb) {
        const int key0 = kb * MLA_KT;
        if (kb + 1 < nt) {
            kt.fetch(key0 + MLA_KT, n);
            vt.fetch(key0 + MLA_KT, n);
        }
        if (key0 <= wlast && wfirst < n) {
            const S *K = Kst + kb % NB * (MLA_KT * LDK), *V = Vst + kb % NB * (MLA_KT * LDV);
            const bool mask = key0 + MLA_KT - 1 > wfirst || key0 + MLA_KT > n;
#pragma unroll 1
            for (int u = 0; u < MLA_KT / 32; ++u) {
                f32x4 P[QT][2];
#pragma unroll
                for (int t = 0; t < QT; ++t) P[t][0] = P[t][1] = zero4();
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const Frag<BF> kf = row8(K + (32 * u + 16 * j + r) * LDK + 32 * k + 8 * g);
#pragma unroll
                        for (int t = 0; t < QT; ++t) P[t][j] = mma8(kf, Q[t][k], P[t][j]);
                    }
                // the mask, where this tile reaches past a query or the sequence
                if (mask) {
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        const int lim = min(q0 + 16 * t + r + off, n - 1) - key0 - 32 * u - 4 * g; // last key seen
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) P[t][j][e] = 16 * j + e <= lim ? P[t][j][e] : -INFINITY;
                    }
                }
                float mx[QT];
                bool raise = false;
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    float x = P[t][0][0];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x = fmaxf(x, P[t][j][e]);
                    mx[t] = x * c2;
                    raise |= mx[t] > m[t] + MLA_RAISE;
                }
                if (__any(raise)) {
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        const float mn = fmaxf(m[t], max4g(mx[t]));
                        const float f = mn == -INFINITY ? 1.f : exp2_fast(m[t] - mn);
                        m[t] = mn;
                        l[t] *= f;
#pragma unroll
                        for (int v = 0; v < MV; ++v) O[t][v] *= f;
                    }
                }
                Frag<BF> pf[QT];
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const float mt = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) P[t][j][e] = exp2_fast(fmaf(P[t][j][e], c2, -mt));
                    const f32x4 sum = P[t][0] + P[t][1];
                    l[t] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    pf[t] = acc8<BF>(P[t][0], P[t][1]);
                }
#pragma unroll
                for (int v = 0; v < MV; ++v) {
                    const Frag<BF> vf = col8(V, LDV, 32 * u, 16 * v, lane);
#pragma unroll
                    for (int t = 0; t < QT; ++t) O[t][v] = mma8(vf, pf[t], O[t][v]);
                }
            }
        }
        if (kb + 1 < nt) {
            // with two buffers the other one's last readers passed the previous barrier
            if (NB == 1) lds_barrier();
            kt.stash(Kst + (kb + 1) % NB * (MLA_KT * LDK), LDK, key0 + MLA_KT, n);
            vt.stash(Vst + (kb + 1) % NB * (MLA_KT * LDV), LDV, key0 + MLA_KT, n);
            lds_barrier();
        }
    }
    S *op = (S *)a.o + (size_t)b * s.Tq * s.H * s.dv + (size_t)h * s.dv;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = q0 + 16 * t + r;
        const float lt = sum4g(l[t]);
        const bool some = i + off < n; // (a query at or past the length has no key)
        const float inv = some && lt != 0.f ? 1.f / lt : 0.f; // (every score -inf: o = 0)
        if (i >= s.Tq) continue;
#pragma unroll
        for (int v = 0; v < MV; ++v) {
            const int c = 16 * v + 4 * g;
            const f32x4 x = some ? O[t][v] * inv : zero4();
            if (c < s.dv) store4(op + (size_t)i * s.H * s.dv + c, x);
        }
        if (a.lse && g == 0)
            a.lse[((size_t)b * s.Tq + i) * s.H + h] =
                some ? (m[t] + __builtin_amdgcn_logf(lt)) * 0.69314718055994531f : -INFINITY;
    }
}

template <bool BF, int DP, int DVP, int NW, int QT>
__global__ __launch_bounds__(NW * 64, 2) void mla_fwd_kernel(MlaFwdArgs a) {
    using H = MlaFwdShape<BF, DP, DVP, NW, QT>;
    __shared__ __align__(16) typename H::S Ks[H::NB * MLA_KT * H::LDK];
    __shared__ __align__(16) typename H::S Vs[H::NB * MLA_KT * H::LDV];
    const int nqb = (a.s.Tq + H::QB - 1) / H::QB, work = a.s.pair ? (nqb + 1) / 2 : nqb;
    int bh, i;
    head_block(blockIdx.x, a.s.B * a.s.H, work, bh, i);
    // the last queries walk longest: they come first; in pairs, a long walk with a short one
    const int parts = a.s.pair && i < nqb - 1 - i ? 2 : 1;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) {
        if (p) lds_barrier(); // (the first block's readers are done)
        mla_fwd_block<BF, DP, DVP, NW, QT>(a, bh, p ? i : nqb - 1 - i, Ks, Vs);
    }
}

template <bool BF, int DP, int DVP, int NW, int QT> hipError_t mla_fwd_start(MlaFwdArgs a, hipStream_t st) {
    const long long work = mla_work(a.s, (long long)a.s.B * a.s.H, a.s.Tq, NW * QT * 16);
    hipLaunchKernelGGL((mla_fwd_kernel<BF, DP, DVP, NW, QT>), dim3((unsigned)work), dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int DP, int DVP> hipError_t mla_fwd_run(const MlaFwdArgs &a, hipStream_t st) {
    if constexpr (BF) {
        constexpr int NW = mla_waves(DP, DVP);
        if (mla_large((long long)a.s.B * a.s.H, a.s.Tq, NW * 32, 8 / NW))
            return mla_fwd_start<BF, DP, DVP, NW, 2>(a, st);
    }
    return mla_fwd_start<BF, DP, DVP, 4, 1>(a, st);
}

template <bool BF> hipError_t mla_fwd_launch(const MlaFwdArgs &a, hipStream_t st) {
    const MlaPad pad = mla_pad(a.s);
    const int D = pad.d;
    if (D == 32) return mla_fwd_run<BF, 32, 32>(a, st);
    if (pad.dv == 64) {
        if (D == 64) return mla_fwd_run<BF, 64, 64>(a, st);
        if (D == 96) return mla_fwd_run<BF, 96, 64>(a, st);
        if (D == 128) return mla_fwd_run<BF, 128, 64>(a, st);
        return mla_fwd_run<BF, 192, 64>(a, st);
    }
    if (D == 64) return mla_fwd_run<BF, 64, 128>(a, st);
    if (D == 96) return mla_fwd_run<BF, 96, 128>(a, st);
    if (D == 128) return mla_fwd_run<BF, 128, 128>(a, st);
    return mla_fwd_run<BF, 192, 128>(a, st);
}

} // namespace gdn
