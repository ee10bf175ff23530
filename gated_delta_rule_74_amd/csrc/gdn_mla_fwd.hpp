// Causal attention of expanded latent-attention heads, forward.
//
//   z_ij = scale (q_i[:dn] . k_j + q_i[dn:] . kr_j),  o_i = sum_j softmax(z_i)_j v_j,
//   lse_i = log sum_j exp z_ij   over the keys j <= i + Tk - Tq, j < len_b
//
// in one pass over the keys with the running maximum and sum of the softmax.
// A workgroup takes NW / WS * QT * 16 queries of one head and walks the keys in
// tiles of 64 (128 with WS = 4) that all its waves share in LDS; a wave holds
// its QT * 16 queries in registers for the whole walk. WS waves hold the same
// queries where there are too few to fill the chip: each takes every WS-th 32
// keys of a tile, and their sums are joined at the end. The products are formed
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
// Wide heads (192 | 128) run at 0.8 of the rate a large matrix product reaches
// (T 16384, 16 heads on 4: 1.39 ms); at 96 | 64 the vector unit (exponentials,
// their sums and the mask: busy half of the time) adds to the matrix unit (a
// third) more than it runs beside it (B8 H16 T4096: 0.46 ms, 0.54 of that rate).
// More waves per SIMD (three, four) or value operands requested ahead do not
// change either. (Times here and in the backward: between events, warm.)
#pragma once

#include "gdn_mla.hpp"

namespace gdn {

constexpr float MLA_RAISE = 8.f; // see above

template <bool BF, int DP, int DVP, int NW, int QT, int WS> struct MlaFwdShape {
    using S = typename Op<BF>::S;
    static constexpr int LDK = DP + MLA_PAD<BF>, LDV = DVP + MLA_PAD<BF>, QB = NW / WS * QT * 16, BT = mla_tile(WS);
    // two tiles where a second workgroup still fits the CU's 160 KB beside them
    static constexpr int NB = 2 * BT * (LDK + LDV) * (int)sizeof(S) <= 80 * 1024 ? 2 : 1;
};

// Block qb of the queries of head bh.
template <bool BF, int DP, int DVP, int NW, int QT, int WS, class S>
__device__ __forceinline__ void mla_fwd_block(const MlaFwdArgs a, int bh, int qb, S *Kst, S *Vst, float2 *ML) {
    using H = MlaFwdShape<BF, DP, DVP, NW, QT, WS>;
    constexpr int LDK = H::LDK, LDV = H::LDV, NB = H::NB, NT = NW * 64, KS = DP / 32, MV = DVP / 16;
    const MlaArgs s = a.s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    constexpr int QB = H::QB, BT = H::BT;
    const int wg = wave / WS, wu = wave % WS; // the wave's queries, its part of each tile
    const int b = bh / s.H, h = bh % s.H, hk = h / (s.H / s.Hk);
    const int hr = s.Hr > 0 ? h / (s.H / s.Hr) : 0;
    const int D = s.dn + s.dr, off = s.Tk - s.Tq;
    const int n = s.lens ? min(max(s.lens[b], 0), s.Tk) : s.Tk;
    const int q0 = qb * QB + wg * QT * 16; // first query of this wave
    const size_t rq = (size_t)s.H * D, rk = (size_t)s.Hk * s.dn, rr = (size_t)s.Hr * s.dr, rv = (size_t)s.Hk * s.dv;
    const S *kp = (const S *)s.k + (size_t)b * s.Tk * rk + (size_t)hk * s.dn;
    const S *krp = s.dr > 0 ? (const S *)s.kr + (size_t)b * s.Tk * rr + (size_t)hr * s.dr : kp;
    const S *vp = (const S *)s.v + (size_t)b * s.Tk * rv + (size_t)hk * s.dv;

    // keys the workgroup has to see: those of its last query that is not padding
    const int last = min(min(qb * QB + QB, s.Tq) - 1 + off, n - 1);
    const int first = qb * QB + off; // position of its first query
    const int nt = first < n ? last / BT + 1 : 0;

    RowTile<BF, DP, BT, NT> kt;
    RowTile<BF, DVP, BT, NT> vt;
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
            Q[t][k] = row8_if(i < s.Tq && c < D, qp + (size_t)i * rq + c);
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
        const int key0 = kb * BT;
        if (kb + 1 < nt) {
            kt.fetch(key0 + BT, n);
            vt.fetch(key0 + BT, n);
        }
        if (key0 <= wlast && wfirst < n) {
            const S *K = Kst + kb % NB * (BT * LDK), *V = Vst + kb % NB * (BT * LDV);
            const bool mask = key0 + BT - 1 > wfirst || key0 + BT > n;
#pragma unroll 1
            for (int u = wu; u < BT / 32; u += WS) {
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
            kt.stash(Kst + (kb + 1) % NB * (BT * LDK), LDK, key0 + BT, n);
            vt.stash(Vst + (kb + 1) % NB * (BT * LDV), LDV, key0 + BT, n);
            lds_barrier();
        }
    }
    if constexpr (WS > 1) {
        // the parts of the walk: common maximum, sums rescaled to it and added
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            l[t] = sum4g(l[t]);
            if (g == 0) ML[(wave * QT + t) * 16 + r] = float2{m[t], l[t]};
        }
        lds_barrier();
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float mm = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < WS; ++w) mm = fmaxf(mm, ML[((wg * WS + w) * QT + t) * 16 + r].x);
#pragma unroll
            for (int w = 0; w < WS; ++w) { // (a part without keys counts for nothing)
                const float2 x = ML[((wg * WS + w) * QT + t) * 16 + r];
                sum += x.y == 0.f ? 0.f : x.y * exp2_fast(x.x - mm);
            }
            const float f = l[t] == 0.f ? 0.f : exp2_fast(m[t] - mm);
#pragma unroll
            for (int v = 0; v < MV; ++v) O[t][v] *= f;
            m[t] = mm;
            l[t] = sum;
        }
        if (!join_parts<MV, QT, WS>(O, (f32x4 *)Vst, wg, wu, lane)) return;
    }
    S *op = (S *)a.o + (size_t)b * s.Tq * s.H * s.dv + (size_t)h * s.dv;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = q0 + 16 * t + r;
        const float lt = WS > 1 ? l[t] : sum4g(l[t]);
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

template <bool BF, int DP, int DVP, int NW, int QT, int WS>
__global__ __launch_bounds__(NW * 64, WS == 4 ? 1 : 2) void mla_fwd_kernel(MlaFwdArgs a) {
    using H = MlaFwdShape<BF, DP, DVP, NW, QT, WS>;
    __shared__ float2 ML[WS > 1 ? NW * QT * 16 : 1];
    __shared__ __align__(16) typename H::S Ks[H::NB * H::BT * H::LDK];
    __shared__ __align__(16) typename H::S Vs[H::NB * H::BT * H::LDV];
    const int nqb = (a.s.Tq + H::QB - 1) / H::QB, work = a.s.pair ? (nqb + 1) / 2 : nqb;
    int bh, i;
    head_block(blockIdx.x, a.s.B * a.s.H, work, bh, i);
    // the last queries walk longest: they come first; in pairs, a long walk with a short one
    const int parts = a.s.pair && i < nqb - 1 - i ? 2 : 1;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) {
        if (p) lds_barrier(); // (the first block's readers are done)
        mla_fwd_block<BF, DP, DVP, NW, QT, WS>(a, bh, p ? i : nqb - 1 - i, Ks, Vs, ML);
    }
}

template <bool BF, int DP, int DVP, int NW, int QT, int WS> hipError_t mla_fwd_start(MlaFwdArgs a, hipStream_t st) {
    const long long work = mla_work(a.s, (long long)a.s.B * a.s.H, a.s.Tq, NW / WS * QT * 16);
    hipLaunchKernelGGL((mla_fwd_kernel<BF, DP, DVP, NW, QT, WS>), dim3((unsigned)work), dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int DP, int DVP> hipError_t mla_fwd_run(const MlaFwdArgs &a, hipStream_t st) {
    const long long heads = (long long)a.s.B * a.s.H;
    if constexpr (BF) {
        constexpr int NW = mla_waves(DP, DVP);
        if (mla_large(heads, a.s.Tq, NW * 32, 8 / NW)) return mla_fwd_start<BF, DP, DVP, NW, 2, 1>(a, st);
    }
    const int split = mla_split<BF>(heads, a.s.Tq, a.s.Tk, DP, DVP);
    if constexpr (mla_fits4<BF>(DP, DVP))
        if (split == 4) return mla_fwd_start<BF, DP, DVP, 4, 1, 4>(a, st);
    if (split == 2) return mla_fwd_start<BF, DP, DVP, 4, 1, 2>(a, st);
    return mla_fwd_start<BF, DP, DVP, 4, 1, 1>(a, st);
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
