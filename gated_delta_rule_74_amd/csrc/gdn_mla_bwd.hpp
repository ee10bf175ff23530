// Causal attention of expanded latent-attention heads, backward.
//
//   P_ij = exp(z_ij - lse_i),  delta_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j dS_ij [k_j | kr_j],   [dk_j | dkr_j] = scale sum_i dS_ij q_i,   dv_j = sum_i P_ij do_i
//
// The probabilities are formed again from the saved lse. Two kernels, so that
// every sum has one owner and a fixed order (no atomics):
//  * mla_bwd_q: a wave holds QT * 16 queries (q, do, and dq in accumulators)
//    and walks the keys; it also forms delta, which it leaves for the other;
//  * mla_bwd_k: a wave holds KT * 16 keys (k, v, and dk, dv in accumulators)
//    and walks the queries of every head that shares them, so a shared head's
//    gradient is summed in registers. Only the rotary key is shared by more
//    heads than that: each key head leaves its part in fp32 and mla_rope_sum
//    adds them up.
// In both, S and dP are formed with the walked rows as accumulator rows, so P
// and dS are at once the operand of the next product (as in the forward), and
// the walked tiles are read row by row for the first two products and by
// transposing reads for the last. The sums P and dS enter in bf16 (rounded to
// nearest even) when the tensors are bf16; everything else is fp32.
// S and dP are formed in both kernels: seven products instead of five, for
// which no sum needs atomics or a second pass. Bound by the matrix products
// and, at narrow heads, as much by the exponentials and the reads of LDS:
// B8 H16 T4096 56 + 32 | 56 0.65 + 0.81 ms (0.62 of the rate a large product
// reaches), T16384 16 heads on 4, 128 + 64 | 128 2.11 + 3.00 ms (0.79 of it).
#pragma once

#include "gdn_mla.hpp"

namespace gdn {

// Blocks with a row that sees at most so many keys form delta from the products,
// at the price of a second walk over them.
constexpr int MLA_EXACT = 256;

// dq of block qb of the queries of head bh, and their delta.
template <bool BF, int DP, int DVP, int NW, int QT, int WS, class S>
__device__ __forceinline__ void mla_bwd_q_block(const MlaBwdArgs a, int bh, int qb, S *Ks, S *Vs, float *Dx) {
    constexpr int LDK = DP + MLA_PAD<BF>, LDV = DVP + MLA_PAD<BF>, NT = NW * 64, KS = DP / 32, VS = DVP / 32,
                  MD = DP / 16;
    const MlaArgs s = a.s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    constexpr int QB = NW / WS * QT * 16, BT = mla_tile(WS);
    const int wg = wave / WS, wu = wave % WS; // the wave's queries, its part of each tile
    const int b = bh / s.H, h = bh % s.H, hk = h / (s.H / s.Hk);
    const int hr = s.Hr > 0 ? h / (s.H / s.Hr) : 0;
    const int D = s.dn + s.dr, off = s.Tk - s.Tq;
    const int n = s.lens ? min(max(s.lens[b], 0), s.Tk) : s.Tk;
    const int q0 = qb * QB + wg * QT * 16;
    const size_t rq = (size_t)s.H * D, rk = (size_t)s.Hk * s.dn, rr = (size_t)s.Hr * s.dr, rv = (size_t)s.Hk * s.dv,
                 ro = (size_t)s.H * s.dv;
    const S *kp = (const S *)s.k + (size_t)b * s.Tk * rk + (size_t)hk * s.dn;
    const S *krp = s.dr > 0 ? (const S *)s.kr + (size_t)b * s.Tk * rr + (size_t)hr * s.dr : kp;
    const S *vp = (const S *)s.v + (size_t)b * s.Tk * rv + (size_t)hk * s.dv;
    const int last = min(min(qb * QB + QB, s.Tq) - 1 + off, n - 1);
    const int nt = qb * QB + off < n ? last / BT + 1 : 0;

    RowTile<BF, DP, BT, NT> kt;
    RowTile<BF, DVP, BT, NT> vt;
    kt.init(kp, rk, s.dn, krp, rr, s.dr, tid);
    vt.init(vp, rv, s.dv, vp, 0, 0, tid);
    if (nt > 0) {
        kt.fetch(0, n);
        vt.fetch(0, n);
    }
    Frag<BF> Q[QT][KS], G[QT][VS]; // q and do as operand columns
    float lse2[QT], delta[QT];
    const S *qp = (const S *)s.q + (size_t)b * s.Tq * rq + (size_t)h * D;
    const S *gp = (const S *)a.dout + (size_t)b * s.Tq * ro + (size_t)h * s.dv;
    const S *op = (const S *)a.o + (size_t)b * s.Tq * ro + (size_t)h * s.dv;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = q0 + 16 * t + r;
        const bool live = i < s.Tq && i + off < n;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int c = 32 * k + 8 * g;
            Q[t][k] = row8_if(live && c < D, qp + (size_t)i * rq + c);
        }
        float d = 0.f;
#pragma unroll
        for (int k = 0; k < VS; ++k) {
            const int c = 32 * k + 8 * g;
            G[t][k] = row8_if(live && c < s.dv, gp + (size_t)i * ro + c);
            d += dot8(G[t][k], row8_if(live && c < s.dv, op + (size_t)i * ro + c));
        }
        const float saved = a.lse[((size_t)b * s.Tq + min(i, s.Tq - 1)) * s.H + h], ls = live ? saved : -INFINITY;
        delta[t] = sum4g(d);
        // a row without keys: every probability is exp2(z - inf) = 0
        lse2[t] = ls == -INFINITY ? INFINITY : ls * (float)LOG2E;
    }
    const float c2 = s.scale * (float)LOG2E;
    const int wlast = min(q0 + QT * 16 - 1 + off, n - 1), wfirst = q0 + off;
    // Where a row sees few keys, dP - delta cancels, and do . o with o rounded
    // to bf16 is not near enough: a first walk forms delta = sum_j P_ij dP_ij
    // from the products themselves. The block's first row sees the fewest.
    if (BF && qb * QB + off < MLA_EXACT) {
        float sum[QT] = {};
        for (int kb = 0; kb < nt; ++kb) {
            const int key0 = kb * BT, next = kb + 1 < nt ? key0 + BT : 0; // (0: for the walk below)
            lds_barrier();
            kt.stash(Ks, LDK, key0, n);
            vt.stash(Vs, LDV, key0, n);
            kt.fetch(next, n);
            vt.fetch(next, n);
            lds_barrier();
#pragma unroll 1
            for (int j = wu; j < BT / 16; j += WS)
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    f32x4 z = zero4(), dp = zero4();
#pragma unroll
                    for (int k = 0; k < KS; ++k) z = mma8(row8(Ks + (16 * j + r) * LDK + 32 * k + 8 * g), Q[t][k], z);
#pragma unroll
                    for (int k = 0; k < VS; ++k) dp = mma8(row8(Vs + (16 * j + r) * LDV + 32 * k + 8 * g), G[t][k], dp);
                    const int lim = min(q0 + 16 * t + r + off, n - 1) - key0 - 16 * j - 4 * g;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[t] = fmaf(e <= lim ? exp2_fast(fmaf(z[e], c2, -lse2[t])) : 0.f, dp[e], sum[t]);
                }
        }
#pragma unroll
        for (int t = 0; t < QT; ++t) delta[t] = sum4g(sum[t]);
        if constexpr (WS > 1) { // (the same order on both waves)
#pragma unroll
            for (int t = 0; t < QT; ++t)
                if (g == 0) Dx[(wave * QT + t) * 16 + r] = delta[t];
            lds_barrier();
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                delta[t] = 0.f;
#pragma unroll
                for (int w = 0; w < WS; ++w) delta[t] += Dx[((wg * WS + w) * QT + t) * 16 + r];
            }
        }
    }
    f32x4 dQ[QT][MD];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int v = 0; v < MD; ++v) dQ[t][v] = zero4();
    wait_vmem(); // (what is held is there: else its first use in the loop waits for the tile in flight)
    for (int kb = 0; kb < nt; ++kb) {
        const int key0 = kb * BT;
        lds_barrier(); // the previous tile's readers are done
        kt.stash(Ks, LDK, key0, n);
        vt.stash(Vs, LDV, key0, n);
        if (kb + 1 < nt) {
            kt.fetch(key0 + BT, n);
            vt.fetch(key0 + BT, n);
        }
        lds_barrier();
        const int nu = key0 > wlast || wfirst >= n ? 0 : BT / 32; // (0: no query of the wave sees the tile)
        const bool mask = key0 + BT - 1 > wfirst || key0 + BT > n;
#pragma unroll 1
        for (int u = wu; u < nu; u += WS) {
            // sixteen keys at a time: dP of only so many is held (192 | 128: 2.29 ms with all 32, 2.10 so; T 16384)
            f32x4 P[QT][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f32x4 dP[QT];
#pragma unroll
                for (int t = 0; t < QT; ++t) P[t][j] = dP[t] = zero4();
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const Frag<BF> kf = row8(Ks + (32 * u + 16 * j + r) * LDK + 32 * k + 8 * g);
#pragma unroll
                    for (int t = 0; t < QT; ++t) P[t][j] = mma8(kf, Q[t][k], P[t][j]);
                }
#pragma unroll
                for (int k = 0; k < VS; ++k) {
                    const Frag<BF> vf = row8(Vs + (32 * u + 16 * j + r) * LDV + 32 * k + 8 * g);
#pragma unroll
                    for (int t = 0; t < QT; ++t) dP[t] = mma8(vf, G[t][k], dP[t]);
                }
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const int lim = mask ? min(q0 + 16 * t + r + off, n - 1) - key0 - 32 * u - 16 * j - 4 * g : 3;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        P[t][j][e] =
                            exp2_fast(fmaf(e <= lim ? P[t][j][e] : -INFINITY, c2, -lse2[t])) * (dP[t][e] - delta[t]);
                }
                in_flight();
            }
            Frag<BF> ds[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t) ds[t] = acc8<BF>(P[t][0], P[t][1]);
#pragma unroll
            for (int v = 0; v < MD; ++v) {
                const Frag<BF> kf = col8(Ks, LDK, 32 * u, 16 * v, lane);
#pragma unroll
                for (int t = 0; t < QT; ++t) dQ[t][v] = mma8(kf, ds[t], dQ[t][v]);
            }
        }
    }
    if constexpr (WS > 1) { // the parts of the walk, one after the other
        if (!join_parts<MD, QT, WS>(dQ, (f32x4 *)Ks, wg, wu, lane)) return;
    }
    S *dqp = (S *)a.dq + (size_t)b * s.Tq * rq + (size_t)h * D;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = q0 + 16 * t + r;
        if (i >= s.Tq) continue;
        if (g == 0) a.delta[((size_t)b * s.H + h) * s.Tq + i] = delta[t];
#pragma unroll
        for (int v = 0; v < MD; ++v) {
            const int c = 16 * v + 4 * g;
            if (c < D) store4(dqp + (size_t)i * rq + c, dQ[t][v] * s.scale);
        }
    }
}

template <bool BF, int DP, int DVP, int NW, int QT, int WS>
__global__ __launch_bounds__(NW * 64, WS == 4 ? 1 : 2) void mla_bwd_q_kernel(MlaBwdArgs a) {
    using S = typename Op<BF>::S;
    constexpr int QB = NW / WS * QT * 16, BT = mla_tile(WS);
    __shared__ __align__(16) S Ks[BT * (DP + MLA_PAD<BF>)];
    __shared__ __align__(16) S Vs[BT * (DVP + MLA_PAD<BF>)];
    __shared__ float Dx[WS > 1 ? NW * QT * 16 : 1];
    const int nqb = (a.s.Tq + QB - 1) / QB, work = a.s.pair ? (nqb + 1) / 2 : nqb;
    int bh, i;
    head_block(blockIdx.x, a.s.B * a.s.H, work, bh, i);
    // the last queries walk longest (a block begins with a barrier, so the tiles may be reused)
    const int parts = a.s.pair && i < nqb - 1 - i ? 2 : 1;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) mla_bwd_q_block<BF, DP, DVP, NW, QT, WS>(a, bh, p ? i : nqb - 1 - i, Ks, Vs, Dx);
}

// x[t][j] += the products of N walked operands with the held ones of tile t.
template <int N, bool BF, int T>
__device__ __forceinline__ void times(f32x4 (&x)[T][2], int j, const Frags<BF, N> &f, const Frag<BF> (&held)[T][N]) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < T; ++t) x[t][j] = mma8(f.f[k], held[t][k], x[t][j]);
}

// dk, dkr and dv of block kb of the keys of key head bh.
template <bool BF, int DP, int DVP, int NW, int KT, int WS, class S>
__device__ __forceinline__ void mla_bwd_k_block(const MlaBwdArgs a, int bh, int kb, S *Qs, S *Gs, float *Ls,
                                                float *Ds) {
    constexpr int LDQ = DP + MLA_PAD<BF>, LDG = DVP + MLA_PAD<BF>, NT = NW * 64, KS = DP / 32, VS = DVP / 32,
                  MD = DP / 16, MV = DVP / 16;
    const MlaArgs s = a.s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    constexpr int KB = NW / WS * KT * 16, BT = mla_tile(WS);
    const int wg = wave / WS, wu = wave % WS; // the wave's keys, its part of each tile
    const int b = bh / s.Hk, hk = bh % s.Hk, per = s.H / s.Hk;
    const int hr = s.Hr > 0 ? hk / (s.Hk / s.Hr) : 0;
    const int D = s.dn + s.dr, off = s.Tk - s.Tq;
    const int n = s.lens ? min(max(s.lens[b], 0), s.Tk) : s.Tk;
    const int key0 = kb * KB, w0 = key0 + wg * KT * 16; // first key of the workgroup, of the wave
    const size_t rq = (size_t)s.H * D, rk = (size_t)s.Hk * s.dn, rr = (size_t)s.Hr * s.dr, rv = (size_t)s.Hk * s.dv,
                 ro = (size_t)s.H * s.dv;
    // queries that see a key of this workgroup: q_lo .. nq - 1, a tile-aligned walk of each head
    const int nq = min(s.Tq, n - off);
    const int t_lo = max(key0 - off, 0) / BT;
    const int tiles = key0 < n && nq > t_lo * BT ? (nq + BT - 1) / BT - t_lo : 0;
    const int total = tiles * per;

    RowTile<BF, DP, BT, NT> qt;
    RowTile<BF, DVP, BT, NT> gt;
    const S *qp = (const S *)s.q + (size_t)b * s.Tq * rq + (size_t)hk * per * D; // first of the heads
    const S *gp = (const S *)a.dout + (size_t)b * s.Tq * ro + (size_t)hk * per * s.dv;
    qt.init(qp, rq, D, qp, 0, 0, tid);
    gt.init(gp, ro, s.dv, gp, 0, 0, tid);
    float lreg = 0.f, dreg = 0.f;
    auto fetch = [&](int x) {
        const int h = hk * per + x / tiles, row0 = (t_lo + x % tiles) * BT;
        qt.fetch(row0, nq, (size_t)(x / tiles) * D);
        gt.fetch(row0, nq, (size_t)(x / tiles) * s.dv);
        if (tid < BT) {
            const int i = min(row0 + tid, nq - 1);
            lreg = a.lse[((size_t)b * s.Tq + i) * s.H + h];
            dreg = a.delta[((size_t)b * s.H + h) * s.Tq + i];
        }
    };
    if (total > 0) fetch(0);
    Frag<BF> K[KT][KS], V[KT][VS]; // keys and values as operand columns
    const S *kp = (const S *)s.k + (size_t)b * s.Tk * rk + (size_t)hk * s.dn;
    const S *krp = s.dr > 0 ? (const S *)s.kr + (size_t)b * s.Tk * rr + (size_t)hr * s.dr : kp;
    const S *vp = (const S *)s.v + (size_t)b * s.Tk * rv + (size_t)hk * s.dv;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int j = w0 + 16 * t + r;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int c = 32 * k + 8 * g;
            K[t][k] = row8_if(j < n && c < D, c < s.dn ? kp + (size_t)j * rk + c : krp + (size_t)j * rr + (c - s.dn));
        }
#pragma unroll
        for (int k = 0; k < VS; ++k) {
            const int c = 32 * k + 8 * g;
            V[t][k] = row8_if(j < n && c < s.dv, vp + (size_t)j * rv + c);
        }
    }
    f32x4 dK[KT][MD], dV[KT][MV];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
        for (int v = 0; v < MD; ++v) dK[t][v] = zero4();
#pragma unroll
        for (int v = 0; v < MV; ++v) dV[t][v] = zero4();
    }
    const float c2 = s.scale * (float)LOG2E;
    wait_vmem(); // (as above)
    for (int x = 0; x < total; ++x) {
        const int row0 = (t_lo + x % tiles) * BT;
        lds_barrier();
        qt.stash(Qs, LDQ, row0, nq);
        gt.stash(Gs, LDG, row0, nq);
        if (tid < BT) {
            Ls[tid] = lreg == -INFINITY ? INFINITY : lreg * (float)LOG2E;
            Ds[tid] = dreg;
        }
        if (x + 1 < total) fetch(x + 1);
        lds_barrier();
        // (0: no query of the tile sees a key of this wave)
        const int nu = row0 + BT - 1 + off < w0 || w0 >= n ? 0 : BT / 32;
        const bool mask = row0 + off < w0 + KT * 16 - 1 || row0 + BT > nq || w0 + KT * 16 > n;
#pragma unroll 1
        for (int u = wu; u < nu; u += WS) {
            f32x4 P[KT][2], dP[KT][2];
            // operands are requested one group ahead of the products that use them
            Frags<BF, KS> qa, qb;
            Frags<BF, VS> ga, gb;
#pragma unroll
            for (int t = 0; t < KT; ++t) P[t][0] = P[t][1] = dP[t][0] = dP[t][1] = zero4();
            qa.rows(Qs, LDQ, 32 * u, lane);
            in_flight();
            ga.rows(Gs, LDG, 32 * u, lane);
            in_flight();
            times<KS>(P, 0, qa, K);
            in_flight();
            qb.rows(Qs, LDQ, 32 * u + 16, lane);
            in_flight();
            times<VS>(dP, 0, ga, V);
            in_flight();
            gb.rows(Gs, LDG, 32 * u + 16, lane);
            in_flight();
            times<KS>(P, 1, qb, K);
            in_flight();
            constexpr int CV = MV < 4 ? MV : 4, CK = MD < 3 ? MD : MD % 4 == 0 ? 4 : 3; // operands requested at a time
            Frags<BF, CV> vc;
            vc.cols(Gs, LDG, 32 * u, 0, lane);
            in_flight();
            times<VS>(dP, 1, gb, V);
            Frag<BF> pf[KT], sf[KT];
#pragma unroll
            for (int t = 0; t < KT; ++t) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i0 = 32 * u + 16 * j + 4 * g; // first of this lane's four rows
                    const f32x4 ls = *reinterpret_cast<const f32x4 *>(Ls + i0);
                    const f32x4 dl = *reinterpret_cast<const f32x4 *>(Ds + i0);
                    if (mask) {
                        // row e sees this lane's key from row j_at - off on; no key at or past n
                        const int j_at = w0 + 16 * t + r, lo = j_at - off - row0 - i0, hi = nq - row0 - i0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            P[t][j][e] = e >= lo && e < hi && j_at < n ? P[t][j][e] : -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        P[t][j][e] = exp2_fast(fmaf(P[t][j][e], c2, -ls[e]));
                        dP[t][j][e] = P[t][j][e] * (dP[t][j][e] - dl[e]);
                    }
                }
                pf[t] = acc8<BF>(P[t][0], P[t][1]);
                sf[t] = acc8<BF>(dP[t][0], dP[t][1]);
            }
            // the next group of operands is requested before the products of the one at hand
            Frags<BF, CK> kc;
#pragma unroll
            for (int v0 = 0; v0 < MV; v0 += CV) {
                Frags<BF, CV> nv;
                in_flight();
                if (v0 + CV < MV) nv.cols(Gs, LDG, 32 * u, 16 * (v0 + CV), lane);
                else kc.cols(Qs, LDQ, 32 * u, 0, lane);
                in_flight();
#pragma unroll
                for (int v = 0; v < CV; ++v)
#pragma unroll
                    for (int t = 0; t < KT; ++t) dV[t][v0 + v] = mma8(vc.f[v], pf[t], dV[t][v0 + v]);
                vc = nv;
            }
#pragma unroll
            for (int v0 = 0; v0 < MD; v0 += CK) {
                Frags<BF, CK> nk;
                in_flight();
                if (v0 + CK < MD) nk.cols(Qs, LDQ, 32 * u, 16 * (v0 + CK), lane);
                in_flight();
#pragma unroll
                for (int v = 0; v < CK; ++v)
#pragma unroll
                    for (int t = 0; t < KT; ++t) dK[t][v0 + v] = mma8(kc.f[v], sf[t], dK[t][v0 + v]);
                kc = nk;
            }
        }
    }
    if constexpr (WS > 1) {
        join_parts<MD, KT, WS>(dK, (f32x4 *)Qs, wg, wu, lane);
        if (!join_parts<MV, KT, WS>(dV, (f32x4 *)Gs, wg, wu, lane)) return;
    }
    S *dkp = (S *)a.dk + (size_t)b * s.Tk * rk + (size_t)hk * s.dn;
    S *dvp = (S *)a.dv + (size_t)b * s.Tk * rv + (size_t)hk * s.dv;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int j = w0 + 16 * t + r;
        if (j >= s.Tk) continue;
#pragma unroll
        for (int v = 0; v < MV; ++v) {
            const int c = 16 * v + 4 * g;
            if (c < s.dv) store4(dvp + (size_t)j * rv + c, dV[t][v]);
        }
#pragma unroll
        for (int v = 0; v < MD; ++v) {
            const int c = 16 * v + 4 * g;
            const f32x4 x = dK[t][v] * s.scale;
            if (c < s.dn) {
                store4(dkp + (size_t)j * rk + c, x);
            } else if (c < D) {
                if (a.dkr_part)
                    store4(a.dkr_part + (((size_t)b * s.Tk + j) * s.Hk + hk) * s.dr + (c - s.dn), x);
                else
                    store4((S *)a.dkr + ((size_t)b * s.Tk + j) * rr + (size_t)hr * s.dr + (c - s.dn), x);
            }
        }
    }
}

// Waves per SIMD. Two leave a wave 256 registers for its operands and both
// accumulators, one 512. bf16: pairs of key tiles beyond 96 | 64 run one (96 |
// 64: 0.87 ms with two, 1.43 with one at the layer shape; 192 | 128, T 16384:
// 3.2 ms as pairs with one wave, 3.8 as single tiles with two); two waves of
// single tiles spill a little at 192 | 128 and are still ahead (B1 T2048, 8
// heads: 65 us, 68 with one). fp32 holds twice the registers, single tiles
// throughout: up to 192 columns in all two waves, with what they spill, are
// ahead (B4 T2048 H16, 56 + 32 | 56: 0.72 ms, 0.82 with one; 96 + 32 | 64: 0.89
// and 0.97), beyond that one (128 | 128: 1.51 ms with two, 1.27 with one; B2
// T700, 8 heads: 140 and 72 us; 192 | 64: 1.51 and 1.27; 96 | 128: 1.26, 1.12).
template <bool BF> constexpr int mla_bwd_k_waves(int kt, int dp, int dvp) {
    if (!BF) return dp + dvp <= 192 ? 2 : 1;
    return kt == 1 || dp + dvp <= 160 ? 2 : 1;
}

template <bool BF, int DP, int DVP, int NW, int KT, int WS>
__global__ __launch_bounds__(NW * 64, WS == 4 ? 1 : mla_bwd_k_waves<BF>(KT, DP, DVP)) void mla_bwd_k_kernel(MlaBwdArgs a) {
    using S = typename Op<BF>::S;
    constexpr int KB = NW / WS * KT * 16, BT = mla_tile(WS);
    __shared__ __align__(16) S Qs[BT * (DP + MLA_PAD<BF>)];
    __shared__ __align__(16) S Gs[BT * (DVP + MLA_PAD<BF>)];
    __shared__ __align__(16) float Ls[BT], Ds[BT];
    const int nkb = (a.s.Tk + KB - 1) / KB, work = a.s.pair ? (nkb + 1) / 2 : nkb;
    int bh, i;
    head_block(blockIdx.x, a.s.B * a.s.Hk, work, bh, i);
    // the first keys are seen by the most queries
    const int parts = a.s.pair && i < nkb - 1 - i ? 2 : 1;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) mla_bwd_k_block<BF, DP, DVP, NW, KT, WS>(a, bh, p ? nkb - 1 - i : i, Qs, Gs, Ls, Ds);
}

template <bool BF, int DP, int DVP, int NW, int QT, int WS> hipError_t mla_bwd_q_start(MlaBwdArgs a, hipStream_t st) {
    const long long work = mla_work(a.s, (long long)a.s.B * a.s.H, a.s.Tq, NW / WS * QT * 16);
    hipLaunchKernelGGL((mla_bwd_q_kernel<BF, DP, DVP, NW, QT, WS>), dim3((unsigned)work), dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int DP, int DVP> hipError_t mla_bwd_q_run(const MlaBwdArgs &a, hipStream_t st) {
    const long long heads = (long long)a.s.B * a.s.H;
    if constexpr (BF) {
        constexpr int NW = mla_waves(DP, DVP);
        if (mla_large(heads, a.s.Tq, NW * 32, 8 / NW)) return mla_bwd_q_start<BF, DP, DVP, NW, 2, 1>(a, st);
    }
    const int split = mla_split<BF>(heads, a.s.Tq, a.s.Tk, DP, DVP);
    if constexpr (mla_fits4<BF>(DP, DVP))
        if (split == 4) return mla_bwd_q_start<BF, DP, DVP, 4, 1, 4>(a, st);
    if (split == 2) return mla_bwd_q_start<BF, DP, DVP, 4, 1, 2>(a, st);
    return mla_bwd_q_start<BF, DP, DVP, 4, 1, 1>(a, st);
}
template <bool BF, int DP, int DVP, int NW, int KT, int WS> hipError_t mla_bwd_k_start(MlaBwdArgs a, hipStream_t st) {
    const long long work = mla_work(a.s, (long long)a.s.B * a.s.Hk, a.s.Tk, NW / WS * KT * 16);
    hipLaunchKernelGGL((mla_bwd_k_kernel<BF, DP, DVP, NW, KT, WS>), dim3((unsigned)work), dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int DP, int DVP> hipError_t mla_bwd_k_run(const MlaBwdArgs &a, hipStream_t st) {
    const long long heads = (long long)a.s.B * a.s.Hk;
    if constexpr (BF)
        if (mla_large(heads, a.s.Tk, 128, mla_bwd_k_waves<BF>(2, DP, DVP)))
            return mla_bwd_k_start<BF, DP, DVP, 4, 2, 1>(a, st);
    const int split = mla_split<BF>(heads, a.s.Tk, (long long)a.s.Tq * (a.s.H / a.s.Hk), DP, DVP);
    if constexpr (mla_fits4<BF>(DP, DVP))
        if (split == 4) return mla_bwd_k_start<BF, DP, DVP, 4, 1, 4>(a, st);
    if (split == 2) return mla_bwd_k_start<BF, DP, DVP, 4, 1, 2>(a, st);
    return mla_bwd_k_start<BF, DP, DVP, 4, 1, 1>(a, st);
}

template <bool BF, bool Q, int DP, int DVP> hipError_t mla_bwd_run(const MlaBwdArgs &a, hipStream_t st) {
    if constexpr (Q) return mla_bwd_q_run<BF, DP, DVP>(a, st);
    else return mla_bwd_k_run<BF, DP, DVP>(a, st);
}
template <bool BF, bool Q> hipError_t mla_bwd_launch(const MlaBwdArgs &a, hipStream_t st) {
    const MlaPad pad = mla_pad(a.s);
    const int D = pad.d;
    if (D == 32) return mla_bwd_run<BF, Q, 32, 32>(a, st);
    if (pad.dv == 64) {
        if (D == 64) return mla_bwd_run<BF, Q, 64, 64>(a, st);
        if (D == 96) return mla_bwd_run<BF, Q, 96, 64>(a, st);
        if (D == 128) return mla_bwd_run<BF, Q, 128, 64>(a, st);
        return mla_bwd_run<BF, Q, 192, 64>(a, st);
    }
    if (D == 64) return mla_bwd_run<BF, Q, 64, 128>(a, st);
    if (D == 96) return mla_bwd_run<BF, Q, 96, 128>(a, st);
    if (D == 128) return mla_bwd_run<BF, Q, 128, 128>(a, st);
    return mla_bwd_run<BF, Q, 192, 128>(a, st);
}

} // namespace gdn
