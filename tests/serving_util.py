"""Bounds of the serving operators' tests, in the terms of latent_util (u = 2^-24
for fp32, h = 2^-8 for a bf16 operand or output): worst-case sums of what the
kernels round."""
import numpy as np

from latent_util import H16, U
from oracle import serving as ref


def shared(q, cache, table, lens, dl, ptable, plens, starts, scale, dtype):
    """fp64 o and lse of the step with prefixes and their bounds: those of the
    plain step over all rows a token sees; the parts a row set is cut into add
    a rescaling each, 2 u of the sums, of which there are fewer than rows."""
    h = H16 if dtype == "bf16" else 0.0
    o, lse, seen = ref.step_shared(q, cache, table, lens, dl, ptable, plens, starts, scale)
    to, tl = np.zeros_like(o), np.zeros_like(lse)
    d = q.shape[-1]
    for (n, s), r in seen.items():
        for g in range(q.shape[2]):
            p = np.exp(scale * r @ q[n, s, g] - lse[n, s, g])
            ez = ((d + 8) * U * scale * np.abs(r) @ np.abs(q[n, s, g])).max()
            rel = np.expm1(2 * ez + (3 * len(r) + 32) * U)
            to[n, s, g] = (rel + h + len(r) * U) * (p @ np.abs(r[:, :dl])) + (h + U) * np.abs(o[n, s, g])
            tl[n, s, g] = ez + (3 * len(r) + 32) * U + 2 * U * abs(lse[n, s, g])
    return o, to, lse, tl


def weights(q, cache, table, lens, lse, old, known, scale, decay):
    """fp64 weights and their bounds. The exponent is a dot product of d terms
    and two roundings of each of its sides, its exponential another; then a sum
    of S H terms and of what was there."""
    N, S, H, d = q.shape
    out = ref.weights(q, cache, table, lens, lse, old, known, scale, decay)
    tol = (S * H + 4) * U * np.abs(out) + 4 * U * np.abs(old)
    pages, page, _ = cache.shape
    for n in range(N):
        rows, good = ref._rows(cache, table[n], lens[n])
        for j in np.flatnonzero(good):
            for s in range(S):
                for h in range(H):
                    if j <= len(rows) - S + s and lse[n, s, h] > -np.inf:
                        z = scale * (q[n, s, h] @ rows[j])
                        e = (d + 8) * U * scale * (np.abs(q[n, s, h]) @ np.abs(rows[j])) + 4 * U * (
                            abs(z) + abs(lse[n, s, h])) + 4 * U
                        tol[table[n, j // page], j % page] += np.exp(z - lse[n, s, h]) * np.expm1(e)
    return out, tol


def commit(k, v, g, beta, A_log, counts, h, additive, logits, norm_k):
    """fp64 states and their bounds: the error of a state carried from token to
    token, with every product and sum's own rounding (8 u for a gate and what
    it enters an exponential with, (dk + 8) u for a sum over the keys)."""
    N, S, H, dk = k.shape
    out = ref.step_commit(k, v, g, beta, A_log, counts, h, additive, logits, norm_k)
    tol = np.zeros_like(out)
    sig = (lambda x: 1 / (1 + np.exp(-x))) if logits else (lambda x: x)
    for n in range(N):
        m, E = h[n].copy(), np.zeros_like(h[n])
        for t in range(min(max(int(counts[n]), 0), S)):
            for j in range(H):
                kk = k[n, t, j]
                rk = 0.0
                if norm_k:
                    kk = kk / np.sqrt((kk * kk).sum() + 1e-6)
                    rk = (dk / 2 + 8) * U
                ka = np.abs(kk)
                x = sig(g[n, t, j]) * np.exp(A_log[j])
                a, ra, b, rb = np.exp(-x), 16 * U * abs(x) + 8 * U, sig(beta[n, t, j]), 8 * U
                u = 0.0 if additive else kk @ m[j]
                eu = 0.0 if additive else ka @ E[j] + ((dk + 8) * U + rk) * (ka @ np.abs(m[j]))
                w = b * (v[n, t, j] - a * u)
                ew = (rb + 4 * U) * np.abs(b) * (np.abs(v[n, t, j]) + a * np.abs(u)) + b * a * (eu + ra * np.abs(u))
                E[j] = a * E[j] + (ra + 4 * U) * a * np.abs(m[j]) + np.outer(ka, ew + (rk + 4 * U) * np.abs(w))
                m[j] = a * m[j] + np.outer(kk, w)
        tol[n] = E * (1 + 1e-3) + U * np.abs(m)  # (second-order terms: below a thousandth of the first)
    return out, tol
