"""fp64 definitions of latent attention, the per-head norm with rotation and
the paged cache (TEST INFRASTRUCTURE ONLY, plain numpy loops over batch and
head; shares no code with the HIP library).

What include/gdn.h states, term by term. Pinned by central finite differences
(the gradients), by closed forms and by a loop over single keys
(tests/test_oracle_latent.py)."""
from __future__ import annotations

import numpy as np


def _keys(k, kr, b, h, H):
    """[Tk, dn + dr] keys head h of sequence b sees."""
    kk = k[b, :, h * k.shape[2] // H]
    return kk if kr is None else np.concatenate([kk, kr[b, :, h * kr.shape[2] // H]], 1)


def attn_probs(q, k, kr, lens, scale):
    """P [B,H,Tq,Tk] and lse [B,Tq,H] (-inf and a zero row where no key is seen)."""
    B, Tq, H, _ = q.shape
    Tk = k.shape[1]
    P = np.zeros((B, H, Tq, Tk))
    lse = np.full((B, Tq, H), -np.inf)
    for b in range(B):
        n = Tk if lens is None else min(max(int(lens[b]), 0), Tk)
        for h in range(H):
            kk = _keys(k, kr, b, h, H)
            for i in range(Tq):
                at = i + Tk - Tq
                if at >= n:
                    continue
                z = scale * (kk[:at + 1] @ q[b, i, h])
                m = z.max()
                w = np.exp(z - m)
                P[b, h, i, :at + 1] = w / w.sum()
                lse[b, i, h] = m + np.log(w.sum())
    return P, lse


def attn_fwd(q, k, kr, v, lens, scale):
    P, lse = attn_probs(q, k, kr, lens, scale)
    B, Tq, H, _ = q.shape
    o = np.zeros((B, Tq, H, v.shape[3]))
    for b in range(B):
        for h in range(H):
            o[b, :, h] = P[b, h] @ v[b, :, h * v.shape[2] // H]
    return o, lse, P


def attn_bwd(q, k, kr, v, lens, scale, do):
    """dq, dk, dkr (None without kr), dv of sum(do * o)."""
    o, _, P = attn_fwd(q, k, kr, v, lens, scale)
    H, dn = q.shape[2], k.shape[3]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dkr = None if kr is None else np.zeros_like(kr)
    for b in range(q.shape[0]):
        for h in range(H):
            hk = h * k.shape[2] // H
            dP = do[b, :, h] @ v[b, :, hk].T
            dS = P[b, h] * (dP - (do[b, :, h] * o[b, :, h]).sum(1, keepdims=True))
            dq[b, :, h] = scale * dS @ _keys(k, kr, b, h, H)
            dkk = scale * dS.T @ q[b, :, h]
            dk[b, :, hk] += dkk[:, :dn]
            if kr is not None:
                dkr[b, :, h * kr.shape[2] // H] += dkk[:, dn:]
            dv[b, :, hk] += P[b, h].T @ do[b, :, h]
    return dq, dk, dkr, dv


def step(q, cache, table, lens, dl, scale):
    """o [N,S,H,dl], lse [N,S,H]; rows of table entries outside the pool are masked."""
    N, S, H, _ = q.shape
    pages, page, d = cache.shape
    o = np.zeros((N, S, H, dl))
    lse = np.full((N, S, H), -np.inf)
    for n in range(N):
        m = min(max(int(lens[n]), 0), table.shape[1] * page)
        pos = np.arange(m)
        pg = table[n, pos // page]
        good = (pg >= 0) & (pg < pages)
        rows = cache[np.where(good, pg, 0), pos % page]
        for s in range(S):
            see = good & (pos <= m - S + s)
            if not see.any():
                continue
            r = rows[see]
            for h in range(H):
                z = scale * (r @ q[n, s, h])
                w = np.exp(z - z.max())
                o[n, s, h] = (w / w.sum()) @ r[:, :dl]
                lse[n, s, h] = z.max() + np.log(w.sum())
    return o, lse


def _halves(r, inter):
    i = np.arange(r // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + r // 2)


def turn(x, pos, freqs, inter, sign=1.0):
    """The last 2 len(freqs) columns of x [M,H,d] turned pairwise."""
    y = x.copy()
    if freqs is None or len(freqs) == 0:
        return y
    a, b = (x.shape[2] - 2 * len(freqs) + c for c in _halves(2 * len(freqs), inter))
    t = sign * pos.astype(np.float64)[:, None, None] * freqs
    y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    y[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
    return y


def norm_rope(x, w, pos, freqs, norm, eps, inter):
    """x [M,H,d] -> y."""
    z = x
    if norm:
        z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    return turn(z, pos, freqs, inter)


def norm_rope_bwd(dy, x, w, pos, freqs, norm, eps, inter):
    """dx, dw."""
    dz = turn(dy, pos, freqs, inter, -1.0)
    if not norm:
        return dz, None
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * inv
    g = dz * (1.0 if w is None else w)
    return inv * (g - xh * (g * xh).mean(-1, keepdims=True)), (dz * xh).sum((0, 1))


def write(c, kr, slots, cache, w, pos, freqs, norm, eps, inter):
    """The cache [slots, dl+dr] afterwards."""
    out = cache.copy()
    row = norm_rope(c[:, None], w, pos, None, norm, eps, inter)[:, 0]
    if kr is not None:
        row = np.concatenate([row, turn(kr[:, None], pos, freqs, inter)[:, 0]], 1)
    for i, s in enumerate(slots):
        if 0 <= s < len(cache):
            out[s] = row[i]
    return out


def page_plan(lens, new, table, stack, n_free, page, cap):
    """One sequence after the other, as the entry point's description reads."""
    N, cols = table.shape
    table, stack, lens = table.copy(), stack.copy(), [min(max(int(x), 0), cols * page) for x in lens]
    free = [int(x) for x in stack[:n_free]]
    for i in range(N):
        if new[i] < 0:
            free += [int(x) for x in table[i, :-(-lens[i] // page)]]
            lens[i] = 0
    free = free[:len(stack)]
    stack[:len(free)] = free
    granted, starts, slots, positions = np.zeros(N, np.int32), np.zeros(N + 1, np.int32), [], []
    tokens = pages = 0
    for i in range(N):
        ask = max(int(new[i]), 0)
        held, end = -(-lens[i] // page), -(-(lens[i] + ask) // page)
        if new[i] < 0 or end > cols:
            ask = 0
        need = end - held if ask else 0
        tokens, pages = tokens + ask, pages + need
        if ask and tokens <= cap and (need == 0 or pages <= len(free)):
            granted[i] = ask
    taken = 0
    for i in range(N):
        a = int(granted[i])
        held, end = -(-lens[i] // page), -(-(lens[i] + a) // page)
        for c in range(held, end):
            table[i, c] = free[len(free) - 1 - taken]
            taken += 1
        for t in range(lens[i], lens[i] + a):
            s = int(table[i, t // page]) * page + t % page
            slots.append(s if table[i, t // page] >= 0 else -1)
            positions.append(t)
        lens[i] += a
        starts[i + 1] = starts[i] + a
    pad = cap - len(slots)
    return {"starts": starts, "granted": granted, "lens": np.array(lens, np.int32).reshape(N),
            "n_free": np.array([len(free) - taken], np.int32), "slots": np.array(slots + [-1] * pad, np.int32),
            "positions": np.array(positions + [0] * pad, np.int32), "block_table": table, "free_pages": stack}
