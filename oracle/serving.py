"""fp64 definitions of the serving operators beside the plain step: shared
prefixes, cached rows' weights, eviction, page return, draft verification and
the state after accepted tokens (TEST INFRASTRUCTURE ONLY, plain numpy loops;
shares no code with the HIP library).

What include/gdn.h states, term by term. Pinned by closed forms, by
distributions and by the definitions of oracle.latent
(tests/test_oracle_serving.py)."""
from __future__ import annotations

import numpy as np


def _rows(cache, table, n):
    """The rows at positions 0 .. n - 1 of a table row, and which of them exist."""
    pages, page, _ = cache.shape
    n = min(max(int(n), 0), len(table) * page)
    pos = np.arange(n)
    pg = table[pos // page]
    good = (pg >= 0) & (pg < pages)
    return cache[np.where(good, pg, 0), pos % page], good


def groups(starts, N):
    """[(first, end)] of every group: starts clamped, one that goes back counts as the largest before it."""
    s = np.maximum.accumulate(np.clip(np.asarray(starts, np.int64), 0, N))
    return list(zip(s[:-1], s[1:]))


def step_shared(q, cache, table, lens, dl, ptable, plens, starts, scale):
    """o [N,S,H,dl], lse [N,S,H], and the rows each token sees ({(n, s): rows})."""
    N, S, H, _ = q.shape
    o, lse, seen = np.zeros((N, S, H, dl)), np.full((N, S, H), -np.inf), {}
    front = {}
    for g, (lo, hi) in enumerate(groups(starts, N)):
        for n in range(lo, hi):
            front[n] = g
    for n in range(N):
        own, good = _rows(cache, table[n], lens[n])
        pre = cache[:0, 0]
        if n in front:
            pre, there = _rows(cache, ptable[front[n]], plens[front[n]])
            pre = pre[there]
        for s in range(S):
            at = len(own) - S + s
            if at < 0:
                continue
            r = np.concatenate([pre, own[:at + 1][good[:at + 1]]])
            if not len(r):
                continue
            seen[n, s] = r
            for h in range(H):
                z = scale * (r @ q[n, s, h])
                w = np.exp(z - z.max())
                o[n, s, h] = (w / w.sum()) @ r[:, :dl]
                lse[n, s, h] = z.max() + np.log(w.sum())
    return o, lse, seen


def weights(q, cache, table, lens, lse, old, known, scale, decay):
    """The weights [pages, page] afterwards."""
    N, S, H, _ = q.shape
    pages, page, _ = cache.shape
    out = old.copy()
    for n in range(N):
        rows, good = _rows(cache, table[n], lens[n])
        m = len(rows)
        k = m - S if known is None else int(known[n])
        for j in range(m):
            if not good[j]:
                continue
            w = 0.0
            for s in range(S):
                if j <= m - S + s:
                    for h in range(H):
                        if lse[n, s, h] > -np.inf:
                            w += np.exp(scale * (q[n, s, h] @ rows[j]) - lse[n, s, h])
            at = table[n, j // page], j % page
            out[at] = (decay * old[at] if j < k else 0.0) + w
    return out


def evict(w, cache, table, lens, keep, first, recent):
    """weights, cache and lengths afterwards, row by row."""
    w, cache = w.copy(), cache.copy()
    pages, page, _ = cache.shape
    out = []
    for n in range(len(lens)):
        L = min(max(int(lens[n]), 0), table.shape[1] * page)
        k = min(max(int(keep[n]), 0), L)
        out.append(k)
        if k == L:
            continue
        a = min(first, k)
        b = min(recent, k - a)
        slot = [(int(table[n, j // page]), j % page) for j in range(L)]
        there = [0 <= s[0] < pages for s in slot]

        def rank(j):  # heavier first, then by position
            if not there[j]:
                return (2, 0.0, j)
            x = w[slot[j]]
            return (0, 0.0, j) if np.isnan(x) else (1, -x, j)

        best = sorted(range(a, L - b), key=rank)[:k - a - b]
        stay = list(range(a)) + sorted(best) + list(range(L - b, L))
        for to, j in enumerate(stay):  # (to <= j: what is read has not been written)
            if there[j] and there[to]:
                w[slot[to]], cache[slot[to]] = w[slot[j]], cache[slot[j]]
    return w, cache, np.array(out, np.int32)


def page_trim(lens, new, table, stack, n_free, page):
    """The stack and its height afterwards."""
    stack, F = stack.copy(), len(stack)
    top = min(max(int(n_free), 0), F)
    for n in range(len(lens)):
        L = min(max(int(lens[n]), 0), table.shape[1] * page)
        m = min(max(int(new[n]), 0), L)
        for c in range(-(-m // page), -(-L // page)):
            if top < F and table[n, c] >= 0:  # (below 0: no page)
                stack[top] = table[n, c]
                top += 1
    return stack, top


def distribution(z, t):
    """softmax(z / t), None where there is none."""
    top = z.max() if not np.isnan(z).any() else np.nan
    if not np.isfinite(top):
        return None
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(z == -np.inf, 0.0, np.exp((z - top) / t))
    return e / e.sum()


def draft_verify(z, draft, u, zq, lens, temp):
    """accepted [N], tokens [N,S+1], logprobs [N,S+1]."""
    N, S1, V = z.shape
    S = S1 - 1
    accepted, tokens, lp = np.zeros(N, np.int32), np.full((N, S1), -1, np.int32), np.zeros((N, S1))
    for n in range(N):
        L = S if lens is None else min(max(int(lens[n]), 0), S)
        t = 1.0 if temp is None else float(temp[n])
        greedy = not t > 0
        heat = 1.0 if greedy else t
        un = [min(max(float(x), 0.0), 1 - 2.0 ** -24) if x == x else 0.0 for x in u[n]]
        i, last = 0, None
        while True:
            p = distribution(z[n, i], heat)
            last = p
            if p is None or i == L:
                break
            x = int(draft[n, i])
            if greedy:
                if x != int(z[n, i].argmax()):
                    break
            elif not 0 <= x < V:
                break
            else:
                q = np.eye(1, V, x)[0] if zq is None else distribution(zq[n, i], heat)
                if q is None:
                    break
                if not un[i] * q[x] < p[x]:
                    last = np.maximum(p - q, 0.0)
                    if last.sum() < 2.0 ** -30:  # (as good as nothing: the distributions are the same)
                        last = p
                    break
            tokens[n, i], lp[n, i] = x, np.log(p[x])
            i += 1
        accepted[n] = i
        if p is None:
            continue
        if greedy:
            v = int(z[n, i].argmax())
        else:
            c = np.cumsum(last)
            v = int(np.searchsorted(c, un[S] * c[-1], side="right"))
        tokens[n, i], lp[n, i] = v, np.log(p[v])
    return accepted, tokens, lp


def step_commit(k, v, g, beta, A_log, counts, h, additive=False, logits=False, norm_k=False):
    """The states [N,H,dk,dv] afterwards."""
    N, S, H, _ = k.shape
    h = h.copy()
    sig = (lambda x: 1 / (1 + np.exp(-x))) if logits else (lambda x: x)
    for n in range(N):
        for t in range(min(max(int(counts[n]), 0), S)):
            for j in range(H):
                kk = k[n, t, j]
                if norm_k:
                    kk = kk / np.sqrt((kk * kk).sum() + 1e-6)
                a, b = np.exp(-sig(g[n, t, j]) * np.exp(A_log[j])), sig(beta[n, t, j])
                m = h[n, j]
                if not additive:
                    m = m - b * np.outer(kk, kk @ m)
                h[n, j] = a * m + b * np.outer(kk, v[n, t, j])
    return h
