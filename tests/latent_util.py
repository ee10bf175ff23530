"""Bounds and device helpers of the latent-attention tests.

The bounds are worst-case sums of what the kernels round, with
u = 2^-24 (fp32, half a step) and h = 2^-8 (bf16, half a step), 0 in fp32:

  z     a dot product of D terms, scaled:  ez = scale (D + 4) u sum|q||k| + 4 u |z|
  P     exp of that, from lse (or the running maximum), which carries ez too:
        eP = P (2 ez_max + (n + 16) u), n terms in the sum; h P more as an operand
  o     P v: sum eP |v| + h sum P |v| + h |o| (output) + n u sum P |v|
  lse   ez_max + (n + 16) u + u |lse|
  dS    P (dP - delta): the two factors' errors, h |dS| as an operand
and so on through the products, absolute values throughout. A tensor element
may be off by its own bound, plus TINY: a factor below 2^-126 (an exponential
far under its row's maximum, a product) may become zero, which takes at most
2^-126 times the other factor from each term; the tests' factors are below
2^12 and their sums have fewer than 2^14 terms, so all of them together stay
below 2^-126 2^12 2^14 = 2^-100."""
import numpy as np
import torch

from oracle import latent as ref

U, H16, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -100
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def dev(x, dtype):
    """A host array as a device tensor of the type, and the values it holds, in fp64."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[dtype])
    return t.cuda(), t.double().numpy()


def ints(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def within(name, got, want, tol):
    got = host(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fine = np.isfinite(want)
    assert (np.isfinite(got) == fine).all(), f"{name}: finite values differ"
    assert (got[~fine] == want[~fine]).all(), f"{name}: infinities differ"
    tol = np.broadcast_to(tol, want.shape) + TINY
    bad = fine & (np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)) > tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside, first at {i}: {got[i]} for {want[i]}, "
                             f"bound {tol[i]}")


def attention(q, k, kr, v, lens, scale, do, dtype):
    """fp64 results and their bounds: {name: (value, bound)}."""
    h = H16 if dtype == "bf16" else 0.0
    B, Tq, H, D = q.shape
    Tk, dn, dv = k.shape[1], k.shape[3], v.shape[3]
    o, lse, P = ref.attn_fwd(q, k, kr, v, lens, scale)
    grads = ref.attn_bwd(q, k, kr, v, lens, scale, do)
    tol = {n: np.zeros_like(x) for n, x in zip(("dq", "dk", "dkr", "dv"), grads) if x is not None}
    to, tl = np.zeros_like(o), np.zeros_like(lse)
    for b in range(B):
        for g in range(H):
            hk, hr = g * k.shape[2] // H, 0 if kr is None else g * kr.shape[2] // H
            kk, vv, p = ref._keys(k, kr, b, g, H), v[b, :, hk], P[b, g]
            az = scale * np.abs(q[b, :, g]) @ np.abs(kk).T  # bounds |z| too
            seen = p > 0
            ez = (((D + 4) * U + 4 * U) * np.where(seen, az, 0)).max(1, keepdims=True)
            n = seen.sum(1, keepdims=True)
            rel = np.expm1(2 * ez + (n + 16) * U)
            pv = p @ np.abs(vv)
            to[b, :, g] = (rel + h + n * U) * pv + (h + U) * np.abs(o[b, :, g])
            ls = np.where(np.isfinite(lse[b, :, g]), lse[b, :, g], 0.0)
            tl[b, :, g] = ez[:, 0] + (n[:, 0] + 16) * U + 2 * U * np.abs(ls)
            ado = np.abs(do[b, :, g])
            adp = ado @ np.abs(vv).T
            dp = do[b, :, g] @ vv.T
            dl = (do[b, :, g] * o[b, :, g]).sum(1, keepdims=True)
            ds = p * (dp - dl)
            edl = (ado * to[b, :, g]).sum(1, keepdims=True) + (dv + 4) * U * (ado * np.abs(o[b, :, g])).sum(
                1, keepdims=True)
            eds = rel * np.abs(ds) + p * ((dv + 4) * U * adp + edl + 4 * U * (np.abs(dp) + np.abs(dl))) * (1 + rel)
            eds = np.where(seen, eds, 0) + h * (np.abs(ds) + eds * seen)
            m = (p > 0).sum(0)[:, None]  # queries that see the key
            tol["dq"][b, :, g] += scale * (eds @ np.abs(kk) + (n + 4) * U * np.abs(ds) @ np.abs(kk))
            tk = scale * (eds.T @ np.abs(q[b, :, g]) + (m + 4) * U * np.abs(ds).T @ np.abs(q[b, :, g]))
            tol["dk"][b, :, hk] += tk[:, :dn]
            if kr is not None:
                tol["dkr"][b, :, hr] += tk[:, dn:]
            tol["dv"][b, :, hk] += (rel + h).T * p.T @ ado + (m + 4) * U * p.T @ ado
    out = {"o": (o, to), "lse": (lse, tl)}
    for n, x in zip(("dq", "dk", "dkr", "dv"), grads):
        if x is not None:
            out[n] = (x, tol[n] * (1 + h) + (h + (H + 4) * U) * np.abs(x))
    return out


def step(q, cache, table, lens, dl, scale, dtype):
    """fp64 o and lse of the paged step and their bounds."""
    h = H16 if dtype == "bf16" else 0.0
    o, lse = ref.step(q, cache, table, lens, dl, scale)
    to, tl = np.zeros_like(o), np.zeros_like(lse)
    pages, page, d = cache.shape
    for n in range(q.shape[0]):
        m = min(max(int(lens[n]), 0), table.shape[1] * page)
        pos = np.arange(m)
        pg = table[n, pos // page]
        good = (pg >= 0) & (pg < pages)
        rows = cache[np.where(good, pg, 0), pos % page]
        for s in range(q.shape[1]):
            r = rows[good & (pos <= m - q.shape[1] + s)]
            if not len(r):
                continue
            for g in range(q.shape[2]):
                z = scale * r @ q[n, s, g]
                p = np.exp(z - lse[n, s, g])
                ez = ((d + 8) * U * scale * np.abs(r) @ np.abs(q[n, s, g])).max()
                rel = np.expm1(2 * ez + (len(r) + 32) * U)
                to[n, s, g] = (rel + h + len(r) * U) * (p @ np.abs(r[:, :dl])) + (h + U) * np.abs(o[n, s, g])
                tl[n, s, g] = ez + (len(r) + 32) * U + 2 * U * abs(lse[n, s, g])
    return o, to, lse, tl
