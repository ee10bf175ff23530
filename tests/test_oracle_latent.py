"""Pins of the fp64 definitions the latent-attention tests compare with
(oracle/latent.py): central finite differences, closed forms, single-key sums."""
import numpy as np
import pytest

from oracle import latent as ref


def rnd(seed, *shape):
    return np.random.Generator(np.random.PCG64(seed)).standard_normal(shape)


def central(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        up = f()
        x[i] = old - eps
        g[i] = (up - f()) / (2 * eps)
        x[i] = old
    return g


@pytest.mark.parametrize("lens", [None, [5, 0, 2]])
def test_attention_gradients_are_the_differences(lens):
    B, Tq, Tk, H, Hk, Hr, dn, dr, dv = 3, 4, 5, 4, 2, 1, 3, 2, 3
    q, k, kr, v = rnd(1, B, Tq, H, dn + dr), rnd(2, B, Tk, Hk, dn), rnd(3, B, Tk, Hr, dr), rnd(4, B, Tk, Hk, dv)
    do = rnd(5, B, Tq, H, dv)
    grads = ref.attn_bwd(q, k, kr, v, lens, 0.7, do)

    def f():
        return (ref.attn_fwd(q, k, kr, v, lens, 0.7)[0] * do).sum()

    for x, g in zip((q, k, kr, v), grads):
        # differences of a function of size ~10: truncation 1e-12, rounding 10 * 2^-53 / 1e-6 ~ 1e-9
        assert np.abs(central(f, x) - g).max() < 1e-7


def test_attention_closed_forms():
    B, T, H, d = 1, 6, 2, 4
    v = rnd(7, B, T, H, d)
    o, lse, _ = ref.attn_fwd(np.zeros((B, T, H, d)), rnd(8, B, T, H, d), None, v, None, 1.0)
    for i in range(T):  # equal scores: the mean of the values so far, lse = log of their number
        assert np.allclose(o[0, i], v[0, :i + 1].mean(0), atol=1e-14) and np.allclose(lse[0, i], np.log(i + 1))
    o, lse, _ = ref.attn_fwd(rnd(9, B, T, H, d), rnd(8, B, T, H, d), None, v, [0], 1.0)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_step_is_attention_over_the_gathered_rows():
    N, S, H, dl, dr, page = 2, 2, 3, 4, 2, 3
    cache, q = rnd(1, 8, page, dl + dr), rnd(2, N, S, H, dl + dr)
    table, lens = np.array([[5, 2, 7], [1, 0, 3]]), np.array([8, 3])
    o, lse = ref.step(q, cache, table, lens, dl, 0.3)
    for n in range(N):
        rows = np.stack([cache[table[n, p // page], p % page] for p in range(lens[n])])[None, :, None]
        e, l, _ = ref.attn_fwd(q[n:n + 1], rows, None, rows[..., :dl], None, 0.3)
        assert np.allclose(o[n], e[0], atol=1e-14) and np.allclose(lse[n], l[0], atol=1e-14)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_gradients_are_the_differences(norm, inter):
    x, dy, w = rnd(1, 3, 2, 7), rnd(2, 3, 2, 7), rnd(3, 7) if norm else None
    pos, fr = np.array([0, 3, 1000000]), np.array([1.0, 0.1])
    dx, dw = ref.norm_rope_bwd(dy, x, w, pos, fr, norm, 1e-6, inter)

    def f():
        return (ref.norm_rope(x, w, pos, fr, norm, 1e-6, inter) * dy).sum()

    assert np.abs(central(f, x) - dx).max() < 1e-7
    if norm:
        assert np.abs(central(f, w) - dw).max() < 1e-7


def test_turn_keeps_lengths_and_adds_angles():
    x, fr = rnd(1, 4, 1, 6), np.array([0.5, 0.25, 0.125])
    a, b = np.array([1, 2, 3, 4]), np.array([10, 20, 30, 40])
    y = ref.turn(x, a, fr, False)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(ref.turn(y, b, fr, False), ref.turn(x, a + b, fr, False))
    assert np.allclose(ref.turn(y, a, fr, False, -1.0), x)


def test_page_plan_invariants():
    r = np.random.Generator(np.random.PCG64(3))
    for _ in range(40):
        N, page, cols = int(r.integers(1, 12)), int(r.integers(1, 5)), int(r.integers(1, 6))
        F = N * cols
        order, lens = r.permutation(F), r.integers(0, cols * page + 1, N)
        table, used = np.full((N, cols), -1), 0
        for i in range(N):
            h = -(-lens[i] // page)
            table[i, :h] = order[used:used + h]
            used += h
        stack = np.full(F, -1)
        stack[:F - used] = order[used:]
        n_free = int(r.integers(0, F - used + 1))
        new = r.integers(-1, 2 * page, N)
        p = ref.page_plan(lens, new, table, stack, n_free, page, int(r.integers(0, 3 * N * page)))
        held = [tuple(p["block_table"][i, :-(-p["lens"][i] // page)]) for i in range(N)]
        mine = [x for h in held for x in h] + list(p["free_pages"][:p["n_free"][0]])
        assert len(mine) == len(set(mine)) and -1 not in mine  # no page twice, none invented
        n = int(p["starts"][-1])
        s = p["slots"][:n]
        assert len(set(s)) == n and (s >= 0).all() and (p["slots"][n:] == -1).all()
        assert (p["granted"] <= np.maximum(new, 0)).all()
