"""Pins of the serving operators' fp64 definitions (oracle/serving.py): closed
forms, agreement with the plain step's definition where the two meet, and the
distribution that draft verification promises."""
import numpy as np

from oracle import latent, serving


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def paged(g, N, S, H, d, page, lens):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = g.permutation(pages)
    table, at = np.full((N, max(max(need), 1)), -1, np.int32), 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
    return g.standard_normal((N, S, H, d)), g.standard_normal((pages, page, d)), table, order[at:]


def test_a_prefix_of_whole_pages_is_a_longer_table():
    g = rng(1)
    lens, page, P = [3, 0, 5, 1], 4, 8
    q, cache, table, _ = paged(g, 5, 2, 3, 8, page, lens + [P])
    q, ptable = q[:4], table[4:, :P // page]
    own = table[:4]
    o, lse, _ = serving.step_shared(q, cache, own, lens, 6, ptable, [P], [1, 4], 0.3)
    long = np.concatenate([np.repeat(ptable, 4, 0), own], 1)
    for n in range(4):
        t, m = (own, lens[n]) if n == 0 else (long, lens[n] + P)
        want, wl = latent.step(q[n:n + 1], cache, t[n:n + 1], [m], 6, 0.3)
        for s in range(2):
            if lens[n] - 2 + s < 0:  # padding: no token
                assert not o[n, s].any() and (lse[n, s] == -np.inf).all()
            else:
                np.testing.assert_allclose(o[n, s], want[0, s], atol=1e-14)
                np.testing.assert_allclose(lse[n, s], wl[0, s], atol=1e-13)


def test_starts_that_go_back_count_as_the_largest_before():
    assert serving.groups([0, 5, 3, 9], 7) == [(0, 5), (5, 5), (5, 7)]
    assert serving.groups([-3, 2], 1) == [(0, 1)]


def test_weights_of_a_token_add_up_to_its_heads():
    g = rng(2)
    lens = [7, 1, 0]
    q, cache, table, _ = paged(g, 3, 1, 4, 8, 4, lens)
    _, lse = latent.step(q, cache, table, lens, 8, 0.5)
    old = np.full(cache.shape[:2], 3.0)
    w = serving.weights(q, cache, table, lens, lse, old, [0, 0, 0], 0.5, 1.0)
    for n, m in enumerate(lens):
        got = sum(w[table[n, j // 4], j % 4] for j in range(m))
        assert abs(got - (4 if m else 0)) < 1e-12
    kept = serving.weights(q, cache, table, lens, lse, old, None, 0.5, 0.5)  # the last row begins anew
    for n, m in enumerate(lens):
        for j in range(m):
            at = table[n, j // 4], j % 4
            assert abs(kept[at] - w[at] - (1.5 if j < m - 1 else 0)) < 1e-12
    held = {(table[n, j // 4], j % 4) for n, m in enumerate(lens) for j in range(m)}
    assert all(w[p, i] == 3 for p in range(w.shape[0]) for i in range(4) if (p, i) not in held)


def test_eviction_keeps_the_heaviest_in_order():
    g = rng(3)
    _, cache, table, _ = paged(g, 1, 1, 1, 4, 3, [10])
    w = np.zeros(cache.shape[:2])
    at = [(table[0, j // 3], j % 3) for j in range(10)]
    for j, x in enumerate([5, 1, 4, 1, 4, np.nan, -0.0, 0.0, 2, 9]):
        w[at[j]] = x
    for keep, first, recent, stay in ((10, 0, 0, range(10)), (12, 0, 0, range(10)), (0, 2, 2, []), (-1, 0, 0, []),
                                      (3, 0, 0, [0, 5, 9]), (5, 0, 0, [0, 2, 4, 5, 9]), (4, 0, 0, [0, 2, 5, 9]),
                                      (8, 0, 0, [0, 1, 2, 3, 4, 5, 8, 9]), (9, 0, 0, [0, 1, 2, 3, 4, 5, 6, 8, 9]),
                                      (4, 2, 1, [0, 1, 5, 9]), (3, 2, 4, [0, 1, 9]), (2, 5, 1, [0, 1])):
        ww, cc, n = serving.evict(w, cache, table, [10], [keep], first, recent)
        assert n[0] == len(stay)
        for to, j in enumerate(stay):
            np.testing.assert_array_equal(cc[at[to]], cache[at[j]])
            np.testing.assert_array_equal(ww[at[to]], w[at[j]])
        for j in range(len(stay), 10):
            np.testing.assert_array_equal(cc[at[j]], cache[at[j]])


def test_page_trim_gives_back_what_a_plan_would_take_again():
    stack, top = serving.page_trim([9, 4, 0, 5], [4, 4, 3, -1], np.arange(12).reshape(4, 3), np.array([70, 71, -1, -1, -1]),
                                   2, 4)
    assert list(stack) == [70, 71, 1, 2, 9] and top == 5  # (10 found no room)


def test_page_trim_gives_back_pages_alone():
    stack, top = serving.page_trim([12, 8, 12], [0, 4, 5], np.array([[3, -1, 7], [5, -4, 6], [-1, 1, -2]]),
                                   np.array([70, 71, -9, -9, -9, -9]), 2, 4)
    assert list(stack) == [70, 71, 3, 7, -9, -9] and top == 4  # (the others hold 1, and no pages, behind their lengths)


def test_verified_drafts_are_distributed_as_the_target():
    """Chance of each emitted token over a fine grid of both random numbers: the target's own."""
    z, zq = np.log(np.array([0.5, 0.2, 0.2, 0.1])), np.log(np.array([0.1, 0.6, 0.2, 0.1]))
    n = 1000
    grid = (np.arange(n) + 0.5) / n
    for q in (zq, None):
        chance = np.zeros(4)
        for x, px in enumerate(np.exp(zq) if q is not None else [0, 1, 0, 0]):
            a, t, lp = serving.draft_verify(np.tile(np.stack([z, zq]), (n, 1, 1)), np.full((n, 1), x),
                                            np.stack([grid, np.full(n, 0.5)], 1),
                                            None if q is None else np.tile(q, (n, 1, 1)), None, None)
            hit = a.mean()
            np.testing.assert_allclose(lp[np.arange(n), 0], z[t[:, 0]], atol=1e-12)
            _, back, _ = serving.draft_verify(np.tile(np.stack([z, zq]), (n, 1, 1)), np.full((n, 1), x),
                                              np.stack([np.full(n, 1.0), grid], 1),
                                              None if q is None else np.tile(q, (n, 1, 1)), None, None)
            chance[x] += px * hit
            if hit < 1:
                chance += px * (1 - hit) * np.bincount(back[:, 0], minlength=4) / n
        np.testing.assert_allclose(chance, np.exp(z), atol=3e-3)  # (two grids of a thousand points)


def test_a_rejected_draft_that_leaves_nothing_draws_from_the_target():
    """Equal distributions, and a draft to which they give nothing: masked, or below what fp64 holds."""
    for z, t in (([0., 1, -np.inf], 1.0), ([0., 0.5, -9], 1e-3), ([0., 1, -23], 1.0)):
        z = np.array(z)
        p = serving.distribution(z, t)
        for u in (0.0, 0.2, 0.9):
            a, tok, lp = serving.draft_verify(np.tile(z, (1, 2, 1)), np.array([[2]]), np.array([[1.0, u]]), z[None, None] + 3,
                                              None, [t])
            want = 2 if p[2] else int(u >= p[0])  # (as long as the draft has a chance, it stands)
            assert a[0] == (p[2] > 0) and tok[0, 0] == want and abs(lp[0, 0] - np.log(p[want])) < 1e-12


def test_greedy_verification_follows_the_largest_logit():
    z = np.array([[[1., 3, 3, 0], [0, 0, 5, 0], [2, 1, 0, 0]]])
    a, t, _ = serving.draft_verify(z, np.array([[1, 3]]), np.ones((1, 3)), None, None, [0.0])
    assert a[0] == 1 and list(t[0]) == [1, 2, -1]
    a, t, _ = serving.draft_verify(z, np.array([[1, 2]]), np.ones((1, 3)), None, None, [-1.0])
    assert a[0] == 2 and list(t[0]) == [1, 2, 0]
    a, t, _ = serving.draft_verify(z, np.array([[2, 2]]), np.ones((1, 3)), None, [0], [np.nan])
    assert a[0] == 0 and list(t[0]) == [1, -1, -1]


def test_rows_without_a_distribution_draw_nothing():
    z = np.zeros((3, 2, 4))
    z[0, 0, 2], z[1, 0, 1], z[2, 0] = np.nan, np.inf, -np.inf
    a, t, lp = serving.draft_verify(z, np.zeros((3, 1), int), np.zeros((3, 2)), None, None, None)
    assert not a.any() and (t == -1).all() and not lp.any()


def test_commit_is_the_serial_recurrence():
    g = rng(4)
    k, v, h = g.standard_normal((1, 2, 1, 2)), g.standard_normal((1, 2, 1, 3)), g.standard_normal((1, 1, 2, 3))
    gg, b, A = np.array([[[0.3], [0.8]]]), np.array([[[0.5], [0.2]]]), np.array([0.1])
    want = h[0, 0]
    np.testing.assert_array_equal(serving.step_commit(k, v, gg, b, A, [0], h)[0, 0], want)
    for t in range(2):
        a = np.exp(-gg[0, t, 0] * np.exp(0.1))
        want = a * (np.eye(2) - b[0, t, 0] * np.outer(k[0, t, 0], k[0, t, 0])) @ want + b[0, t, 0] * np.outer(
            k[0, t, 0], v[0, t, 0])
        np.testing.assert_allclose(serving.step_commit(k, v, gg, b, A, [t + 1], h)[0, 0], want, atol=1e-14)
