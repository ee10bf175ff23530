"""Shared prefixes, cached rows' weights, eviction, page return, draft
verification and the state after accepted tokens against their fp64 definitions,
at sizes and masks where they can go wrong, and a serving loop of them
together. The bounds are the worst-case rounding sums of serving_util."""
import numpy as np
import pytest
import torch

import gated_delta_rule_74_amd as gdn
import serving_util as bound
from gpu_util import say
from latent_util import TYPES, U, dev, host, ints, rng, within
from oracle import latent
from oracle import serving as ref

pytestmark = pytest.mark.gpu


def tables(g, lens, page, extra=0, order=None):
    """Block tables of sequences, the pool's size, and its pages not in use."""
    need = [-(-max(n, 0) // page) for n in lens]
    order = g.permutation(sum(need) + 2 + extra) if order is None else order
    t, at = np.full((len(lens), max(max(need, default=0), 1)), -1, np.int32), 0
    for n, k in enumerate(need):
        t[n, :k] = order[at:at + k]
        at += k
    return t, order, order[at:]


def pool(g, dtype, pages, page, d, used):
    """Cache rows; those not in `used` [(table, lens)] are NaN, as uninitialised memory may be."""
    c = g.standard_normal((pages, page, d))
    keep = np.zeros((pages, page), bool)
    for t, lens in used:
        for n, m in enumerate(lens):
            for j in range(m):
                if 0 <= t[n, j // page] < pages:
                    keep[t[n, j // page], j % page] = True
    t, f = dev(c, dtype)
    t[torch.from_numpy(~keep).cuda()] = float("nan")
    f[~keep] = 0.0
    return t, f


# ---------------------------------------------------------------- shared prefixes

# N, S, H, dl, dr, page, own lengths, prefix lengths, starts
SHARED = [
    (1, 1, 1, 16, 0, 1, [1], [1], [0, 1]),
    (3, 1, 4, 32, 8, 4, [5, 1, 0], [0], [0, 3]),
    (3, 1, 4, 32, 8, 4, [5, 1, 0], [3], [0, 3]),
    (4, 2, 3, 48, 16, 16, [1, 2, 17, 0], [65, 64], [1, 2, 4]),
    (5, 3, 8, 128, 32, 24, [40, 3, 1, 2, 100], [300, 0, 129], [0, 2, 2, 4]),
    (5, 1, 16, 128, 64, 64, [1, 3, 64, 65, 30], [1025], [0, 5]),
    (7, 2, 16, 64, 0, 16, [2, 9, 2, 30, 4, 5, 6], [257, 31], [0, 6, 7]),
    (4, 1, 24, 192, 24, 16, [7, 1, 33, 2], [400], [0, 3]),
    (3, 2, 16, 256, 64, 64, [2, 70, 5], [333, 64], [0, 1, 3]),
    (4, 3, 8, 320, 32, 16, [3, 20, 4, 5], [97], [0, 4]),
    (3, 4, 16, 512, 64, 64, [4, 130, 5], [500], [0, 3]),
    (2, 1, 2, 512, 32, 16, [9, 1], [40, 33], [0, 1, 2]),
    (3, 1, 4, 256, 0, 128, [3, 2, 1], [200], [-1, 99]),       # starts past the batch
    (4, 1, 4, 64, 8, 16, [3, 2, 1, 4], [50, 60, 70], [0, 3, 1, 4]),  # starts that go back
]


def shared_inputs(case, dtype, seed):
    N, S, H, dl, dr, page, lens, plens, starts = case
    g, d = rng(seed), dl + dr
    t, order, rest = tables(g, lens, page, sum(-(-x // page) for x in plens))
    pt, _, _ = tables(g, plens, page, order=rest)
    q, qf = dev(g.standard_normal((N, S, H, d)), dtype)
    cache, cf = pool(g, dtype, len(order), page, d, [(t, lens), (pt, plens)])
    return (q, cache, ints(t), ints(lens), dl, ints(pt), ints(plens), ints(starts)), (qf, cf, t, lens, dl, pt, plens, starts)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(map(str, c[:6])) + f"-{len(c[7])}")
def test_shared_prefixes(case, dtype):
    say(f"shared {case} {dtype}")
    a, f = shared_inputs(case, dtype, 9100)
    scale = (case[3] + case[4]) ** -0.5
    o, lse = gdn.mla_step_shared(*a, scale=scale)
    want, to, wl, tl = bound.shared(*f, scale, dtype)
    within("o", o, want, to)
    within("lse", lse, wl, tl)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,dl", [(16, 128), (128, 64), (8, 512)])
def test_shared_prefix_of_many_queries(dtype, H, dl):
    """Enough blocks of queries that shares begin and end inside walks; sequences of no group before and after."""
    N, S, dr, page = 20, 2, 32, 16
    g = rng(9200)
    case = (N, S, H, dl, dr, page, [2 + int(x) for x in g.integers(0, 40, N)], [700, 1, 333], [2, 3, 11, 19])
    say(f"shared, many queries {H} {dl} {dtype}")
    a, f = shared_inputs(case, dtype, 9201)
    o, lse = gdn.mla_step_shared(*a, scale=0.1)
    pick = [0, 2, 3, 10, 11, 18, 19]
    starts = [max(0, sum(p < s for p in pick)) for s in case[8]]
    sub = (f[0][pick], f[1], f[2][pick], [case[6][n] for n in pick], dl, f[5], f[6], starts)
    want, to, wl, tl = bound.shared(*sub, 0.1, dtype)
    within("o", o[pick], want, to)
    within("lse", lse[pick], wl, tl)


@pytest.mark.parametrize("dl,dr", [(64, 32), (48, 48), (112, 16), (128, 64), (192, 32), (176, 56), (256, 64), (384, 32)])
def test_shared_prefix_of_full_blocks(dl, dr):
    """Every width's kernel for groups that fill blocks of queries, the last one in part; an odd page."""
    case = (20, 1, 32, dl, dr, 24, [1 + 7 * n for n in range(20)], [450, 131], [0, 11, 20])
    say(f"shared, full blocks {dl} {dr}")
    a, f = shared_inputs(case, "bf16", 9240)
    o, lse = gdn.mla_step_shared(*a, scale=0.1)
    pick = [0, 10, 11, 19]
    want, to, wl, tl = bound.shared(f[0][pick], f[1], f[2][pick], [case[6][n] for n in pick], dl, f[5], f[6], [0, 2, 4],
                                    0.1, "bf16")
    within("o", o[pick], want, to)
    within("lse", lse[pick], wl, tl)


@pytest.mark.parametrize("dtype,dl", [("bf16", 128), ("bf16", 512), ("fp32", 64), ("fp32", 320)])
def test_own_rows_of_many_queries(dtype, dl):
    """More queries in a sequence than a block holds: its own rows are walked once for each block, the last one's mask
    inside the later blocks."""
    case = (3, 9, 16, dl, 16, 16, [9, 200, 70], [300], [0, 2])
    say(f"shared, own blocks {dtype} {dl}")
    a, f = shared_inputs(case, dtype, 9210)
    o, lse = gdn.mla_step_shared(*a, scale=0.1)
    want, to, wl, tl = bound.shared(*f, 0.1, dtype)
    within("o", o, want, to)
    within("lse", lse, wl, tl)


@pytest.mark.parametrize("H", [1, 4, 16])
def test_own_rows_apart_in_fp32(H):
    """Too many own rows for one launch to take both, with queries that leave waves idle, and a prefix of its own."""
    N = 40
    case = (N, 1, H, 64, 0, 16, [1 + 23 * n for n in range(N)], [90, 200], [0, 20, N])
    say(f"shared, own rows apart {H}")
    a, f = shared_inputs(case, "fp32", 9220)
    o, lse = gdn.mla_step_shared(*a, scale=0.1)
    pick = [0, 1, 19, 20, 38, 39]
    want, to, wl, tl = bound.shared(f[0][pick], f[1], f[2][pick], [case[6][n] for n in pick], 64, f[5], f[6], [0, 3, 6],
                                    0.1, "fp32")
    within("o", o[pick], want, to)
    within("lse", lse[pick], wl, tl)


@pytest.mark.parametrize("dtype,H,dl,N,G", [("bf16", 4, 64, 150, 70), ("fp32", 1, 64, 150, 70), ("fp32", 16, 32, 150, 70),
                                            ("bf16", 16, 256, 150, 100), ("bf16", 1, 16, 4500, 300), ("fp32", 2, 16, 4500, 300)])
def test_shared_prefixes_of_many_groups(dtype, H, dl, N, G):
    """More groups and sequences than a wave has lanes; groups of none and of one among them, prefixes of nothing."""
    say(f"shared, many groups {dtype} {H} {dl} {N} {G}")
    g = rng(9250)
    starts = np.sort(g.integers(1, N - 1, G + 1))
    plens = [int(x) for x in g.integers(0, 150, G)]
    plens[::7] = [0] * len(plens[::7])
    lens = [int(x) for x in g.integers(0, 60, N)]
    case = (N, 2, H, dl, 16, 8, lens, plens, [int(x) for x in starts])
    a, f = shared_inputs(case, dtype, 9251)
    o, lse = gdn.mla_step_shared(*a, scale=0.1)
    pick = sorted({0, 1, int(starts[0]), int(starts[0]) - 1, N // 2, N // 3, int(starts[-1]) - 1, int(starts[-1]), N - 1})
    want, to, wl, tl = bound.shared(f[0][pick], f[1], f[2][pick], [lens[n] for n in pick], dl, f[5], f[6],
                                    [sum(p < s for p in pick) for s in case[8]], 0.1, dtype)
    within("o", o[pick], want, to)
    within("lse", lse[pick], wl, tl)


def test_caches_past_32_bits():
    """Pages whose elements lie past 2^32 of the cache: the same results, bit for bit, as from a small cache."""
    page, dl, dr, N = 64, 512, 64, 3
    d, far = dl + dr, 2 ** 32 // (64 * 576) + 40
    case = (N, 2, 16, dl, dr, page, [130, 2, 64], [200], [0, 2])
    a, _ = shared_inputs(case, "bf16", 9230)
    small = a[1]
    pages = small.shape[0]
    big = torch.empty((far, page, d), dtype=torch.bfloat16, device="cuda")
    move = torch.cat([torch.arange(pages // 2), far - pages + torch.arange(pages // 2, pages)]).int().cuda()
    big[move.long()] = small
    there = lambda t: torch.where(t >= 0, move[t.clamp(min=0).long()], t).contiguous()  # noqa: E731
    assert big.numel() > 2 ** 32 and int(there(a[2]).max()) * page * d > 2 ** 32
    o, lse = gdn.mla_step_shared(*a, scale=0.05)
    bo, bl = gdn.mla_step_shared(a[0], big, there(a[2]), a[3], dl, there(a[5]), *a[6:], scale=0.05)
    assert torch.equal(o, bo) and torch.equal(lse, bl)
    ws, wb = torch.zeros((pages, page), device="cuda"), torch.zeros((far, page), device="cuda")
    own_o, own_lse = gdn.mla_step(a[0], small, a[2], a[3], dl, scale=0.05)
    gdn.mla_weights(a[0], small, a[2], a[3], own_lse, ws, scale=0.05)
    gdn.mla_weights(a[0], big, there(a[2]), a[3], own_lse, wb, scale=0.05)
    assert float(ws.sum()) > 0 and torch.equal(wb[move.long()], ws)
    keep = ints([70, 1, 20])
    out = gdn.mla_evict(ws, small, a[2], a[3], keep, first=2, recent=3)
    far_out = gdn.mla_evict(wb, big, there(a[2]), a[3], keep, first=2, recent=3)
    assert torch.equal(out, far_out) and torch.equal(wb[move.long()], ws)
    assert torch.equal(big[move.long()].view(torch.int16), small.view(torch.int16))


def test_shared_prefix_masks():
    """Table entries outside the pool mask their rows, of prefixes too; a prefix that leaves nothing; no groups."""
    case = (3, 1, 4, 32, 8, 4, [5, 2, 1], [9, 8], [0, 2, 3])
    a, f = shared_inputs(case, "fp32", 9300)
    a, f = list(a), list(f)
    f[5] = f[5].copy()
    f[5][0, 1], f[5][1, :] = 10 ** 6, -1
    f[2] = f[2].copy()
    f[2][2, 0] = -7
    a[2], a[5] = ints(f[2]), ints(f[5])
    o, lse = gdn.mla_step_shared(*a, scale=0.2)
    want, to, wl, tl = bound.shared(*f, 0.2, "fp32")
    assert wl[2, 0, 0] == -np.inf  # (nothing left for the last sequence)
    within("o", o, want, to)
    within("lse", lse, wl, tl)
    # negative and overlong lengths are clamped
    a[6], f[6] = ints([-4, 1000]), [-4, 1000]
    o, lse = gdn.mla_step_shared(*a, scale=0.2)
    want, to, wl, tl = bound.shared(*f, 0.2, "fp32")
    within("o", o, want, to)
    within("lse", lse, wl, tl)
    # no group at all: the plain step, bit for bit
    none = (ints(np.zeros((0, 3))), ints([]), ints([0]))
    o, lse = gdn.mla_step_shared(*a[:5], *none, scale=0.2)
    po, pl = gdn.mla_step(*a[:5], scale=0.2)
    assert torch.equal(o, po) and torch.equal(lse, pl)


def test_shared_agrees_with_a_longer_table():
    """A prefix of whole pages as the front of every table: the same as the plain step, within both bounds; bits repeat."""
    case = (6, 2, 8, 64, 32, 16, [2, 40, 3, 100, 7, 2], [160], [0, 6])
    a, f = shared_inputs(case, "fp32", 9400)
    o, lse = gdn.mla_step_shared(*a, scale=0.1)
    long = torch.cat([a[5].expand(6, -1), a[2]], 1).contiguous()
    po, pl = gdn.mla_step(a[0], a[1], long, a[3] + 160, 64, scale=0.1)
    want, to, wl, tl = bound.shared(*f, 0.1, "fp32")
    within("o", o, host(po), 2 * to)
    within("lse", lse, host(pl), 2 * tl)
    for _ in range(3):
        o2, l2 = gdn.mla_step_shared(*a, scale=0.1)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    single = gdn.mla_step_shared(a[0][:, 1].contiguous(), *a[1:], scale=0.1)  # [N, H, d]: one token each
    assert single[0].shape == (6, 8, 64)


def test_sharp_scores_and_large_values():
    """A prefix whose scores leave the running maximum far behind again and again."""
    case = (4, 1, 4, 32, 0, 16, [3, 1, 9, 2], [300], [0, 4])
    a, f = shared_inputs(case, "fp32", 9500)
    o, lse = gdn.mla_step_shared(*a, scale=40.0)
    want, to, wl, tl = bound.shared(*f, 40.0, "fp32")
    within("o", o, want, to)
    within("lse", lse, wl, tl)


def test_nan_in_a_prefix_reaches_its_group_alone():
    case = (4, 1, 4, 32, 0, 16, [3, 1, 9, 2], [100, 70], [0, 2, 4])
    a, f = shared_inputs(case, "bf16", 9600)
    o, _ = gdn.mla_step_shared(*a, scale=0.2)
    a[1][f[5][0, 2], 3, 5] = float("nan")
    o2, _ = gdn.mla_step_shared(*a, scale=0.2)
    assert o2[:2].isnan().any() and torch.equal(o2[2:], o[2:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dl", [64, 128, 512])
def test_nan_in_an_own_row_reaches_its_sequence_alone(dl, dtype):
    """The last draft's row: the sequence's other tokens do not see it, but share its tile (as in mla_step). Their lse,
    and all of other sequences, stay as they were."""
    case = (4, 3, 4, dl, 16, 16, [3, 20, 9, 70], [100, 70], [0, 2, 4])
    a, f = shared_inputs(case, dtype, 9610)
    o, lse = gdn.mla_step_shared(*a, scale=0.2)
    for bad in (float("nan"), float("inf")):
        row = a[1][f[2][1, 19 // 16], 19 % 16]
        was = row.clone()
        row[5] = bad
        o2, lse2 = gdn.mla_step_shared(*a, scale=0.2)
        others = [0, 2, 3]
        assert torch.equal(o2[others], o[others]) and torch.equal(lse2[others], lse[others])
        assert torch.equal(lse2[1, :2], lse[1, :2]) and o2[1, 2].isnan().any()
        row.copy_(was)


# ---------------------------------------------------------------- weights of cached rows

WEIGHTS = [
    (1, 1, 1, 16, 1, [1], None, 1.0),
    (3, 1, 4, 40, 4, [5, 0, 1], None, 0.5),
    (3, 3, 2, 64, 16, [2, 17, 100], None, 0.95),
    (2, 8, 16, 160, 64, [700, 30], [0, 0], 1.0),
    (2, 2, 24, 576, 24, [600, 1], [300, 7], 0.0),
    (2, 32, 8, 320, 16, [40, 513], [100, 5], 1.0),
    (1, 5, 7, 88, 3, [64], [-5], 0.25),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "-".join(map(str, c[:5])))
def test_weights(case, dtype):
    say(f"weights {case} {dtype}")
    N, S, H, d, page, lens, known, decay = case
    decay = float(np.float32(decay))
    g, scale = rng(9700), d ** -0.5
    t, order, _ = tables(g, lens, page)
    q, qf = dev(g.standard_normal((N, S, H, d)), dtype)
    cache, cf = pool(g, dtype, len(order), page, d, [(t, lens)])
    old, oldf = dev(g.random((len(order), page)), "fp32")
    _, lsef = latent.step(qf, cf, t, lens, d, scale)
    lse, lsef = dev(lsef, "fp32")
    before = old.clone()
    got = gdn.mla_weights(q, cache, ints(t), ints(lens), lse, old, None if known is None else ints(known), scale=scale,
                          decay=decay)
    assert got is old
    want, tol = bound.weights(qf, cf, t, lens, lsef, oldf, known, scale, decay)
    within("weights", got, want, tol)
    held = np.zeros(got.shape, bool)
    for n, m in enumerate(lens):
        for j in range(m):
            held[t[n, j // page], j % page] = True
    assert torch.equal(got[torch.from_numpy(~held).cuda()], before[torch.from_numpy(~held).cuda()])
    again = gdn.mla_weights(q, cache, ints(t), ints(lens), lse, before, None if known is None else ints(known),
                            scale=scale, decay=decay)
    assert torch.equal(got, again)


def test_weights_of_the_unusual():
    """Entries outside the pool, stale NaN weights of new rows, tokens that saw nothing, one token each as [N, H, d]."""
    g, page, d = rng(9800), 4, 32
    lens = [9, 3, 1]
    t, order, _ = tables(g, lens, page)
    q, qf = dev(g.standard_normal((3, 4, d)), "fp32")
    cache, cf = pool(g, "fp32", len(order), page, d, [(t, lens)])
    t[0, 1], t[2, 0] = -1, len(order)
    _, lsef = latent.step(qf[:, None], cf, t, lens, d, 0.2)
    lse, lsef = dev(lsef, "fp32")
    assert torch.isinf(lse[2]).all()
    old = torch.full((len(order), page), 2.0, device="cuda")
    old[t[0, 2], 0] = float("nan")  # (the new token's row)
    oldf = host(old)
    got = gdn.mla_weights(q, cache, ints(t), ints(lens), lse[:, 0].contiguous(), old, scale=0.2)
    want, tol = bound.weights(qf[:, None], cf, t, lens, lsef, np.nan_to_num(oldf), None, 0.2, 1.0)
    within("weights", got, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d", [(100, 40), (150, 88), (256, 160)])
def test_weights_of_many_sequences(N, d, dtype):
    """Waves that walk 32, 64 and 128 rows, the next sixteen requested while these are used; picked sequences."""
    say(f"weights, many sequences {N} {d} {dtype}")
    g, page, scale = rng(9710), 64, d ** -0.5
    S, H, lens = 2, 3, [int(x) for x in g.integers(0, 2113, N)]
    lens[:9] = [2112, 0, 1, 2, 511, 512, 513, 16, 1056]
    t, order, _ = tables(g, lens, page)
    q, qf = dev(g.standard_normal((N, S, H, d)), dtype)
    cache, cf = pool(g, dtype, len(order), page, d, [(t, lens)])
    pick = [0, 1, 2, 3, 4, 5, 6, 7, 8, N - 2, N - 1]
    sub = (qf[pick], cf, t[pick], [lens[n] for n in pick])
    some = latent.step(*sub, d, scale)[1]
    lse = np.zeros((N, S, H))
    lse[pick] = some
    lse, lsef = dev(lse, "fp32")
    old, oldf = dev(g.random((len(order), page)), "fp32")
    known = [max(0, n - 40) for n in lens]
    before = old.clone()
    gdn.mla_weights(q, cache, ints(t), ints(lens), lse, old, ints(known), scale=scale, decay=0.5)
    want, tol = bound.weights(*sub, lsef[pick], oldf, [known[n] for n in pick], scale, 0.5)
    at = np.zeros(want.shape, bool)
    held = np.zeros(want.shape, bool)
    for n, m in enumerate(lens):
        j = np.arange(m)
        held[t[n, j // page], j % page] = True
        if n in pick:
            at[t[n, j // page], j % page] = True
    assert at.sum() == sum(lens[n] for n in pick)
    rows = torch.from_numpy(at).cuda()
    within("weights", old[rows], want[at], tol[at])
    rows = torch.from_numpy(~held).cuda()
    assert torch.equal(old[rows], before[rows])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [24, 64, 88, 128, 152, 184, 224, 248, 320, 360, 448, 488, 512, 576])
def test_weights_of_every_width(d, many, dtype):
    """Every number of column steps, with queries that stay in LDS and with more of them."""
    say(f"weights, width {d} {many} {dtype}")
    g, page, lens = rng(9720), 16, [37]
    S, H = (33, 24) if many else (2, 5)
    t, order, _ = tables(g, lens, page)
    scale = d ** -0.5
    q, qf = dev(g.standard_normal((1, S, H, d)), dtype)
    cache, cf = pool(g, dtype, len(order), page, d, [(t, lens)])
    lse, lsef = dev(latent.step(qf, cf, t, lens, d, scale)[1], "fp32")
    old, oldf = dev(g.random((len(order), page)), "fp32")
    gdn.mla_weights(q, cache, ints(t), ints(lens), lse, old, ints([20]), scale=scale, decay=0.5)
    want, tol = bound.weights(qf, cf, t, lens, lsef, oldf, [20], scale, 0.5)
    within("weights", old, want, tol)


# ---------------------------------------------------------------- eviction

EVICT = [
    # d, page, lens, keep, first, recent
    (8, 1, [1, 0, 5], [0, 0, 3], 0, 0),
    (16, 3, [10, 7, 1], [4, 7, 1], 1, 2),
    (40, 16, [100, 257, 256, 0], [50, 200, 0, 3], 4, 8),
    (160, 64, [700, 64, 513, 300], [333, 10, 512, -3], 4, 64),
    (576, 64, [1000, 3], [400, 2], 0, 300),
    (72, 24, [3000, 2999, 1024], [1500, 2998, 1], 16, 0),
]


def evict_inputs(case, dtype, seed, ties):
    d, page, lens, keep, first, recent = case
    g = rng(seed)
    t, order, _ = tables(g, lens, page)
    cache, cf = pool(g, dtype, len(order), page, d, [(t, lens)])
    w = g.standard_normal((len(order), page))
    if ties:
        w = np.round(w)  # (with zeros of both signs)
        w[g.random(w.shape) < 0.05] = np.nan
        w[g.random(w.shape) < 0.05] = np.inf
        w[g.random(w.shape) < 0.05] = -np.inf
    w, wf = dev(w, "fp32")
    return (w, cache, ints(t), ints(lens), ints(keep)), (wf, cf, t, lens, keep)


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{c[0]}-{c[1]}-{len(c[2])}")
def test_eviction(case, dtype, ties):
    say(f"evict {case} {dtype} {ties}")
    a, f = evict_inputs(case, dtype, 9900, ties)
    w0, c0 = a[0].clone(), a[1].clone()
    out = gdn.mla_evict(*a, first=case[4], recent=case[5])
    # the definition on row numbers: what stands in each slot afterwards
    number = np.arange(c0.shape[0] * c0.shape[1], dtype=np.float64).reshape(c0.shape[:2] + (1,))
    _, at, lens = ref.evict(f[0], number, f[2], case[2], case[3], case[4], case[5])
    at = torch.from_numpy(at[..., 0].astype(np.int64).ravel()).cuda()
    assert (host(out) == lens).all()
    assert torch.equal(bits(a[1]).flatten(0, 1), bits(c0).flatten(0, 1)[at])
    assert torch.equal(bits(a[0]).flatten(), bits(w0).flatten()[at])


def test_eviction_of_a_long_sequence():
    """Hundreds of segments, each waiting for those its rows move into; the same bits every time."""
    n, page, d = 70000, 64, 64
    say("evict, long")
    g = torch.Generator("cuda").manual_seed(5)
    pages = -(-n // page) + 3
    t = torch.randperm(pages, generator=g, device="cuda")[:-3].to(torch.int32)[None].contiguous()
    c0 = torch.randint(-2 ** 31, 2 ** 31 - 1, (pages, page, d), generator=g, device="cuda", dtype=torch.int32).view(torch.float32)
    w0 = torch.rand((pages, page), generator=g, device="cuda")
    w0[torch.rand((pages, page), generator=g, device="cuda") < 0.3] = 0.25  # (many equal ones, the bar among them)
    for keep in (69999, 35000, 52000, 1, 0):
        c, w = c0.clone(), w0.clone()
        out = gdn.mla_evict(w, c, t, ints([n]), ints([keep]), first=3, recent=100)
        slots = (t[0].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
        a = min(3, keep)
        b = min(100, keep - a)
        key = w0.flatten()[slots].cpu().numpy()
        best = np.lexsort((np.arange(a, n - b), -key[a:n - b]))[:keep - a - b] + a
        stay = torch.from_numpy(np.concatenate([np.arange(a), np.sort(best), np.arange(n - b, n)])).cuda()
        wc, ww = c0.flatten(0, 1).clone(), w0.flatten().clone()
        wc[slots[:keep]], ww[slots[:keep]] = wc[slots[stay]], ww[slots[stay]]
        assert int(out) == keep
        assert torch.equal(bits(c).flatten(0, 1), bits(wc)) and torch.equal(w.flatten(), ww)


def test_eviction_with_entries_outside_the_pool():
    case = (16, 4, [30, 11], [9, 4], 2, 3)
    a, f = evict_inputs(case, "fp32", 9950, False)
    t = f[2].copy()
    t[0, 1], t[0, 4], t[1, 0] = -1, 10 ** 7, -5
    w0, c0 = a[0].clone(), a[1].clone()
    gdn.mla_evict(a[0], a[1], ints(t), a[3], a[4], first=2, recent=3)
    number = np.arange(c0.shape[0] * c0.shape[1], dtype=np.float64).reshape(c0.shape[:2] + (1,))
    _, at, _ = ref.evict(f[0], number, t, case[2], case[3], 2, 3)
    at = torch.from_numpy(at[..., 0].astype(np.int64).ravel()).cuda()
    assert torch.equal(bits(a[1]).flatten(0, 1), bits(c0).flatten(0, 1)[at])
    assert torch.equal(bits(a[0]).flatten(), bits(w0).flatten()[at])


# table rows of more than 8192 rows, and of more than one workgroup of the choice takes
EVICT_WIDE = [
    (8, 64, [20000, 0, 9000, 3], [12345, 0, 8999, 2], 4, 300),
    (40, 24, [32760, 8193], [1, 4000], 0, 0),
    (8, 64, [40000, 5000, 0, 33001, 8192], [30000, 1200, 0, 17, 8191], 4, 64),
    (16, 16, [33000, 16385, 40016], [32999, 16384, 3], 0, 2),
]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("case", EVICT_WIDE, ids=lambda c: f"{c[0]}-{c[1]}-{max(c[2])}")
def test_eviction_of_several_long_sequences(case, ties):
    test_eviction(case, "bf16", ties)


def test_eviction_of_thousands_of_sequences():
    """More sequences than a wave has lanes, many times over: which of them a workgroup works on is found in two steps."""
    g, N = rng(9962), 4500
    lens = [int(x) for x in g.integers(0, 9, N)]
    keep = [int(x) for x in g.integers(-1, 10, N)]
    test_eviction((8, 4, lens, keep, 1, 1), "bf16", True)


# ---------------------------------------------------------------- pages given back

@pytest.mark.parametrize("N,page,most,room", [(1, 1, 3, 9), (3, 16, 100, 50), (1025, 16, 200, 0), (2500, 3, 40, 10 ** 5),
                                              (4, 64, 60000, 7)])
def test_page_trim(N, page, most, room):
    say(f"trim {N} {page} {most}")
    g = rng(9960)
    lens, new = g.integers(-2, most + 3, N), g.integers(-5, most + 5, N)
    cols = -(-most // page)
    t = g.integers(0, 10 ** 6, (N, cols)).astype(np.int32)
    n_free = 5
    stack = np.full(n_free + room + 1, -1, np.int32)
    stack[:n_free] = np.arange(n_free) + 7
    want, top = ref.page_trim(lens, new, t, stack, n_free, page)
    s, f = ints(stack), ints([n_free])
    out = gdn.page_trim(ints(lens), ints(new), ints(t), s, f, page)
    assert int(out) == top and int(f) == n_free and (s.cpu().numpy() == want).all()
    s = ints(stack)
    assert gdn.page_trim(ints(lens), ints(new), ints(t), s, f, page, n_free_out=f) is f
    assert int(f) == top and (s.cpu().numpy() == want).all()


@pytest.mark.parametrize("N,page,most,room", [(1, 1, 3, 9), (3, 16, 100, 50), (1025, 16, 200, 10 ** 5), (2500, 3, 40, 7000),
                                              (4, 64, 60000, 3500), (300, 16, 700, 10 ** 5)])
@pytest.mark.parametrize("share", [0.001, 0.3, 1.0])
def test_page_trim_leaves_out_entries_that_are_no_page(N, page, most, room, share):
    """Entries below 0, which page_plan would hand out again: the others are pushed in their order."""
    say(f"trim, no pages {N} {page} {most} {share}")
    g = rng(9961)
    lens, new, cols = g.integers(-2, most + 3, N), g.integers(-5, most // 2, N), -(-most // page)
    t = g.integers(0, 10 ** 6, (N, cols)).astype(np.int32)
    none = g.random(t.shape) < share
    t[none] = g.choice([-1, -5, -2 ** 31], none.sum())
    stack = np.full(5 + room + 1, -9, np.int32)
    stack[:5] = np.arange(5) + 7
    want, top = ref.page_trim(lens, new, t, stack, 5, page)
    assert (want[:top] >= 0).all()
    s = ints(stack)
    out = gdn.page_trim(ints(lens), ints(new), ints(t), s, ints([5]), page)
    assert int(out) == top and (s.cpu().numpy() == want).all()


# ---------------------------------------------------------------- draft verification

def drafts(N, S, V, dtype, seed, with_q, ragged, heat, close=0.7):
    g = rng(seed)
    z = 2.0 * g.standard_normal((N, S + 1, V))
    z[g.random(z.shape) < 0.1] = -np.inf
    z[..., g.integers(0, V, 1)] = 1.0
    zq = z[:, :S] + close * np.where(np.isfinite(z[:, :S]), g.standard_normal((N, S, V)), 0)
    z, zf = dev(z, dtype)
    zq, zqf = dev(zq, dtype)
    temp = None if heat is None else np.float32(g.choice(heat, N))
    draft = np.zeros((N, S), np.int32)
    for n in range(N):
        for i in range(S):
            t = 1.0 if temp is None or not temp[n] > 0 else float(temp[n])
            draft[n, i] = zf[n, i].argmax() if temp is not None and not temp[n] > 0 and g.random() < 0.6 else (
                g.choice(V, p=ref.distribution(zqf[n, i], t)))
    u = g.random((N, S + 1)).astype(np.float32)
    lens = g.integers(-1, S + 2, N) if ragged else None
    return dict(logits=z, draft=draft, uniforms=u, draft_logits=zq if with_q else None, draft_lens=lens,
                temperature=temp), (zf, draft, u, zqf if with_q else None, lens, temp)


def check_verify(a, f):
    put = dict(a, draft=ints(a["draft"]), uniforms=torch.from_numpy(a["uniforms"]).cuda(),
               draft_lens=None if a["draft_lens"] is None else ints(a["draft_lens"]),
               temperature=None if a["temperature"] is None else torch.from_numpy(a["temperature"]).cuda())
    acc, tok, lp = gdn.draft_verify(**put)
    wa, wt, wl = ref.draft_verify(*f)
    assert (host(acc) == wa).all(), (acc, wa)
    assert (host(tok) == wt).all(), np.argwhere(host(tok) != wt)
    within("logprobs", lp, wl, U * np.abs(wl) + 1e-10)  # one rounding of what fp64 holds to 2^-40
    again = gdn.draft_verify(**put, want_logprobs=False)
    assert again[2] is None and torch.equal(again[0], acc) and torch.equal(again[1], tok)
    return wa


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,S,V", [(1, 0, 1), (2, 1, 2), (5, 2, 7), (9, 3, 8), (7, 8, 63), (40, 4, 1000), (6, 2, 8191),
                                   (6, 1, 8193), (5, 5, 20001), (3, 2, 65792), (2, 1, 131072)])
def test_draft_verify(N, S, V, dtype):
    say(f"verify {N} {S} {V} {dtype}")
    for k, (with_q, ragged, heat) in enumerate([(True, False, None), (False, True, [0.7, 0.0, 1.3]),
                                                (True, True, [0.0, 1.0, 0.5, 2.0, -1.0])]):
        check_verify(*drafts(N, S, V, dtype, 9970 + k, with_q, ragged, heat))


def test_verify_many_sequences():
    """A batch large enough that every branch is taken many times."""
    say("verify, many")
    wa = check_verify(*drafts(600, 3, 300, "fp32", 9980, True, True, [0.0, 0.8, 1.0]))
    assert set(wa) == {0, 1, 2, 3}


@pytest.mark.parametrize("heat", [1e-3, 1e-30, 1e30, float("inf"), float("nan")])
def test_verify_extreme_temperatures(heat):
    say(f"verify at {heat}")
    check_verify(*drafts(12, 2, 500, "fp32", 9985, True, False, [heat]))


def test_verify_unusual_numbers():
    """Uniforms at and past their ends, drafts outside the vocabulary, rows without a distribution, equal distributions."""
    a, f = drafts(24, 2, 77, "fp32", 9990, True, False, [0.0, 1.0])
    z, draft, u, zq, lens, temp = f
    for n, x in enumerate([0.0, 1.0, 1 - 2.0 ** -24, np.nan, -3.0, 7.0, 1e-40]):
        u[n] = x
    draft[7, 0], draft[8, 1], draft[9, 0], draft[10, 0] = -1, 77, 2 ** 31 - 1, -2 ** 31
    for n, (i, v) in enumerate([(0, np.nan), (1, np.inf), (2, np.nan)]):
        z[11 + n, i, 5] = v
    z[14, 0], z[15, 1] = -np.inf, -np.inf
    zq[16, 0, 3], zq[17, 1, 4], zq[18, 0] = np.nan, np.inf, -np.inf
    zq[19:22] = z[19:22, :2]  # p = q: every draft is accepted
    u[19:22] = 1.0
    temp[16:22] = 1.0
    a["logits"], a["draft_logits"] = dev(z, "fp32")[0], dev(zq, "fp32")[0]
    wa = check_verify(a, f)
    assert (wa[19:22] == 2).all() and wa[7] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [9, 5000])
def test_verify_where_a_rejected_draft_leaves_nothing(V, dtype):
    """Drafts that neither model gives any probability, masked or far below at a low temperature, before equal
    distributions: rejected, and the token is drawn from p. Equal with the same logits, with others a constant apart
    (1, which both types hold beside multiples of 1/16 below 8), and as one token alone."""
    say(f"verify, nothing left {V} {dtype}")
    g, N = rng(9991), 24
    z = np.round(16 * g.standard_normal((N, 2, V)).clip(-4, 4)) / 16
    z[:, :, 5] = -np.inf
    draft, temp = np.full((N, 1), 5, np.int32), np.ones(N, np.float32)
    zq = z[:, :1] + np.where(np.arange(N) % 2, 1.0, 0.0)[:, None, None]
    z[12:, :, 5], zq[12:, :, 5] = -4, -4  # p = q = 0 only as numbers: e^-4000 and less
    z[12:, :, 3] += 8
    zq[12:, :, 3] += 8 + np.where(np.arange(12, N) % 2, 1 / 16, 0)[:, None]
    temp[12:] = 1e-3
    u = g.random((N, 2)).astype(np.float32)
    u[::5, 1], u[1::5, 1] = 0.0, 1.0
    a = dict(logits=dev(z, dtype)[0], draft=draft, uniforms=u, draft_logits=dev(zq, dtype)[0], draft_lens=None, temperature=temp)
    wa = check_verify(a, (dev(z, dtype)[1], draft, u, dev(zq, dtype)[1], None, temp))
    assert not wa.any()


@pytest.mark.parametrize("V", [2 ** 20 + 5, 2 ** 26 - 3])
def test_verify_large_vocabularies(V):
    """Equal logits: the token of u is floor(u V), whatever the number of pieces. (A term passes fewer than 2^11
    additions, a lane's, a wave's and the pieces': a border is off by less than 2^11 2^-53 V < 2^-16 of a place; and by
    2048 places times the exponential's 2^-34, 2^-23, inside a piece. u V is kept 0.01 away from borders.) Greedy: the
    first largest, in the last piece."""
    say(f"verify, V {V}")
    z = torch.zeros((2, 1, V), dtype=torch.bfloat16, device="cuda")
    z[1, 0, V - 2] = 1.0
    z[1, 0, V - 1] = 1.0
    draft, heat = torch.zeros((2, 0), dtype=torch.int32, device="cuda"), torch.tensor([0.7, 0.0], device="cuda")
    for place in (0, 1, 2047, 2048, V // 3, V - 2049, V - 1):
        # the fp32 number nearest the middle of the place, and the place that this one lies in
        u = torch.tensor([[(place + 0.5) / V], [0.5]], dtype=torch.float32)
        x = float(u[0, 0]) * V
        if abs(x - round(x)) < 0.01:
            continue
        accepted, tokens, logprobs = gdn.draft_verify(z, draft, u.cuda(), temperature=heat)
        assert accepted.tolist() == [0, 0] and tokens[:, 0].tolist() == [min(int(x), V - 1), V - 2]
        assert abs(float(logprobs[0, 0]) + np.log(V)) < 2 ** -20 * np.log(V)


@pytest.mark.parametrize("V", [2 ** 20 + 5, 2 ** 26 - 20001])
def test_verify_every_part_of_a_large_vocabulary(V):
    """Equal logits, as above: places at both ends, between, and in the last piece, none of them skipped: u goes up by
    single steps until u V lies at least 0.1 from a border."""
    say(f"verify, all of V {V}")
    z = torch.zeros((1, 1, V), dtype=torch.bfloat16, device="cuda")
    none, ran = torch.zeros((1, 0), dtype=torch.int32, device="cuda"), 0
    for place in (0, 2047, 2048, 64 * 2048 - 1, 64 * 2048, V // 3, V // 2, V - V // 5, V - 5000, (V - 1) // 2048 * 2048):
        u = np.float32((place + 0.5) / V)
        while float(u) * V < place or not 0.1 <= float(u) * V % 1 <= 0.9:
            u = np.nextafter(u, np.float32(1))
        x = int(float(u) * V)
        assert place <= x < V and u < 1 and x // 2048 == place // 2048, (place, x)
        _, tokens, _ = gdn.draft_verify(z, none, torch.tensor([[float(u)]], device="cuda"))
        assert tokens.tolist() == [[x]], (place, tokens)
        ran += x // 2048 == (V - 1) // 2048
    assert ran >= 1


def test_verify_ties_and_steps():
    """Two tokens that share all of the mass, exactly: borders that a rounding would move."""
    z = np.full((4, 1, 9000), -np.inf)
    z[:, 0, [17, 8500]] = 3.0
    u = np.array([[0.0], [0.5 - 2.0 ** -25], [0.5], [1 - 2.0 ** -24]], np.float32)
    acc, tok, lp = gdn.draft_verify(dev(z, "fp32")[0], ints(np.zeros((4, 0))), torch.from_numpy(u).cuda())
    assert tok[:, 0].tolist() == [17, 17, 8500, 8500] and (lp - np.log(0.5)).abs().max() < 1e-7 and not acc.any()


# ---------------------------------------------------------------- states after accepted tokens

@pytest.mark.parametrize("flags", [(False, False, False), (True, False, False), (False, True, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,S,H,dk,dv", [(1, 1, 1, 1, 1), (3, 3, 2, 16, 16), (9, 3, 4, 56, 56), (4, 7, 3, 64, 64), (3, 2, 2, 7, 33),
                                         (2, 4, 2, 128, 128), (3, 5, 1, 65, 20), (2, 2, 2, 30, 101)])
def test_step_commit(N, S, H, dk, dv, dtype, flags):
    say(f"commit {N} {S} {H} {dk} {dv} {dtype} {flags}")
    additive, logits, norm_k = flags
    g = rng(9995)
    k, kf = dev(g.standard_normal((N, S, H, dk)) * (1 if norm_k else dk ** -0.5), dtype)
    v, vf = dev(g.standard_normal((N, S, H, dv)), dtype)
    draw = g.standard_normal if logits else g.random
    gg, gf = dev(draw((N, S, H)), "fp32")
    b, bf = dev(draw((N, S, H)), "fp32")
    A, Af = dev(g.standard_normal(H), "fp32")
    h, hf = dev(g.standard_normal((N, H, dk, dv)), "fp32")
    counts = g.integers(-1, S + 2, N)
    how = dict(additive=additive, gate_logits=logits, norm_k=norm_k)
    got = gdn.step_commit(k, v, gg, b, A, ints(counts), h, **how)
    want, tol = bound.commit(kf, vf, gf, bf, Af, counts, hf, additive, logits, norm_k)
    within("h", got, want, tol)
    assert torch.equal(got[torch.from_numpy(counts <= 0).cuda()], h[torch.from_numpy(counts <= 0).cuda()])
    # from nothing, and in place
    zero = gdn.step_commit(k, v, gg, b, A, ints(counts), **how)
    want0, tol0 = bound.commit(kf, vf, gf, bf, Af, counts, 0 * hf, additive, logits, norm_k)
    within("h from zero", zero, want0, tol0)
    there = h.clone()
    assert gdn.step_commit(k, v, gg, b, A, ints(counts), there, there, **how) is there and torch.equal(there, got)


def test_commit_reads_no_token_past_its_count():
    g = rng(9996)
    k, v = (dev(g.standard_normal((2, 4, 1, 8)), "bf16")[0] for _ in range(2))
    gg, b = (dev(g.random((2, 4, 1)), "fp32")[0] for _ in range(2))
    h, A = dev(g.standard_normal((2, 1, 8, 8)), "fp32")[0], torch.zeros(1, device="cuda")
    want = gdn.step_commit(k, v, gg, b, A, ints([2, 0]), h)
    for t in (k, v, gg, b):
        t[0, 2:], t[1] = float("nan"), float("nan")
    assert torch.equal(gdn.step_commit(k, v, gg, b, A, ints([2, 0]), h), want)


def test_commit_without_tokens_and_at_odd_addresses():
    h = torch.randn(3, 2, 8, 8, device="cuda")
    none = torch.zeros(3, 0, 2, 8, device="cuda")
    out = gdn.step_commit(none, none, none[..., 0], none[..., 0], torch.zeros(2, device="cuda"), ints([1, 1, 1]), h)
    assert torch.equal(out, h)
    # a state that begins on no 16-byte boundary
    g = rng(9997)
    k, v = (dev(g.standard_normal((3, 2, 2, 8)), "fp32")[0] for _ in range(2))
    gg, b, A = dev(g.random((3, 2, 2)), "fp32")[0], dev(g.random((3, 2, 2)), "fp32")[0], torch.zeros(2, device="cuda")
    odd = torch.empty(h.numel() + 1, device="cuda")[1:].view(h.shape)
    odd.copy_(h)
    want = gdn.step_commit(k, v, gg, b, A, ints([2, 1, 0]), h)
    assert torch.equal(gdn.step_commit(k, v, gg, b, A, ints([2, 1, 0]), odd), want)


# ---------------------------------------------------------------- streams, graphs, and all of it together

def all_calls(seed, dtype="bf16"):
    """One call of every operator, as (function of nothing, outputs' names): inputs are kept, states copied first."""
    sh, _ = shared_inputs((5, 2, 8, 64, 32, 16, [2, 40, 3, 100, 7], [300, 33], [0, 3, 5]), dtype, seed)
    ev, _ = evict_inputs((40, 16, [100, 257, 0], [50, 200, 3], 4, 8), dtype, seed, False)
    ve, _ = drafts(9, 3, 9000, dtype, seed, True, True, [0.0, 1.0])
    g = rng(seed)
    k, v = (dev(g.standard_normal((4, 3, 2, 56)), dtype)[0] for _ in range(2))
    gg, b, h = dev(g.random((4, 3, 2)), "fp32")[0], dev(g.random((4, 3, 2)), "fp32")[0], dev(
        g.standard_normal((4, 2, 56, 56)), "fp32")[0]
    A, counts = torch.zeros(2, device="cuda"), ints([0, 1, 3, 2])
    wt = torch.rand(sh[1].shape[:2], device="cuda")
    put = [ints(ve["draft"]), torch.from_numpy(ve["uniforms"]).cuda(), ve["draft_logits"], ints(ve["draft_lens"]),
           torch.from_numpy(ve["temperature"]).cuda()]
    t, lens, new, stack, free = ints(np.arange(30).reshape(3, 10)), ints([80, 3, 150]), ints([3, 3, 30]), ints(
        np.full(40, -1)), ints([4])

    def run():
        o, lse = gdn.mla_step_shared(*sh, scale=0.1)
        w = gdn.mla_weights(sh[0], sh[1], sh[2], sh[3], lse, wt.clone(), scale=0.1, decay=0.5)
        ew, ec = ev[0].clone(), ev[1].clone()
        el = gdn.mla_evict(ew, ec, *ev[2:], first=4, recent=8)
        s = stack.clone()
        n = gdn.page_trim(lens, new, t, s, free, 16)
        acc, tok, lp = gdn.draft_verify(ve["logits"], *put)
        hh = gdn.step_commit(k, v, gg, b, A, counts, h)
        return [o, lse, w, ew, ec, el, s, n, acc, tok, lp, hh]

    return run


def same(x, y):
    return all(torch.equal(bits(a) if a.is_floating_point() else a, bits(b) if b.is_floating_point() else b)
               for a, b in zip(x, y))


def test_captured_and_replayed():
    say("graph")
    run, other = all_calls(1), all_calls(2, "fp32")
    want, want2 = run(), other()
    torch.cuda.synchronize()
    graphs = []
    for f in (run, other):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = f()
        graphs.append((gr, out))
    for i in range(4):
        for (gr, out), w, f in zip(graphs, (want, want2), (run, other)):
            gr.replay()
            torch.cuda.synchronize()
            assert same(out, w), i
            assert same(f(), w), i
            torch.cuda.synchronize()


def test_two_streams_at_once():
    say("two streams")
    runs = [all_calls(3), all_calls(4, "fp32")]
    want = [f() for f in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(3):
        for s, f in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    assert all(same(x, want[i % 2]) for i, x in enumerate(got))


def test_two_evictions_at_once():
    """Moves of more segments than the chip holds workgroups, on two streams together: every wait ends, each is as alone."""
    page, N, n, d = 64, 96, 2048, 160
    cols, streams, runs = n // page, [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(9700 + i)
        table = torch.randperm(N * cols, generator=g, device="cuda").int().view(N, cols)
        cache = torch.randn((N * cols, page, d), generator=g, device="cuda").bfloat16()
        w = torch.randn((N * cols, page), generator=g, device="cuda")
        lens = torch.randint(1, n + 1, (N,), generator=g, device="cuda").int()
        keep = lens // 2
        alone = (w.clone(), cache.clone())
        out = gdn.mla_evict(*alone, table, lens, keep, first=4, recent=16)
        runs.append((w, cache, table, lens, keep, alone, out))
    torch.cuda.synchronize()
    for _ in range(3):
        copies = [(w.clone(), cache.clone()) for w, cache, *_ in runs]
        torch.cuda.synchronize()
        outs = []
        for s, c, r in zip(streams, copies, runs):
            with torch.cuda.stream(s):
                outs.append(gdn.mla_evict(*c, *r[2:5], first=4, recent=16))
        torch.cuda.synchronize()
        for c, r, o in zip(copies, runs, outs):
            assert torch.equal(o, r[6]) and torch.equal(c[0], r[5][0]) and torch.equal(bits(c[1]), bits(r[5][1]))


def test_workspaces_of_the_callers():
    say("workspaces")
    a, _ = shared_inputs(SHARED[4], "bf16", 11)
    big = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # (as floats: NaN)
    assert same(gdn.mla_step_shared(*a, scale=0.1, workspace=big), gdn.mla_step_shared(*a, scale=0.1))
    small = torch.empty(8, dtype=torch.uint8, device="cuda")  # too small: one of its own
    assert same(gdn.mla_step_shared(*a, scale=0.1, workspace=small), gdn.mla_step_shared(*a, scale=0.1))
    with pytest.raises(TypeError):
        gdn.mla_step_shared(*a, scale=0.1, workspace=small.float())
    e, _ = evict_inputs(EVICT[3], "bf16", 12, False)
    w, c = e[0].clone(), e[1].clone()
    big.fill_(255)
    assert same([gdn.mla_evict(*e, first=4, workspace=big), e[0], e[1]], [gdn.mla_evict(w, c, *e[2:], first=4), w, c])


def test_a_serving_loop():
    """Sequences behind a shared prefix: drafted tokens are written, attended to, verified, the rejected ones taken
    back, weights gathered and rows evicted, step after step, against the same loop over plain arrays in fp64."""
    say("serving loop")
    g = rng(77)
    N, S, H, dl, dr, page, V, P = 4, 2, 4, 32, 16, 4, 50, 13
    d, scale, budget, dk = dl + dr, 0.15, 14, 16
    pages, cols = 60, 12
    order = g.permutation(pages)
    pre, rest = order[:-(-P // page)], order[-(-P // page):]
    c0 = g.standard_normal((pages, page, d))
    cache, cf = dev(c0, "fp32")
    ptable, plens, starts = ints(pre[None]), ints([P]), ints([0, N])
    table, stack, n_free = ints(np.full((N, cols), -1)), ints(rest), ints([len(rest)])
    lens, weights = ints(np.zeros(N)), torch.full((pages, page), float("nan"), device="cuda")
    h, hf = dev(np.zeros((N, H, dk, dk)), "fp32")
    A, Af = dev(g.standard_normal(H), "fp32")
    rows = [np.zeros((0, d)) for _ in range(N)]   # each sequence's cached rows, and their weights
    mass = [np.zeros(0) for _ in range(N)]
    htol = np.zeros_like(hf)
    front = np.stack([cf[pre[j // page], j % page] for j in range(P)])
    for step in range(9):
        T = S + 1
        plan = gdn.page_plan(lens, ints([T] * N), table, stack, n_free, page, N * T, lens_out=lens, n_free_out=n_free)
        assert plan["granted"].tolist() == [T] * N
        new, newf = dev(g.standard_normal((N, T, d)), "fp32")
        gdn.mla_write(new[..., :dl].reshape(N * T, dl).contiguous(), new[..., dl:].reshape(N * T, dr).contiguous(),
                      plan["slots"], cache, norm=False)
        q, qf = dev(g.standard_normal((N, T, H, d)), "fp32")
        o, lse = gdn.mla_step_shared(q, cache, table, lens, dl, ptable, plens, starts, scale=scale)
        gdn.mla_weights(q, cache, table, lens, lse, weights, scale=scale, decay=0.5)
        # the same over plain arrays
        rows = [np.concatenate([r, newf[n]]) for n, r in enumerate(rows)]
        most = max(len(r) for r in rows)
        flat = np.zeros((N + 1, most + P, d))
        for n, r in enumerate(rows):
            flat[n, :len(r)] = r
        flat[N, :P] = front
        ids = np.arange(N)[:, None].astype(np.int32)
        real = [len(r) for r in rows]
        f = (qf, flat, ids, real, dl, np.array([[N]], np.int32), [P], [0, N])
        want, to, wl, tl = bound.shared(*f, scale, "fp32")
        within("o", o, want, to)
        within("lse", lse, wl, tl)
        old = np.zeros((N + 1, most + P))
        for n in range(N):
            old[n, :len(mass[n])] = mass[n]
        wm, wt = bound.weights(qf, flat, ids, real, host(lse), old, None, scale, 0.5)
        # drafts verified
        a, vf = drafts(N, S, V, "fp32", 500 + step, True, False, [0.0, 1.0])
        acc, tok, _ = gdn.draft_verify(a["logits"], ints(a["draft"]), torch.from_numpy(a["uniforms"]).cuda(),
                                       a["draft_logits"], None, torch.from_numpy(a["temperature"]).cuda())
        wa, wtok, _ = ref.draft_verify(*vf)
        assert (host(acc) == wa).all() and (host(tok) == wtok).all()
        # the recurrent layers' states, and the rejected tokens' rows and pages
        k, kf = dev(g.standard_normal((N, T, H, dk)) / 4, "fp32")
        v, vv = dev(g.standard_normal((N, T, H, dk)), "fp32")
        gg, gf = dev(g.random((N, T, H)), "fp32")
        b, bf = dev(g.random((N, T, H)), "fp32")
        before = host(h)
        gdn.step_commit(k, v, gg, b, A, acc + 1, h, h)
        hw, ht = bound.commit(kf, vv, gf, bf, Af, wa + 1, before, False, False, False)
        within("h", h, hw, ht)
        kept = lens - (S - acc)
        gdn.page_trim(lens, kept, table, stack, n_free, page, n_free_out=n_free)
        lens = kept
        rows = [r[:len(r) - (S - x)] for r, x in zip(rows, wa)]
        assert lens.tolist() == [len(r) for r in rows]
        tb = table.cpu().numpy()
        for n, r in enumerate(rows):
            at = [(tb[n, j // page], j % page) for j in range(len(r))]
            got = np.array([float(weights[p, i]) for p, i in at])
            assert (np.abs(got - wm[n, :len(r)]) <= wt[n, :len(r)] + 1e-6 * wm[n, :len(r)]).all()
            mass[n] = got
        # rows of least weight go once a sequence passes its budget
        fewer = gdn.mla_evict(weights, cache, table, lens, ints([budget] * N), first=1, recent=3)
        gdn.page_trim(lens, fewer, table, stack, n_free, page, n_free_out=n_free)
        for n in range(N):
            m = len(rows[n])
            if m > budget:
                best = sorted(range(1, m - 3), key=lambda j: (-mass[n][j], j))[:budget - 4]
                stay = [0] + sorted(best) + list(range(m - 3, m))
                rows[n], mass[n] = rows[n][stay], mass[n][stay]
        lens = fewer
        assert lens.tolist() == [len(r) for r in rows]
        tb, c = table.cpu().numpy(), host(cache)
        for n, r in enumerate(rows):
            for j in range(len(r)):
                assert (c[tb[n, j // page], j % page] == r[j]).all()
        # no page is lost or given twice
        held = [int(p) for n, r in enumerate(rows) for p in tb[n, :-(-len(r) // page)]]
        free = stack[:int(n_free)].tolist()
        assert sorted(held + free) == sorted(int(x) for x in rest)


def test_positions_behind_a_prefix_and_after_evictions():
    """page_plan counts the rows a sequence holds. With what it has in front and what it has lost added, every cached
    rotary key is turned by its token's place in the whole text, prefix, evicted rows and sequences that end included."""
    say("positions")
    g = rng(78)
    N, P, dl, dr, page, pages, cols, cap = 5, 6, 16, 8, 4, 80, 12, 16
    stack, n_free, table = ints(g.permutation(pages)), ints([pages]), ints(np.full((N, cols), -1))
    lens, weights, front = ints(np.zeros(N)), torch.zeros((pages, page), device="cuda"), ints([P, 0, P, 0, P])
    cache, away = torch.full((pages, page, dl + dr), float("nan"), device="cuda"), front.clone()
    freqs = 100.0 ** (-np.arange(dr // 2) / (dr // 2))
    fr = torch.tensor(freqs, device="cuda")
    held = [[] for _ in range(N)]  # the rows of each sequence: key before its turn, place in the text
    told = [int(x) for x in front]  # tokens of the text so far
    for step in range(12):
        new = g.integers(0, 5, N)
        if step in (5, 9):
            new[step % N] = -1
            away[step % N], held[step % N], told[step % N] = front[step % N], [], int(front[step % N])
        plan = gdn.page_plan(lens, ints(new), table, stack, n_free, page, cap, lens_out=lens, n_free_out=n_free)
        seq = torch.searchsorted(plan["starts"], torch.arange(cap, dtype=torch.int32, device="cuda"), right=True) - 1
        positions = plan["positions"] + away[seq.clamp(max=N - 1)]
        c, kr = torch.zeros((cap, dl), device="cuda"), dev(g.standard_normal((cap, dr)), "fp32")
        gdn.mla_write(c, kr[0], plan["slots"], cache, None, positions, fr, norm=False)
        t = 0
        for n, k in enumerate(plan["granted"].tolist()):
            for _ in range(k):
                held[n].append((kr[1][t], told[n]))
                told[n] += 1
                t += 1
        # some new tokens are taken back (their places are given again), then rows are dropped (theirs are not)
        back = np.minimum(g.integers(0, 3, N), np.maximum(plan["granted"].cpu().numpy(), 0))
        kept = lens - ints(back)
        gdn.page_trim(lens, kept, table, stack, n_free, page, n_free_out=n_free)
        for n, k in enumerate(back):
            held[n] = held[n][:len(held[n]) - k]
            told[n] -= k
        weights.copy_(torch.rand((pages, page), generator=torch.Generator("cuda").manual_seed(step), device="cuda"))
        w, tb = host(weights), table.cpu().numpy()
        fewer = gdn.mla_evict(weights, cache, table, kept, ints([7] * N), first=1, recent=2)
        away += kept - fewer
        gdn.page_trim(kept, fewer, table, stack, n_free, page, n_free_out=n_free)
        lens = fewer
        for n, rows in enumerate(held):
            m = len(rows)
            if m > 7:
                best = sorted(range(1, m - 2), key=lambda j: (-w[tb[n, j // page], j % page], j))[:4]
                held[n] = [rows[j] for j in [0] + sorted(best) + [m - 2, m - 1]]
        assert lens.tolist() == [len(r) for r in held]
        got, tb = host(cache), table.cpu().numpy()
        for n, rows in enumerate(held):
            for j, (k, place) in enumerate(rows):
                want = latent.turn(k[None, None], np.array([place]), freqs, False)[0, 0]
                x = got[tb[n, j // page], j % page, dl:]
                # two products with a sine or cosine, each off by 2^-21 and ten roundings
                assert (np.abs(x - want) <= 2 * (2.0 ** -21 + 10 * U) * np.abs(k).max()).all(), (step, n, j, place)
    assert max(told) > P + 14 and int((away - front).max()) > 0
