"""Latent attention (expanded forward and backward, paged step), the per-head
norm with rotation, the cache write and the page plan against their fp64
definitions, at sizes and masks where they can go wrong. The bounds are the
worst-case rounding sums of latent_util."""
import numpy as np
import pytest
import torch

import gated_delta_rule_74_amd as gdn
from gpu_util import say
from latent_util import H16, TYPES, U, attention, dev, host, ints, rng, step, within
from oracle import latent as ref

pytestmark = pytest.mark.gpu

# B, Tq, past, H, Hk, Hr, dn, dr, dv, lens
ATTN = [
    (1, 1, 0, 1, 1, 1, 8, 8, 8, None),
    (1, 2, 0, 2, 1, 1, 16, 8, 8, None),
    (2, 63, 0, 2, 2, 1, 16, 16, 16, [63, 1]),
    (2, 64, 0, 4, 2, 2, 56, 32, 56, None),
    (3, 65, 0, 4, 4, 1, 56, 32, 56, [65, 0, 64]),
    (1, 129, 0, 2, 1, 1, 128, 64, 128, None),
    (2, 130, 0, 2, 2, 2, 64, 0, 64, [129, 7]),
    (2, 17, 100, 4, 1, 1, 32, 16, 24, [117, 101]),
    (3, 70, 63, 2, 2, 1, 40, 24, 72, [64, 63, 133]),
    (1, 257, 1, 2, 2, 1, 96, 32, 48, None),
    (1, 1, 200, 8, 2, 1, 24, 8, 104, None),
    (2, 140, 0, 2, 1, 1, 8, 64, 128, [-5, 1000]),
]


def attn_inputs(case, dtype, seed, sharp=1.0):
    B, Tq, past, H, Hk, Hr, dn, dr, dv, lens = case
    g, Tk = rng(seed), Tq + past
    shapes = [(B, Tq, H, dn + dr), (B, Tk, Hk, dn), (B, Tk, Hr, dr) if dr else None, (B, Tk, Hk, dv), (B, Tq, H, dv)]
    pairs = [(None, None) if s is None else dev(g.standard_normal(s) * (sharp if i < 3 else 1), dtype)
             for i, s in enumerate(shapes)]
    return [p[0] for p in pairs], [p[1] for p in pairs], None if lens is None else ints(lens), (dn + dr) ** -0.5


def run_attn(t, lens, scale):
    q, k, kr, v, do = t
    o, lse = gdn.mla_fwd(q, k, v, kr, lens, scale=scale)
    r = gdn.mla_bwd(q, k, v, o, lse, do, kr, lens, scale=scale)
    return {"o": o, "lse": lse, "dq": r["dq"], "dk": r["dk"], "dkr": r["dk_rope"], "dv": r["dv"]}


def check_attn(case, dtype, seed, sharp=1.0):
    t, f, lens, scale = attn_inputs(case, dtype, seed, sharp)
    got = run_attn(t, lens, scale)
    q, k, kr, v, do = f
    want = attention(q, k, kr, v, case[-1], scale, do, dtype)
    for n, (x, tol) in want.items():
        within(n, got[n], x, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(map(str, c[:9])))
def test_attention(case, dtype):
    say(f"attention {case} {dtype}")
    check_attn(case, dtype, 7900)


# B, Tq, past, H, Hk, Hr, dn, dr, dv: heads enough that every size of block is taken, paired and not
MANY = [
    (16, 300, 37, 64, 64, 16, 56, 32, 56), (16, 300, 0, 64, 64, 16, 128, 64, 128), (64, 140, 0, 16, 8, 8, 32, 16, 40),
    (16, 257, 3, 64, 32, 32, 96, 24, 64), (16, 270, 0, 64, 64, 64, 32, 0, 32), (8, 270, 0, 64, 64, 16, 64, 0, 104),
    # blocks of 64 rows: more than two for each CU, fewer
    (4, 200, 0, 64, 64, 16, 56, 32, 56), (4, 200, 10, 64, 32, 16, 128, 64, 128), (4, 210, 0, 64, 64, 16, 32, 0, 24),
    (2, 200, 0, 64, 64, 16, 56, 32, 56), (2, 190, 30, 64, 32, 16, 128, 64, 128), (2, 200, 0, 64, 64, 64, 104, 0, 64),
]


def slices_within(f, got, case, dtype, lens, scale, where):
    """The heads that share rotary head g of sequence b, for every (b, g) of `where`."""
    H, Hk, Hr = case[3:6]
    parts = {"q": H, "k": Hk, "kr": Hr, "v": Hk, "do": H, "o": H, "lse": H, "dq": H, "dk": Hk, "dkr": Hr, "dv": Hk}

    def cut(n, x, b, g):
        per = parts[n] // Hr
        return None if x is None else x[b:b + 1, :, g * per:(g + 1) * per]

    for b, g in where:
        q, k, kr, v, do = (cut(n, x, b, g) for n, x in zip(("q", "k", "kr", "v", "do"), f))
        for n, (x, tol) in attention(q, k, kr, v, None if lens is None else lens[b:b + 1], scale, do, dtype).items():
            within(f"{n} of sequence {b}, group {g}", cut(n, got[n], b, g), x, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_attention_with_many_heads(case, dtype):
    say(f"attention, many heads {case} {dtype}")
    B, Tq, past, Hr = case[0], case[1], case[2], case[5]
    lens = [Tq + past - 9 * b for b in range(B)]
    lens[-1] = 0
    t, f, ln, scale = attn_inputs(case + (lens,), dtype, 7910)
    got = run_attn(t, ln, scale)
    slices_within(f, got, case, dtype, lens, scale, [(0, 0), (0, Hr - 1), (B // 2, Hr // 2), (B - 2, Hr - 1)])
    assert not got["o"][-1, past:].any() and not got["dk"][-1].any() and not got["dv"][-1].any()


def test_attention_beyond_32_bit_offsets():
    """Keys of more than 2^32 bytes, the last head checked."""
    case = (1, 16, 14984, 600, 600, 600, 128, 0, 8)
    say(f"attention {case} fp32")
    B, Tq, past, H, dn, dv = 1, 16, 14984, 600, 128, 8
    make = lambda *s: torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(s[1]))  # noqa: E731
    t = [make(B, Tq, H, dn), make(B, Tq + past, H, dn), None, make(B, Tq + past, H, dv), make(B, Tq, H, dv)]
    assert t[1].numel() * 4 > 2 ** 32
    got = run_attn(t, None, 0.1)
    f = [None if x is None else host(x[:, :, -1:]) for x in t]
    want = attention(f[0], f[1], None, f[3], None, 0.1, f[4], "fp32")
    for n, (x, tol) in want.items():
        within(n, got[n][:, :, -1:], x, tol)


def test_a_chunk_of_shared_heads_after_a_long_context():
    """Few queries of many heads beside many keys of few: every tensor is small, B Tk H D is not."""
    B, Tq, past, H, Hk, Hr, dn, dr, dv = 1, 24, 131072, 128, 16, 16, 128, 64, 128
    say(f"attention {Tq} queries after {past} keys, {H} heads on {Hk}, bf16")
    assert B * (Tq + past) * H * (dn + dr) >= 2 ** 31
    gen = torch.Generator("cuda").manual_seed(7904)
    q, k, kr, v, do = (torch.randn(s, device="cuda", generator=gen).bfloat16() for s in (
        (B, Tq, H, dn + dr), (B, Tq + past, Hk, dn), (B, Tq + past, Hr, dr), (B, Tq + past, Hk, dv), (B, Tq, H, dv)))
    scale = (dn + dr) ** -0.5
    got = run_attn([q, k, kr, v, do], None, scale)
    f = [host(x) for x in (q[:, :, -8:], k[:, :, -1:], kr[:, :, -1:], v[:, :, -1:], do[:, :, -8:])]
    for n, (x, tol) in attention(*f[:4], None, scale, f[4], "bf16").items():
        within(n, got[n][:, :, -x.shape[2]:], x, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_with_sharp_scores(dtype):
    """Scores far apart: the maximum moves late, most weights vanish."""
    say(f"attention, scores of +-100, {dtype}")
    check_attn((1, 200, 30, 2, 2, 1, 56, 32, 56, None), dtype, 7901, sharp=6.0)


def test_rising_scores_move_the_maximum_in_every_tile():
    """Keys that grow along the sequence by more than the lazy maximum allows."""
    say("attention, scores rising by 40 a tile")
    B, T, d = 1, 300, 16
    k = np.zeros((B, T, 1, d))
    k[0, :, 0, 0] = np.arange(T) * 0.625
    q = np.zeros((B, T, 1, d))
    q[..., 0] = 4.0
    g = rng(5)
    v, do = g.standard_normal((B, T, 1, 8)), g.standard_normal((B, T, 1, 8))
    pairs = [dev(x, "fp32") for x in (q, k, v, do)]
    got = run_attn([pairs[0][0], pairs[1][0], None, pairs[2][0], pairs[3][0]], None, 0.25)
    want = attention(pairs[0][1], pairs[1][1], None, pairs[2][1], None, 0.25, pairs[3][1], "fp32")
    for n, (x, tol) in want.items():
        within(n, got[n], x, tol)


def fp32_delta(q, k, kr, v, scale, do):
    """fp64 dq and dk of one sequence of unshared heads, and bounds of latent_util's kind. Rows that see up to
    256 keys: without the rounding of o to bf16, delta being sum P dP, formed in fp32 from the products. Rows
    after them may take delta = do . o, whose o carries the two roundings of its bound there (P as an operand:
    h sum P |v|; the output: h |o|), so edl grows by |do| . (h sum P |v| + h |o|) (1 + rel)."""
    dq, dk, _, _ = ref.attn_bwd(q, k, kr, v, None, scale, do)
    o, _, P = ref.attn_fwd(q, k, kr, v, None, scale)
    D, dv, tq, tk = q.shape[3], v.shape[3], np.zeros_like(dq), np.zeros_like(dk)
    for h in range(q.shape[2]):
        kk, vv, p, g = ref._keys(k, kr, 0, h, q.shape[2]), v[0, :, h], P[0, h], do[0, :, h]
        n = (p > 0).sum(1, keepdims=True)
        ez = ((D + 8) * U * scale * np.abs(q[0, :, h]) @ np.abs(kk).T * (p > 0)).max(1, keepdims=True)
        rel = np.expm1(2 * ez + (n + 16) * U)
        dp, adp = g @ vv.T, np.abs(g) @ np.abs(vv).T
        dl = (p * dp).sum(1, keepdims=True)
        edl = ((rel + n * U) * np.abs(dp) * p + (dv + 4) * U * adp * p * (1 + rel)).sum(1, keepdims=True)
        eo = (rel + n * U) * (p @ np.abs(vv)) + H16 * (p @ np.abs(vv) + np.abs(o[0, :, h])) * (1 + rel)
        edl += np.where(n > 256, (np.abs(g) * eo).sum(1, keepdims=True), 0.0)
        ds = p * (dp - dl)
        eds = rel * np.abs(ds) + p * ((dv + 4) * U * adp + edl + 4 * U * (np.abs(dp) + np.abs(dl))) * (1 + rel)
        eds = eds + H16 * (np.abs(ds) + eds)  # an operand in bf16
        m = (p > 0).sum(0)[:, None]
        tq[0, :, h] = scale * (eds @ np.abs(kk) + (n + 4) * U * np.abs(ds) @ np.abs(kk))
        tk[0, :, h] = scale * (eds.T @ np.abs(q[0, :, h]) + (m + 4) * U * np.abs(ds).T @ np.abs(q[0, :, h]))[
            :, :k.shape[3]]
    return {n: (x, t * (1 + H16) + (H16 + 8 * U) * np.abs(x)) for n, x, t in (("dq", dq, tq), ("dk", dk, tk))}


@pytest.mark.parametrize("B,H,Tq,past,dn,dr,dv", [
    (16, 32, 256, 0, 128, 64, 128), (16, 32, 256, 1, 128, 64, 128), (16, 32, 256, 30, 128, 64, 128),
    (16, 32, 250, 255, 128, 64, 128), (32, 32, 128, 140, 56, 32, 56), (3, 4, 70, 1, 56, 32, 56),
    (3, 4, 70, 230, 56, 32, 56)])
def test_gradients_of_rows_that_see_few_keys(B, H, Tq, past, dn, dr, dv):
    """Values one bf16 step apart: dP - delta is as small as the rounding of o, and is kept free of it in
    every size of block, wherever the cached keys let the block begin."""
    say(f"attention backward, B {B} H {H} Tq {Tq} after {past}, values a step apart, bf16")
    gen = torch.Generator("cuda").manual_seed(7905)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    Tk = Tq + past
    q, do = (0.05 * r(B, Tq, H, dn + dr)).bfloat16(), r(B, Tq, H, dv).bfloat16()
    k, kr = (1 + 0.25 * r(B, Tk, H, dn)).bfloat16(), (1 + 0.25 * r(B, Tk, H, dr)).bfloat16()
    v = torch.where(r(B, Tk, H, dv) > 0, 1.0, 1.0 + 2.0 ** -7).bfloat16()
    scale = (dn + dr) ** -0.5
    got = run_attn([q, k, kr, v, do], None, scale)
    for b, h in ((0, 0), (B - 1, H - 1)):
        f = [host(x[b:b + 1, :, h:h + 1]) for x in (q, k, kr, v, do)]
        for n, (x, tol) in fp32_delta(*f[:4], scale, f[4]).items():
            within(f"{n} of sequence {b}, head {h}", got[n][b:b + 1, :, h:h + 1], x, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_is_not_read_and_its_gradients_are_zero(dtype):
    """NaN past the lengths changes nothing; padded rows get zeros."""
    say(f"attention, NaN in the padding, {dtype}")
    case = (3, 90, 20, 4, 2, 1, 24, 8, 16, [110, 37, 0])
    t, _, lens, scale = attn_inputs(case, dtype, 7902)
    clean = run_attn(t, lens, scale)
    for b, n in enumerate(case[-1]):
        for x in t[1:4]:
            x[b, n:] = float("nan")
        t[0][b, max(0, n - 20):] = float("nan")
        t[4][b, max(0, n - 20):] = float("nan")
    dirty = run_attn(t, lens, scale)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    for b, n in enumerate(case[-1]):
        assert not dirty["dk"][b, n:].any() and not dirty["dv"][b, n:].any() and not dirty["dkr"][b, n:].any()
        assert not dirty["o"][b, max(0, n - 20):].any() and not dirty["dq"][b, max(0, n - 20):].any()
        assert (dirty["lse"][b, max(0, n - 20):] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,past,H,dn,dr,dv", [(1, 700, 0, 2, 56, 32, 56), (1, 500, 130, 16, 16, 16, 16),
                                                 (4, 520, 40, 64, 56, 32, 56), (16, 600, 0, 64, 128, 64, 128)])
def test_how_far_a_nan_reaches(B, T, past, H, dn, dr, dv, dtype):
    """NaN in a key's and value's row leaves queries more than 160 positions before it as they were, NaN in a
    query's and its gradient's row the gradients of keys more than 160 after it and all other queries."""
    say(f"attention, one NaN row, B {B} T {T} after {past} H {H} {dn} + {dr} | {dv} {dtype}")
    t, _, lens, scale = attn_inputs((B, T, past, H, H, H, dn, dr, dv, None), dtype, 7906)
    clean = run_attn(t, lens, scale)
    at, i = past + 333, 333  # position of the row, its query
    others = torch.arange(T, device="cuda") != i
    for x, name in enumerate(("q", "k", "k_rope", "v", "do")):
        of_query = name in ("q", "do")
        row = i if of_query else at
        keep = t[x][0, row].clone()
        t[x][0, row] = float("nan")
        dirty = run_attn(t, lens, scale)
        t[x][0, row] = keep
        for n in clean:
            assert torch.equal(dirty[n][1:], clean[n][1:]), (name, n)
        if not of_query:
            assert dirty["dq"][0, i:].isnan().any()
            for n in ("o", "lse", "dq"):
                assert torch.equal(dirty[n][0, :i - 160], clean[n][0, :i - 160]), (name, n)
        else:
            assert dirty["dk"][0, at].isnan().any()
            for n in ("dk", "dkr", "dv"):
                assert torch.equal(dirty[n][0, at + 161:], clean[n][0, at + 161:]), (name, n)
            for n in ("o", "lse", "dq"):
                assert torch.equal(dirty[n][0, others], clean[n][0, others]), (name, n)


def test_attention_is_reproducible_and_keeps_to_its_buffers():
    say("attention twice, guard rows around every output")
    case = (2, 100, 0, 4, 2, 1, 56, 32, 56, [100, 77])
    t, _, lens, scale = attn_inputs(case, "bf16", 7903)
    a, b = run_attn(t, lens, scale), run_attn(t, lens, scale)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    q, k, kr, v, do = t
    flat = torch.full((64 + q.numel() + 64,), 7.0, dtype=q.dtype, device="cuda")
    out = {"dq": flat[64:-64].view_as(q)}
    gdn.mla_bwd(q, k, v, a["o"], a["lse"], do, kr, lens, scale=scale, out=out)
    assert torch.equal(out["dq"], a["dq"]) and (flat[:64] == 7).all() and (flat[-64:] == 7).all()


def test_no_query_leaves_zero_gradients():
    say("attention backward without queries")
    z = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, v = z(2, 0, 4, 24), z(2, 5, 2, 16), z(2, 5, 2, 8)
    o, lse = gdn.mla_fwd(q, k, v, z(2, 5, 1, 8))
    r = gdn.mla_bwd(q, k, v, o, lse, z(2, 0, 4, 8), z(2, 5, 1, 8))
    assert o.shape == (2, 0, 4, 8) and not r["dk"].any() and not r["dv"].any() and not r["dk_rope"].any()


def test_autograd_against_differences():
    """Gradients through LatentAttention and NormRope against central
    differences of the fp64 definition along random directions."""
    say("autograd of norm, rotation and attention")
    B, T, H, dn, dr, dv = 2, 21, 4, 16, 8, 16
    g = rng(11)
    raw = {"q": g.standard_normal((B, T, H, dn + dr)), "k": g.standard_normal((B, T, 2, dn)),
           "kr": g.standard_normal((B, T, 1, dr)), "v": g.standard_normal((B, T, 2, dv)),
           "w": 1 + 0.1 * g.standard_normal(dn + dr)}
    do, pos = g.standard_normal((B, T, H, dv)), np.tile(np.arange(T), (B, 1))
    fr = 100.0 ** (-np.arange(dr // 2) / (dr // 2))
    lens, scale = [T, 13], 0.3

    def f64(p):
        qn = ref.norm_rope(p["q"].reshape(B * T, H, -1), p["w"], pos.ravel(), fr, True, 1e-6, False)
        kr = ref.norm_rope(p["kr"].reshape(B * T, 1, -1), None, pos.ravel(), fr, False, 1e-6, False)
        o = ref.attn_fwd(qn.reshape(B, T, H, -1), p["k"], kr.reshape(B, T, 1, -1), p["v"], lens, scale)[0]
        return (o * do).sum()

    t = {n: torch.tensor(x, dtype=torch.float32, device="cuda", requires_grad=True) for n, x in raw.items()}
    ps, ft = ints(pos), torch.tensor(fr, device="cuda")
    qn = gdn.NormRope.apply(t["q"], t["w"], ps, ft)
    kr = gdn.NormRope.apply(t["kr"], None, ps, ft, False)
    o = gdn.LatentAttention.apply(qn, t["k"], t["v"], kr, ints(lens), scale)
    o.backward(torch.tensor(do, dtype=torch.float32, device="cuda"))
    p32 = {n: host(x) for n, x in t.items()}
    for n in raw:
        d = rng(12).standard_normal(raw[n].shape)
        up, down = ({**p32, n: p32[n] + e * d} for e in (1e-5, -1e-5))
        want, have = (f64(up) - f64(down)) / 2e-5, (host(t[n].grad) * d).sum()
        # fp32 gradients: every term off by at most ~2^-18 of sum |grad| |d|; the differences by 1e-8
        assert abs(want - have) <= 2.0 ** -18 * np.abs(host(t[n].grad) * d).sum() + 1e-6, n


# N, S, H, dl, dr, page, cols, lens
STEP = [
    (1, 1, 1, 16, 0, 1, 3, [2]),
    (3, 1, 16, 128, 32, 64, 4, [200, 1, 0]),
    (2, 3, 16, 128, 32, 16, 9, [140, 2]),
    (2, 2, 5, 48, 8, 24, 8, [190, 25]),
    (1, 1, 16, 512, 64, 64, 20, [1237]),
    (2, 4, 24, 256, 64, 16, 12, [177, 128]),
    (1, 7, 3, 496, 40, 7, 60, [419]),
    (4, 1, 8, 64, 64, 128, 3, [384, 1000, -3, 129]),
    (1, 1, 33, 80, 16, 32, 40, [1280]),
    (130, 1, 4, 32, 8, 16, 40, [i * i % 641 for i in range(130)]),
    (67, 2, 2, 384, 16, 32, 8, [(37 * i) % 250 for i in range(67)]),
    (3, 1, 2, 192, 64, 64, 190, [12160, 5, 9001]),
    # tables wide enough for two query blocks per workgroup
    (6, 2, 12, 128, 40, 16, 2500, [700, 0, 33, 64, 2, 1]),
    (5, 1, 40, 256, 64, 64, 700, [150, 1, 128, 0, 63]),
    (4, 1, 20, 176, 8, 32, 1600, [129, 300, 31, 7]),
]


def paged(case, dtype, seed):
    N, S, H, dl, dr, page, cols, lens = case
    g = rng(seed)
    pages = N * cols + 3
    table = g.permutation(pages)[:N * cols].reshape(N, cols)
    cache = g.standard_normal((pages, page, dl + dr))
    for n in range(N):  # entries past the length may be anything; so may the rows no sequence holds
        used = -(-min(max(lens[n], 0), cols * page) // page)
        table[n, used:] = [-1, 1 << 30, -(1 << 31)][n % 3]
    q, qf = dev(g.standard_normal((N, S, H, dl + dr)) * 2, dtype)
    c, cf = dev(cache, dtype)
    return q, qf, c, cf, table.astype(np.int32), (dl + dr) ** -0.5


def spoil(c, table, lens, page):
    """NaN in every cache row that no sequence holds."""
    held = torch.zeros(c.shape[:2], dtype=torch.bool)
    for n, m in enumerate(lens):
        for p in range(min(max(m, 0), table.shape[1] * page)):
            held[table[n, p // page], p % page] = True
    c[~held.cuda()] = float("nan")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c[:7])))
def test_step(case, dtype):
    say(f"paged step {case} {dtype}")
    N, S, H, dl, dr, page, cols, lens = case
    q, qf, c, cf, table, scale = paged(case, dtype, 7910)
    spoil(c, table, lens, page)
    o, lse = gdn.mla_step(q, c, ints(table), ints(lens), dl, scale=scale)
    wo, to, wl, tl = step(qf, cf, table, lens, dl, scale, dtype)
    within("o", o, wo, to)
    within("lse", lse, wl, tl)
    again = gdn.mla_step(q, c, ints(table), ints(lens), dl, scale=scale)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dl,H", [(48, 3), (80, 1), (112, 2), (176, 5), (336, 1), (496, 3)])
def test_step_joins_widths_that_leave_threads_over(dl, H):
    """One long sequence in many parts, its columns dealt to a number of threads that does not divide the workgroup."""
    say(f"paged step, many parts of {dl} columns")
    case = (1, 1, H, dl, 8, 64, 120, [7600])
    q, qf, c, cf, table, scale = paged(case, "fp32", 7913)
    o, lse = gdn.mla_step(q, c, ints(table), ints(case[-1]), dl, scale=scale)
    wo, to, wl, tl = step(qf, cf, table, case[-1], dl, scale, "fp32")
    within("o", o, wo, to)
    within("lse", lse, wl, tl)


def test_step_masks_pages_outside_the_pool():
    say("paged step, bad table entries inside the length")
    case = (2, 2, 4, 64, 8, 8, 12, [90, 33])
    q, qf, c, cf, table, scale = paged(case, "fp32", 7911)
    table[0, 3], table[0, 7], table[1, 0], table[1, 4] = -1, len(cf), 1 << 30, -(1 << 31)
    o, lse = gdn.mla_step(q, c, ints(table), ints(case[-1]), 64, scale=scale)
    wo, to, wl, tl = step(qf, cf, table, case[-1], 64, scale, "fp32")
    within("o", o, wo, to)
    within("lse", lse, wl, tl)


def test_step_with_every_page_outside_the_pool():
    say("paged step, no readable row")
    q, qf, c, cf, table, scale = paged((2, 1, 4, 64, 8, 8, 40, [300, 5]), "bf16", 7912)
    o, lse = gdn.mla_step(q, c, ints(np.full_like(table, -1)), ints([300, 5]), 64, scale=scale)
    assert not o.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("n", [5, 90, 40000])
def test_step_with_a_nan_query(n):
    """NaN in one head's query: that head gets NaN, cut into parts or not, the others what they had."""
    say(f"step, a NaN query, {n} rows")
    page, dl, dr, H = 64, 64, 16, 3
    pages = -(-n // page)
    g = rng(17)
    cache, _ = dev(g.standard_normal((pages, page, dl + dr)), "bf16")
    q, _ = dev(g.standard_normal((1, H, dl + dr)), "bf16")
    table = ints(np.arange(pages)[None])
    o, lse = gdn.mla_step(q, cache, table, ints([n]), dl, scale=0.1)
    q[0, 1, 0] = float("nan")
    o1, lse1 = gdn.mla_step(q, cache, table, ints([n]), dl, scale=0.1)
    assert o1[0, 1].isnan().all() and lse1[0, 1].isnan()
    for h in (0, 2):
        assert torch.equal(o[0, h], o1[0, h]) and torch.equal(lse[0, h], lse1[0, h])


def test_step_beyond_32_bit_offsets():
    """Rows past 2^32 bytes (and 2^31 elements) of the cache, written and read there."""
    say("cache of 5.4 GB: write and step at its end")
    page, d, dl, dr = 64, 576, 512, 64
    pages = 73000  # 2.7e9 elements
    cache = torch.empty((pages, page, d), dtype=torch.bfloat16, device="cuda")
    g = rng(3)
    ids = np.array([[pages - 1, 60000, 59000, pages - 7]])
    n = 4 * page - 5
    c, cf = dev(g.standard_normal((n, dl)), "bf16")
    kr, krf = dev(g.standard_normal((n, dr)), "bf16")
    slots = ids[0, np.arange(n) // page] * page + np.arange(n) % page
    gdn.mla_write(c, kr, ints(slots), cache, norm=False)
    rows = cache[torch.from_numpy(ids[0]).cuda().long()].view(-1, d)[:n]
    assert torch.equal(rows, torch.cat([c, kr], 1))
    q, qf = dev(g.standard_normal((1, 1, 16, d)), "bf16")
    o, lse = gdn.mla_step(q, cache, ints(ids), ints([n]), dl, scale=d ** -0.5)
    small = np.zeros((4, page, d))
    small.reshape(-1, d)[:n] = np.concatenate([cf, krf], 1)
    wo, to, wl, tl = step(qf, small, np.arange(4)[None], [n], dl, d ** -0.5, "bf16")
    within("o", o, wo, to)
    within("lse", lse, wl, tl)


# M, H, d, r, interleaved, norm, weight
NORM = [
    (1, 1, 2, 2, True, True, True), (3, 2, 7, 4, False, True, True), (5, 3, 7, 2, True, True, False),
    (33, 16, 88, 32, False, True, True), (33, 16, 88, 32, True, True, True), (9, 4, 56, 14, False, True, True),
    (70, 1, 512, 512, False, True, True), (70, 1, 64, 64, True, False, False), (17, 8, 200, 0, False, True, True),
    (300, 5, 24, 16, False, True, True), (2, 1, 509, 508, False, True, True), (11, 3, 40, 40, False, False, False),
    (1000, 1, 1, 0, False, True, True),
    # rows enough for several per thread
    (3001, 16, 88, 32, False, True, True), (4100, 9, 128, 64, True, True, True), (50001, 1, 64, 16, False, True, False),
    # interleaved turns that begin inside eight columns
    (21, 3, 64, 12, True, True, True), (6, 2, 8, 2, True, True, False), (300, 16, 24, 22, True, False, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)))
def test_norm_rope(case, dtype):
    say(f"norm and rotation {case} {dtype}")
    M, H, d, r, inter, norm, weight = case
    g, h = rng(7920), H16 if dtype == "bf16" else 0.0
    x, xf = dev(g.standard_normal((M, H, d)), dtype)
    dy, dyf = dev(g.standard_normal((M, H, d)), dtype)
    w, wf = dev(1 + 0.1 * g.standard_normal(d), "fp32") if weight else (None, None)
    pos = g.integers(0, 2 ** 31 - 1, M)
    pos[0] = 0
    fr = 10000.0 ** (-np.arange(r // 2) / max(r // 2, 1)) if r else None
    args = (w, ints(pos), torch.tensor(fr, device="cuda")) if r else (w, None, None)
    kw = dict(norm=norm, eps=1e-6, interleaved=inter)
    y = gdn.norm_rope(x, *args, **kw)
    back = gdn.norm_rope_bwd(dy, x, *args, **kw)
    want = ref.norm_rope(xf, wf, pos, fr, norm, 1e-6, inter)
    wdx, wdw = ref.norm_rope_bwd(dyf, xf, wf, pos, fr, norm, 1e-6, inter)
    # sine and cosine: the angle to 2^-24 of a turn (pi 2^-24 each side of rounding) and a few steps; far positions:
    # the fp64 product of position and frequency is off by 2^31 2^-53 radians at most
    ang = 8 * U + 2.0 ** -21
    ww = 1.0 if wf is None else np.abs(wf)
    inv = 1 / np.sqrt((xf ** 2).mean(-1, keepdims=True) + 1e-6) if norm else np.ones((M, H, 1))
    row = np.abs(xf) * inv * ww
    pair = row + np.abs(ref.turn(row, np.zeros(M), fr, inter)) + (row.max(-1, keepdims=True) if r else 0)
    within("y", y, want, (h + U) * np.abs(want) + ((d + 16) * U + ang) * pair)
    dz = np.abs(dyf) + (np.abs(dyf).max(-1, keepdims=True) if r else 0)  # bounds |dz|
    xh = np.abs(xf) * inv
    big = inv * (dz * ww + xh * (dz * ww * xh).mean(-1, keepdims=True)) if norm else dz
    within("dx", back["dx"], wdx, (h + U) * np.abs(wdx) + ((2 * d + 32) * U + 2 * ang) * big)
    if weight:
        within("dw", back["dw"], wdw, ((M * H + d + 32) * U + 2 * ang) * (dz * xh).sum((0, 1)))
    else:
        assert back["dw"] is None
    inplace = x.clone()
    gdn.norm_rope(inplace, *args, y=inplace, **kw)
    assert torch.equal(inplace, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,dl,dr,page,inter,norm", [(1, 8, 0, 1, False, True), (37, 128, 32, 16, False, True),
                                                     (300, 512, 64, 64, True, True), (65, 24, 8, 7, False, False),
                                                     (5, 72, 64, 3, True, False), (4500, 512, 64, 64, False, True),
                                                     (8300, 200, 16, 16, True, True)])
def test_write(n, dl, dr, page, inter, norm, dtype):
    say(f"cache write {n} {dl} {dr} {page} {dtype}")
    g, h = rng(7930), H16 if dtype == "bf16" else 0.0
    pages = -(-n // page) + 2
    c, cf = dev(g.standard_normal((n, dl)), dtype)
    kr, krf = dev(g.standard_normal((n, dr)), dtype) if dr else (None, None)
    w, wf = dev(1 + 0.1 * g.standard_normal(dl), "fp32") if norm else (None, None)
    pos, slots = g.integers(0, 1 << 20, n), g.permutation(pages * page)[:n]
    if n > 4:
        slots[:4] = [-1, pages * page, 2 ** 31 - 1, -(2 ** 31)]
    cache, before = dev(g.standard_normal((pages, page, dl + dr)), dtype)
    fr = 10000.0 ** (-np.arange(dr // 2) / max(dr // 2, 1)) if dr else None
    got = gdn.mla_write(c, kr, ints(slots), cache, w, ints(pos), torch.tensor(fr, device="cuda") if dr else None,
                        norm=norm, interleaved=inter)
    assert got is cache
    before = before.reshape(-1, dl + dr)
    want = ref.write(cf, krf, slots, before, wf, pos, fr, norm, 1e-6, inter)
    touched = np.zeros(len(before), bool)
    touched[slots[(slots >= 0) & (slots < len(before))]] = True
    assert (host(cache).reshape(-1, dl + dr)[~touched] == before[~touched]).all()
    bound = (h + U) * np.abs(want) + ((dl + 16) * U + 2.0 ** -21) * (np.abs(want) + np.abs(want).max(-1, keepdims=True)) * 2
    within("cache", cache.view(-1, dl + dr), want, np.where(touched[:, None], bound, 0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
def test_write_without_frequencies_copies_the_rotary_key(inter, dtype):
    """Infinities, NaN and negative zeros arrive as they are, beside any partner."""
    say(f"cache write without frequencies, non-finite columns, {dtype}")
    n, dl, dr = 9, 16, 8
    c, _ = dev(rng(7931).standard_normal((n, dl)), dtype)
    kr, _ = dev(rng(7932).standard_normal((n, dr)), dtype)
    inf = float("inf")
    for i, (col, x) in enumerate([(0, inf), (4, -inf), (7, float("nan")), (3, inf), (1, -0.0), (5, -0.0)]):
        kr[i, col] = x
    kr[6], kr[7, ::2] = inf, -inf
    cache = torch.zeros((3, 4, dl + dr), dtype=TYPES[dtype], device="cuda")
    slots = rng(7933).permutation(12)[:n]
    gdn.mla_write(c, kr, ints(slots), cache, interleaved=inter)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    got = cache.view(12, dl + dr)[torch.from_numpy(slots).cuda(), dl:].contiguous()
    assert torch.equal(got.view(bits), kr.view(bits))


def plan_inputs(seed, N, page, cols, most, free=None):
    g = rng(seed)
    F = N * cols + 1
    lens = g.integers(0, cols * page + 1, N)
    order, used = g.permutation(F), 0
    table = np.full((N, cols), -1)
    for i in range(N):
        k = -(-lens[i] // page)
        table[i, :k] = order[used:used + k]
        used += k
    stack = np.full(F, -1)
    stack[:F - used] = order[used:]
    new = np.where(g.random(N) < 0.2, -1, g.integers(0, most + 1, N))
    return lens, new, table, stack, F - used if free is None else min(free, F - used)


@pytest.mark.parametrize("seed,N,page,cols,most,free,cap", [
    (1, 1, 1, 1, 1, None, 1), (2, 7, 4, 5, 9, None, 40), (3, 7, 4, 5, 9, 3, 40), (4, 64, 16, 8, 40, None, 100),
    (5, 1024, 16, 4, 20, 500, 9000), (6, 1025, 3, 6, 7, None, 4096), (7, 2500, 5, 7, 3, 900, 4097),
    (8, 300, 64, 64, 3000, None, 300000), (9, 40, 1, 30, 30, 11, 0), (10, 3, 24, 9, 200, 0, 500)])
def test_page_plan(seed, N, page, cols, most, free, cap):
    say(f"page plan N {N} page {page} cols {cols} cap {cap}")
    lens, new, table, stack, n_free = plan_inputs(seed, N, page, cols, most, free)
    t = [ints(x) for x in (lens, new, table, stack, [n_free])]
    want = ref.page_plan(lens, new, table.astype(np.int32), stack.astype(np.int32), n_free, page, cap)
    for rep in range(2):  # with separate lens and n_free the same call gives the same again
        got = gdn.page_plan(*t, page, cap)
        for n, x in want.items():
            assert np.array_equal(got[n].cpu().numpy(), x), (rep, n)
    t = [ints(x) for x in (lens, new, table, stack, [n_free])]
    got = gdn.page_plan(*t, page, cap, lens_out=t[0], n_free_out=t[4])
    for n, x in want.items():
        assert np.array_equal(got[n].cpu().numpy(), x), ("in place", n)


def test_page_plan_without_sequences():
    e = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    got = gdn.page_plan(e(0), e(0), e(0, 3), ints([4, 5, 6, -1]), ints([3]), 8, 5)
    assert got["starts"].tolist() == [0] and got["n_free"].tolist() == [3]
    assert got["slots"].tolist() == [-1] * 5 and got["positions"].tolist() == [0] * 5


def test_page_plan_with_lengths_out_of_range():
    """Lengths outside the table and counts outside the stack are clamped."""
    lens, new = np.array([-4, 100, 3]), np.array([2, 1, 2 ** 31 - 1])
    table, stack = np.array([[-1, -1], [0, 1], [2, -1]], np.int32), np.array([3, 4, 5, 6, -1, -1, -1], np.int32)
    want = ref.page_plan(lens, new, table, stack, 4, 4, 9)
    got = gdn.page_plan(ints(lens), ints(new), ints(table), ints(stack), ints([4]), 4, 9)
    for n, x in want.items():
        assert np.array_equal(got[n].cpu().numpy(), x), n


def serve(x, W, dtype, ready, page=8):
    """The hybrid layer pair a token at a time: gated delta rule step, page
    plan, cache write, absorbed step. x [B,T,...] inputs; returns the outputs."""
    B, T = x["q"].shape[:2]
    ty, dl, dr, H = TYPES[dtype], W["c"], W["dr"], x["q"].shape[2]
    i32 = dict(dtype=torch.int32, device="cuda")
    cols = -(-T // page)
    table, lens = torch.full((B, cols), -1, **i32), torch.zeros(B, **i32)
    stack, n_free = torch.arange(B * cols, **i32).flip(0).contiguous(), torch.full((1,), B * cols, **i32)
    cache = torch.full((B * cols, page, dl + dr), float("nan"), dtype=ty, device="cuda")
    new, h, outs = torch.ones(B, **i32), None, []
    for t in range(T):
        g = {n: x["gdn"][n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")}
        y, h = gdn.step(g["q"], g["k"], g["v"], g["g"], g["beta"], x["A_log"], h)
        p = gdn.page_plan(lens, new, table, stack, n_free, page, B, lens_out=lens, n_free_out=n_free)
        gdn.mla_write(x["c"][:, t].contiguous(), x["kr"][:, t, 0].contiguous(), p["slots"], cache, x["wc"],
                      p["positions"], x["freqs"])
        qn = gdn.norm_rope(x["q"][:, t].contiguous(), x["wq"], p["positions"], x["freqs"])
        qa = torch.cat([torch.einsum("bhd,hdl->bhl", qn[..., :W["dn"]].float(), W["uk"]).to(ty), qn[..., W["dn"]:]], -1)
        o, _ = gdn.mla_step(qa.contiguous(), cache, table, lens, dl, scale=W["scale"])
        outs.append((y, torch.einsum("bhl,hdl->bhd", o.float(), W["uv"])))
        ready.append(p)
    return torch.stack([a for a, _ in outs], 1), torch.stack([b for _, b in outs], 1)


def test_prompt_and_token_by_token_agree():
    """The whole run as it is used: prompt through norm_rope, mla_fwd and the
    gated delta rule's forward; the same tokens one by one through page_plan,
    mla_write, norm_rope, mla_step and gdn.step. Both forms, in fp32, compute
    the same numbers."""
    say("hybrid layer pair: prompt against single tokens")
    B, T, H, dn, dr, dv, dl = 3, 37, 4, 16, 8, 16, 32
    g = rng(21)
    f = lambda *s: torch.tensor(g.standard_normal(s), dtype=torch.float32, device="cuda")  # noqa: E731
    x = {"q": f(B, T, H, dn + dr), "c": f(B, T, dl), "kr": f(B, T, 1, dr), "wq": 1 + 0.1 * f(dn + dr),
         "wc": 1 + 0.1 * f(dl), "freqs": torch.tensor(100.0 ** (-np.arange(dr // 2) / 4), device="cuda"),
         "A_log": 0.1 * f(H),
         "gdn": {"q": f(B, T, H, 16), "k": torch.nn.functional.normalize(f(B, T, H, 16), dim=-1), "v": f(B, T, H, 16),
                 "g": torch.sigmoid(f(B, T, H)), "beta": torch.sigmoid(f(B, T, H))}}
    W = {"uk": f(H, dn, dl) / dl ** 0.5, "uv": f(H, dv, dl) / dl ** 0.5, "c": dl, "dr": dr, "dn": dn,
         "scale": (dn + dr) ** -0.5}
    pos = ints(np.tile(np.arange(T), (B, 1)))
    cn = gdn.norm_rope(x["c"][:, :, None].contiguous(), x["wc"])[:, :, 0]
    k, v = (torch.einsum("btl,hdl->bthd", cn, W[n]).contiguous() for n in ("uk", "uv"))
    kr = gdn.norm_rope(x["kr"], None, pos, x["freqs"], norm=False)
    o, _ = gdn.mla_fwd(gdn.norm_rope(x["q"], x["wq"], pos, x["freqs"]), k, v, kr, scale=W["scale"])
    d = x["gdn"]
    y, _, _ = gdn.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], x["A_log"])
    plans = []
    y1, o1 = serve(x, W, "fp32", plans)
    assert plans[-1]["lens"].tolist() == [T] * B
    # both within fp32 rounding of sums of ~100 terms of size 1 (2^-24 * 100 = 6e-6), an order to spare
    assert (o - o1).abs().max() <= 1e-4 * o.abs().max()
    assert (y - y1).abs().max() <= 1e-4 * y.abs().max()


def graph_of(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()  # (library and allocator warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


def test_graphs_replay_what_the_eager_calls_compute():
    """Attention forward and backward, and the decode chain (plan, write,
    norm, step), captured; replayed with new inputs in between eager calls."""
    say("captured attention and decode chain, three replays each")
    case = (2, 100, 0, 4, 2, 1, 56, 32, 56, [100, 61])
    t, _, lens, scale = attn_inputs(case, "bf16", 7940)
    g, out = graph_of(lambda: run_attn(t, lens, scale))
    N, page, cols, dl, dr = 5, 8, 6, 64, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    table, cache = torch.full((N, cols), -1, **i32), torch.zeros((N * cols, page, dl + dr), device="cuda")
    stack, n_free = torch.arange(N * cols, **i32), torch.full((1,), N * cols, **i32)
    lens_d, new = torch.zeros(N, **i32), torch.full((N,), 3, **i32)
    c, kr, q = torch.randn(N * 3, dl, device="cuda"), torch.randn(N * 3, dr, device="cuda"), torch.randn(
        N, 3, 4, dl + dr, device="cuda")
    fr = torch.tensor([1.0, 0.5, 0.2, 0.1, 0.05, 0.02, 0.01, 0.005], dtype=torch.float64, device="cuda")

    def decode(lo, nf):
        p = gdn.page_plan(lens_d, new, table, stack, n_free, page, N * 3, lens_out=lo, n_free_out=nf)
        gdn.mla_write(c, kr, p["slots"], cache, None, p["positions"], fr)
        return gdn.mla_step(q, cache, table, p["lens"], dl, scale=0.1) + (p["lens"], p["n_free"])

    g2, out2 = graph_of(lambda: decode(None, None))
    for rep in range(3):
        for x in t:
            x.copy_(torch.randn_like(x))
        for x in (c, kr, q):
            x.copy_(torch.randn_like(x))
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        eager, eager2 = run_attn(t, lens, scale), decode(None, None)
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(out[n], eager[n]), (rep, n)
        for a, b in zip(out2, eager2):
            assert torch.equal(a, b), rep
        decode(lens_d, n_free)  # the sequences grow for the next replay
    assert lens_d.tolist() == [9] * N


def test_calls_run_on_the_current_stream():
    """Work queued behind a slow kernel on a side stream sees its results."""
    say("attention and step on a side stream behind pending writes")
    case = (1, 64, 0, 2, 2, 1, 16, 8, 16, None)
    t, _, lens, scale = attn_inputs(case, "bf16", 7950)
    want = run_attn(t, lens, scale)
    late = [torch.zeros_like(x) for x in t]
    big = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            big = big @ big * 1e-3
        for a, b in zip(late, t):
            a.copy_(b)
        got = run_attn(late, lens, scale)
    s.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_two_calls_at_once():
    """Attention and paged steps on two streams at the same time, each with its own workspace."""
    say("attention and step on two streams at once")
    t, _, lens, scale = attn_inputs((2, 700, 0, 8, 4, 2, 56, 32, 56, [700, 333]), "bf16", 7951)
    q, qf, c, cf, table, sc = paged((9, 1, 16, 128, 32, 64, 40, [2000, 5, 0, 800, 64, 65, 1, 2559, 7]), "bf16", 7952)
    ln = ints([2000, 5, 0, 800, 64, 65, 1, 2559, 7])
    table = ints(table)

    def both():
        return run_attn(t, lens, scale), gdn.mla_step(q, c, table, ln, 128, scale=sc)

    want = both()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for s, out in zip(streams, got):
            with torch.cuda.stream(s):
                out.append(both())
    torch.cuda.synchronize()
    for r, (o, lse) in got[0] + got[1]:
        for n in want[0]:
            assert torch.equal(r[n], want[0][n]), n
        assert torch.equal(o, want[1][0]) and torch.equal(lse, want[1][1])


def test_autograd_with_broadcast_gradients_and_once():
    """The gradient of a plain sum arrives broadcast; a second derivative is refused."""
    say("autograd: sum, second derivative")
    t, _, _, scale = attn_inputs((1, 33, 0, 2, 1, 1, 16, 8, 16, None), "fp32", 7953)
    q, k, kr, v = (x.requires_grad_() for x in t[:4])
    gdn.LatentAttention.apply(q, k, v, kr, None, scale).sum().backward()
    want = run_attn([q.detach(), k.detach(), kr.detach(), v.detach(), torch.ones_like(t[4])], None, scale)
    for x, n in ((q, "dq"), (k, "dk"), (kr, "dkr"), (v, "dv")):
        assert torch.equal(x.grad, want[n]), n
    g, = torch.autograd.grad(gdn.LatentAttention.apply(q, k, v, kr, None, scale).square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_launches_are_bracketed():
    """The timing aid names and times every new kernel."""
    say("launch timer over the new calls")
    t, _, lens, scale = attn_inputs((1, 80, 0, 4, 2, 1, 16, 8, 16, None), "bf16", 7960)
    q, qf, c, cf, table, sc = paged((2, 1, 4, 64, 8, 8, 40, [300, 5]), "bf16", 7961)
    x, w = torch.randn(4, 2, 16, device="cuda"), torch.ones(16, device="cuda")
    with gdn.LaunchTimer(16) as lt:
        run_attn(t, lens, scale)
        gdn.mla_step(q, c, ints(table), ints([300, 5]), 64, scale=sc)
        gdn.norm_rope_bwd(gdn.norm_rope(x, w), x, w)
    assert lt.kinds() == ["mla_fwd", "mla_bwd_q", "mla_bwd_k", "mla_rope_sum", "mla_step", "mla_join", "norm_rope",
                          "norm_rope_bwd", "norm_sum"]
    assert all(ms > 0 for ms in lt.durations_ms())


def test_refusals_on_the_device():
    say("refusals with device tensors")
    q = torch.zeros(1, 4, 2, 24, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16, device="cuda")
    kr = torch.zeros(1, 4, 1, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gdn.mla_fwd(q.transpose(1, 2), k, k, kr)
    with pytest.raises(TypeError):
        gdn.mla_fwd(q.half(), k.half(), k.half(), kr.half())
    with pytest.raises(TypeError):
        gdn.mla_fwd(q, k, k, kr, torch.tensor([4], device="cuda"))  # int64 lengths
    with pytest.raises(gdn.GdnError) as e:
        gdn.mla_fwd(q, k, k, kr, scale=-1.0)
    assert e.value.status == 1
    with pytest.raises(gdn.GdnError) as e:
        gdn.mla_fwd(torch.zeros(1, 4, 2, 12, dtype=torch.bfloat16, device="cuda"), k[..., :12].contiguous(), k)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        gdn.norm_rope(q, None, None, torch.ones(4, dtype=torch.float64, device="cuda"))


def test_more_turned_columns_than_int32_holds_are_refused():
    """(2^32 + 8 turned columns would have been taken for eight.)"""
    x, pos = torch.zeros(3, 2, 16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    far = torch.ones(1, dtype=torch.float64, device="cuda").expand(2 ** 31 + 4)
    with pytest.raises(ValueError, match="too large"):
        gdn.norm_rope(x, None, pos, far)
