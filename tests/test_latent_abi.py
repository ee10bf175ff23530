"""Argument checks of the latent-attention and paged-cache entry points: every
call here returns before a device is touched."""
import ctypes

import pytest
import torch

import gated_delta_rule_74_amd as gdn
from test_abi import EINVAL, EUNSUPPORTED, EWORKSPACE, L, fake  # noqa: F401

NAN = float("nan")


def mla(**over):
    d = dict(B=2, Tq=9, Tk=9, H=4, Hk=2, Hr=1, dn=16, dr=8, dv=16, dtype=1, scale=0.2)
    d.update(over)
    return gdn.MlaShape(*[d[n] for n, _ in gdn.MlaShape._fields_])


def fwd(L, s, **over):  # noqa: F811
    a = dict(q=fake(1), k=fake(2), kr=fake(3), v=fake(4), lens=None, o=fake(5), lse=fake(6))
    a.update(over)
    return L.gdn_mla_fwd(ctypes.byref(s), a["q"], a["k"], a["kr"], a["v"], a["lens"], a["o"], a["lse"], None)


def bwd(L, s, ws=fake(20), ws_bytes=1 << 20, **over):  # noqa: F811
    a = dict(q=fake(1), k=fake(2), kr=fake(3), v=fake(4), lens=None, o=fake(5), lse=fake(6), do=fake(7), dq=fake(8),
             dk=fake(9), dkr=fake(10), dv=fake(11))
    a.update(over)
    return L.gdn_mla_bwd(ctypes.byref(s), *[a[n] for n in ("q", "k", "kr", "v", "lens", "o", "lse", "do", "dq", "dk",
                                                           "dkr", "dv")], ws, ws_bytes, None)


BAD_MLA = [("B", 0, EINVAL), ("H", 0, EINVAL), ("Hk", 0, EINVAL), ("Hk", 3, EINVAL), ("Hr", 3, EINVAL),
           ("Hr", 0, EINVAL), ("Tq", -1, EINVAL), ("Tq", 10, EINVAL), ("dn", 0, EINVAL), ("dn", 12, EUNSUPPORTED),
           ("dn", 136, EUNSUPPORTED), ("dr", -8, EINVAL), ("dr", 72, EUNSUPPORTED), ("dr", 4, EUNSUPPORTED),
           ("dv", 136, EUNSUPPORTED), ("dv", 0, EINVAL), ("dtype", 2, EINVAL), ("scale", 0.0, EINVAL),
           ("scale", -1.0, EINVAL), ("scale", NAN, EINVAL), ("scale", float("inf"), EINVAL), ("Tk", 1 << 30, EINVAL)]


@pytest.mark.parametrize("key,val,code", BAD_MLA)
def test_attention_rejects_bad_shapes(L, key, val, code):  # noqa: F811
    s = mla(**{key: val})
    assert fwd(L, s) == code and L.gdn_last_error_detail()
    assert bwd(L, s) == code
    assert L.gdn_mla_bwd_workspace_size(ctypes.byref(s)) == 0


def test_attention_is_limited_by_its_tensors(L):  # noqa: F811
    """Few key heads and few queries beside many keys: what counts is what each tensor holds."""
    size = lambda s: L.gdn_mla_bwd_workspace_size(ctypes.byref(s))  # noqa: E731
    chunk = dict(B=1, Tq=512, Tk=131584, H=128, Hk=16, Hr=1, dn=128, dr=64, dv=128)
    assert size(mla(**chunk)) >= 4 * 128 * 512
    assert size(mla(**{**chunk, "Tq": 1, "Tk": (1 << 20) - 1})) > 0
    # one tensor at a time at its limit: q, o, k, k_rope, v
    wide, tall = dict(B=1, H=256, Hk=256, Hr=1), dict(B=1, Tq=1, H=256, Hk=256, Hr=256)
    for n, s in (("q", dict(wide, Tq=1 << 16, Tk=1 << 16, Hk=1, dn=64, dr=64, dv=8)),
                 ("o", dict(wide, Tq=1 << 16, Tk=1 << 16, Hk=1, dn=8, dr=0, dv=128)),
                 ("k", dict(tall, Tk=1 << 16, dn=128, dr=0, dv=8)), ("v", dict(tall, Tk=1 << 16, dn=8, dr=0, dv=128)),
                 ("k_rope", dict(tall, Tk=1 << 17, dn=8, dr=64, dv=8))):
        assert size(mla(**s)) == 0 and b"too large" in L.gdn_last_error_detail(), n
        fewer = {k: s[k] - 1 for k in ("Tq", "Tk") if s.get(k, 0) > 1}
        assert size(mla(**{**s, **fewer})) > 0, n
    # more heads than a launch has workgroups
    assert size(mla(B=1 << 20, H=16, Hk=16, Tq=1, Tk=1, dn=8, dr=0, dv=8)) == 0


def test_step_refuses_more_workgroups_than_a_launch_holds(L):  # noqa: F811
    for shape in (dict(N=1 << 24, S=1, H=1), dict(N=1, S=1 << 23, H=8)):
        s = gdn.MlaStepShape(shape["N"], shape["S"], shape["H"], 16, 0, 1, 10, 4, 5, 0.1)
        assert L.gdn_mla_step_workspace_size(ctypes.byref(s)) == 0
        assert b"launch" in L.gdn_last_error_detail()


def test_attention_rejects_null_misaligned_aliased_and_small_workspaces(L):  # noqa: F811
    s = mla()
    need = L.gdn_mla_bwd_workspace_size(ctypes.byref(s))
    assert need >= 4 * (2 * 4 * 9 + 2 * 9 * 2 * 8)
    assert L.gdn_mla_fwd(None, *[None] * 8) == EINVAL
    for n in ("q", "k", "kr", "v", "o"):
        assert fwd(L, s, **{n: None}) == EINVAL
    assert fwd(L, s, q=ctypes.c_void_p(fake(1).value + 2)) == EINVAL
    assert fwd(L, s, lens=ctypes.c_void_p(fake(9).value + 2)) == EINVAL
    assert fwd(L, s, o=fake(4)) == EINVAL and b"overlaps" in L.gdn_last_error_detail()
    assert fwd(L, s, lse=fake(5)) == EINVAL
    for n in ("lse", "o", "do", "dq", "dk", "dkr", "dv"):
        assert bwd(L, s, **{n: None}) == EINVAL
    assert bwd(L, s, dq=fake(1)) == EINVAL and bwd(L, s, dk=fake(8)) == EINVAL and bwd(L, s, dv=fake(20)) == EINVAL
    assert bwd(L, s, ws=None) == EWORKSPACE and bwd(L, s, ws_bytes=need - 1) == EWORKSPACE
    assert bwd(L, s, ws=ctypes.c_void_p(fake(20).value + 16)) == EINVAL
    empty = mla(Tq=0)  # no query: nothing to launch
    assert fwd(L, empty, q=None, k=None, v=None, kr=None, o=None, lse=None) == 0


def step(L, ws=None, ws_bytes=0, over=None, **shape):  # noqa: F811
    d = dict(N=3, S=1, H=4, dl=32, dr=8, dtype=1, pages=10, page_size=4, max_pages=5, scale=0.1)
    d.update(shape)
    s = gdn.MlaStepShape(*[d[n] for n, _ in gdn.MlaStepShape._fields_])
    a = dict(q=fake(1), cache=fake(2), table=fake(3), lens=fake(4), o=fake(5), lse=fake(6))
    a.update(over or {})
    return L.gdn_mla_step(ctypes.byref(s), *[a[n] for n in ("q", "cache", "table", "lens", "o", "lse")], ws, ws_bytes,
                          None)


@pytest.mark.parametrize("key,val,code", [
    ("N", -1, EINVAL), ("S", -1, EINVAL), ("H", 0, EINVAL), ("dl", 0, EINVAL), ("dl", 24, EUNSUPPORTED),
    ("dl", 528, EUNSUPPORTED), ("dr", -8, EINVAL), ("dr", 4, EUNSUPPORTED), ("dr", 72, EUNSUPPORTED),
    ("dtype", 5, EINVAL), ("pages", 0, EINVAL), ("page_size", 0, EINVAL), ("max_pages", 0, EINVAL),
    ("pages", 1 << 30, EINVAL), ("max_pages", 1 << 30, EINVAL), ("scale", 0.0, EINVAL), ("scale", NAN, EINVAL)])
def test_step_rejects_bad_shapes(L, key, val, code):  # noqa: F811
    assert step(L, **{key: val}) == code


def test_step_rejects_bad_buffers(L):  # noqa: F811
    for n in ("q", "cache", "table", "lens", "o"):
        assert step(L, over={n: None}) == EINVAL
    assert step(L, over={"o": fake(2)}) == EINVAL and step(L, over={"lse": fake(5)}) == EINVAL
    assert step(L, over={"cache": ctypes.c_void_p(fake(2).value + 8)}) == EINVAL
    assert step(L, max_pages=1000) == EWORKSPACE  # long enough to be split
    assert step(L, max_pages=1000, ws=fake(20), ws_bytes=16) == EWORKSPACE
    assert step(L, max_pages=1000, ws=ctypes.c_void_p(fake(20).value + 4), ws_bytes=1 << 29) == EINVAL
    none = dict.fromkeys(("q", "cache", "table", "lens", "o", "lse"))
    assert step(L, N=0, over=none) == 0 and step(L, S=0, over=none) == 0


def test_sizes_next_to_int32_are_refused(L):  # noqa: F811
    """Positions are looked up a few tiles ahead, in int32: a context next to 2^31 would wrap there."""
    ok = dict(N=1, H=1)
    for page, cols, code in ((1024, 2 ** 21 - 2, EWORKSPACE), (1024, 2 ** 21 - 1, EINVAL)):
        assert step(L, max_pages=cols, page_size=page, **ok) == code, cols
        s = gdn.MlaStepShape(1, 1, 1, 32, 8, 1, 10, page, cols, 0.1)
        assert (L.gdn_mla_step_workspace_size(ctypes.byref(s)) > 0) == (code == EWORKSPACE)
    far = [ctypes.c_void_p((i + 1) << 40) for i in range(11)]  # (no two of them overlap)
    for cols in (2 ** 31 - 1, 2 ** 31 - 2047):
        assert L.gdn_page_plan(1, cols, 20, 16, 64, *far, None) == EINVAL
        assert b"too large" in L.gdn_last_error_detail()


def test_norm_rope_validation(L):  # noqa: F811
    def call(M=4, H=2, d=16, r=8, dtype=1, flags=1, eps=1e-6, x=fake(1), w=fake(2), pos=fake(3), fr=fake(4), y=fake(5)):
        return L.gdn_norm_rope(M, H, d, r, dtype, flags, eps, x, w, pos, fr, y, None)

    for bad in (dict(M=-1), dict(H=0), dict(d=0), dict(r=7), dict(r=18), dict(r=-2), dict(dtype=3), dict(flags=4),
                dict(eps=0.0), dict(eps=NAN), dict(x=None), dict(y=None), dict(pos=None), dict(fr=None),
                dict(flags=0), dict(M=1 << 30), dict(y=ctypes.c_void_p(fake(1).value + 16)), dict(y=fake(2)),
                dict(x=ctypes.c_void_p(fake(1).value + 8)), dict(fr=ctypes.c_void_p(fake(4).value + 4))):
        assert call(**bad) == EINVAL, bad
    assert call(d=520) == EUNSUPPORTED
    assert call(M=0, x=None, y=None, pos=None, fr=None) == 0

    def back(M=4, H=2, d=16, r=8, flags=1, dy=fake(1), x=fake(2), w=fake(3), dx=fake(6), dw=fake(7), ws=fake(20),
             n=1 << 20):
        return L.gdn_norm_rope_bwd(M, H, d, r, 1, flags, 1e-6, dy, x, w, fake(4), fake(5), dx, dw, ws, n, None)

    for bad in (dict(dy=None), dict(x=None), dict(dx=None), dict(flags=0), dict(dx=fake(1)), dict(dw=fake(3)),
                dict(ws=ctypes.c_void_p(fake(20).value + 4))):
        assert back(**bad) == EINVAL, bad
    assert back(ws=None) == EWORKSPACE and back(n=8) == EWORKSPACE
    assert back(M=0, dy=None, x=None, dx=None, dw=None, ws=None) == 0


def test_write_validation(L):  # noqa: F811
    def call(n=4, dl=16, dr=8, dtype=1, flags=1, eps=1e-6, c=fake(1), kr=fake(2), w=fake(3), pos=fake(4), fr=fake(5),
             slots=fake(6), cache=fake(7), n_slots=100):
        return L.gdn_mla_write(n, dl, dr, dtype, flags, eps, c, kr, w, pos, fr, slots, cache, n_slots, None)

    for bad in (dict(n=-1), dict(dl=0), dict(dr=-8), dict(dtype=9), dict(flags=4), dict(eps=0.0), dict(flags=0),
                dict(n_slots=-1), dict(n_slots=1 << 31), dict(c=None), dict(kr=None), dict(slots=None),
                dict(cache=None), dict(pos=None), dict(cache=fake(1)), dict(c=ctypes.c_void_p(fake(1).value + 4))):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dl=12), dict(dl=520), dict(dr=12), dict(dr=72)):
        assert call(**bad) == EUNSUPPORTED, bad
    assert call(n=0, c=None, kr=None, slots=None) == 0 and call(n_slots=0) == 0


def test_page_plan_validation(L):  # noqa: F811
    names = ("lens", "new", "table", "stack", "n_free", "lens_out", "n_free_out", "granted", "starts", "slots", "pos")

    def call(N=4, cols=5, F=20, page=16, cap=64, **over):
        a = {n: fake(i + 1) for i, n in enumerate(names)}
        a.update(over)
        return L.gdn_page_plan(N, cols, F, page, cap, *[a[n] for n in names], None)

    for bad in (dict(N=-1), dict(cols=0), dict(F=0), dict(page=0), dict(cap=-1), dict(N=1 << 20, cols=1 << 12),
                dict(granted=fake(9)), dict(slots=fake(3)), dict(lens_out=fake(2)), dict(n_free_out=fake(1)),
                dict(lens_out=ctypes.c_void_p(fake(1).value + 4)), dict(table=ctypes.c_void_p(fake(3).value + 2))):
        assert call(**bad) == EINVAL, bad
    for n in names:
        assert call(**{n: None}) == EINVAL, n


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q, k = torch.zeros(1, 3, 2, 24), torch.zeros(1, 3, 2, 16)
    with pytest.raises(ValueError):
        gdn.mla_fwd(q, k, k)  # q wider than k, no rotary key
    with pytest.raises(ValueError):
        gdn.mla_fwd(q[..., :16], k, k)  # host tensors
    with pytest.raises(ValueError):
        gdn.mla_fwd(q[0], k, k)
    with pytest.raises(ValueError):
        gdn.mla_step(torch.zeros(2, 3), torch.zeros(4, 2, 24), torch.zeros(2, 2, dtype=torch.int32),
                     torch.zeros(2, dtype=torch.int32), 16, scale=1.0)
    with pytest.raises(ValueError):
        gdn.norm_rope(torch.zeros(3, 2, 8), torch.zeros(8), norm=False)
    with pytest.raises(ValueError):
        gdn.norm_rope(torch.zeros(3))
    with pytest.raises(ValueError):
        gdn.mla_write(torch.zeros(3, 16), None, torch.zeros(3), torch.zeros(4, 2, 24))
    with pytest.raises(ValueError):
        gdn.page_plan(*[torch.zeros(3)] * 2, torch.zeros(3), torch.zeros(3), torch.zeros(1), 4, 8)


def test_binding_refuses_what_int32_does_not_hold_and_missing_tensors():
    i32 = dict(dtype=torch.int32)
    plan = [torch.zeros(3, **i32), torch.zeros(3, **i32), torch.zeros(3, 2, **i32), torch.zeros(6, **i32),
            torch.zeros(1, **i32)]
    for page, cap in ((2 ** 32 + 4, 8), (4, 2 ** 32 + 8), (4, -1), (0, 2 ** 31)):
        with pytest.raises(ValueError):
            gdn.page_plan(*plan, page, cap)
    for k in range(5):
        with pytest.raises(ValueError):
            gdn.page_plan(*[None if i == k else t for i, t in enumerate(plan)], 4, 8)
    wide = torch.zeros(1, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="too large"):
        gdn.norm_rope(wide.expand(1, 2 ** 32 + 8))
    long = wide.expand(1, 2 ** 32 + 64, 1, 8)
    with pytest.raises(ValueError, match="too large"):
        gdn.mla_fwd(wide.expand(1, 64, 1, 8), long, long)
    with pytest.raises(ValueError, match="too large"):
        gdn.mla_step(wide.expand(1, 1, 24), wide.expand(2 ** 32 + 1, 2, 24), torch.zeros(1, 2, **i32),
                     torch.zeros(1, **i32), 16, scale=1.0)
    with pytest.raises(ValueError, match="too large"):
        gdn.mla_write(wide.expand(1, 2 ** 32 + 8), None, torch.zeros(1, **i32), wide.expand(1, 1, 2 ** 32 + 8))
    empty = torch.zeros(1, 3, 2, 0)
    with pytest.raises(ValueError):
        gdn.mla_fwd(empty, empty, empty)
    with pytest.raises(ValueError):
        gdn.mla_step(torch.zeros(1, 1, 24), torch.zeros(1, 2, 24), torch.zeros(1, 2, **i32), None, 16, scale=1.0)
    with pytest.raises(ValueError):
        gdn.mla_write(torch.zeros(1, 16), None, None, torch.zeros(1, 2, 16))


def test_binding_refuses_more_rotary_heads_than_int32_holds():
    """(2^32 + 1 rotary heads would have been taken for one.)"""
    wide = torch.zeros(1, dtype=torch.bfloat16)
    q, k = torch.zeros(1, 1, 2, 24, dtype=torch.bfloat16), torch.zeros(1, 1, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="too large"):
        gdn.mla_fwd(q, k, k, wide.expand(1, 1, 2 ** 32 + 1, 8))
