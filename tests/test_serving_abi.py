"""Argument checks of the serving operators beside the plain step: every call
here returns before a device is touched."""
import ctypes

import pytest
import torch

import gated_delta_rule_74_amd as gdn
from test_abi import EINVAL, EUNSUPPORTED, EWORKSPACE, L, fake  # noqa: F401

NAN = float("nan")


def off(i, by):
    return ctypes.c_void_p(fake(i).value + by)


def paged(**over):
    d = dict(N=3, S=1, H=4, dl=32, dr=8, dtype=1, pages=10, page_size=4, max_pages=5, scale=0.1)
    d.update(over)
    return gdn.MlaStepShape(*[d[n] for n, _ in gdn.MlaStepShape._fields_])


BAD_PAGED = [("N", -1, EINVAL), ("S", -1, EINVAL), ("H", 0, EINVAL), ("dl", 0, EINVAL), ("dl", 24, EUNSUPPORTED),
             ("dl", 528, EUNSUPPORTED), ("dr", -8, EINVAL), ("dr", 4, EUNSUPPORTED), ("dtype", 5, EINVAL),
             ("pages", 0, EINVAL), ("page_size", 0, EINVAL), ("max_pages", 0, EINVAL), ("max_pages", 1 << 30, EINVAL),
             ("scale", 0.0, EINVAL), ("scale", NAN, EINVAL)]


def shared(L, s=None, G=2, cols=3, ws=fake(20), ws_bytes=1 << 30, **over):  # noqa: F811
    s = paged() if s is None else s
    a = dict(q=fake(1), cache=fake(2), table=fake(3), lens=fake(4), pt=fake(5), pl=fake(6), starts=fake(7), o=fake(8),
             lse=fake(9))
    a.update(over)
    return L.gdn_mla_step_shared(ctypes.byref(s), G, cols, *[a[n] for n in ("q", "cache", "table", "lens", "pt", "pl",
                                                                            "starts", "o", "lse")], ws, ws_bytes, None)


@pytest.mark.parametrize("key,val,code", BAD_PAGED)
def test_shared_and_weights_reject_bad_shapes(L, key, val, code):  # noqa: F811
    s = paged(**{key: val})
    assert shared(L, s) == code and L.gdn_last_error_detail()
    assert L.gdn_mla_step_shared_workspace_size(ctypes.byref(s), 2, 3) == 0
    assert weigh(L, s) == code


def test_shared_rejects_bad_prefixes_and_buffers(L):  # noqa: F811
    assert shared(L, G=-1) == EINVAL and shared(L, cols=0) == EINVAL and shared(L, cols=1 << 30) == EINVAL
    assert shared(L, G=1 << 20, cols=1 << 11) == EINVAL
    for n in ("q", "cache", "table", "lens", "pt", "pl", "starts", "o"):
        assert shared(L, **{n: None}) == EINVAL, n
    assert shared(L, o=fake(2)) == EINVAL and b"overlaps" in L.gdn_last_error_detail()
    assert shared(L, lse=fake(8)) == EINVAL and shared(L, cache=off(2, 8)) == EINVAL and shared(L, starts=off(7, 2)) == EINVAL
    s = paged()
    need = L.gdn_mla_step_shared_workspace_size(ctypes.byref(s), 2, 3)
    assert need > 0
    assert shared(L, ws=None) == EWORKSPACE and shared(L, ws_bytes=need - 1) == EWORKSPACE
    assert shared(L, ws=off(20, 16)) == EINVAL and shared(L, o=fake(20)) == EINVAL
    # nothing to do: no token, and no prefix means the plain step
    none = {n: None for n in ("q", "cache", "table", "lens", "pt", "pl", "starts", "o", "lse")}
    assert shared(L, paged(N=0), ws=None, ws_bytes=0, **none) == 0
    assert shared(L, paged(S=0), ws=None, ws_bytes=0, **none) == 0
    assert L.gdn_mla_step_shared_workspace_size(ctypes.byref(s), 0, 0) == L.gdn_mla_step_workspace_size(ctypes.byref(s))
    assert shared(L, G=0, cols=0, ws=None, ws_bytes=0) in (EWORKSPACE,)


def weigh(L, s=None, decay=1.0, **over):  # noqa: F811
    s = paged() if s is None else s
    a = dict(q=fake(1), cache=fake(2), table=fake(3), lens=fake(4), lse=fake(5), known=None, w=fake(6))
    a.update(over)
    return L.gdn_mla_weights(ctypes.byref(s), decay, *[a[n] for n in ("q", "cache", "table", "lens", "lse", "known",
                                                                      "w")], None)


def test_weights_reject_bad_arguments(L):  # noqa: F811
    for decay in (-0.1, 1.1, NAN):
        assert weigh(L, decay=decay) == EINVAL
    for n in ("q", "cache", "table", "lens", "lse", "w"):
        assert weigh(L, **{n: None}) == EINVAL, n
    assert weigh(L, w=fake(2)) == EINVAL and weigh(L, w=off(6, 2)) == EINVAL and weigh(L, q=off(1, 8)) == EINVAL
    assert weigh(L, paged(N=0), q=None, cache=None, table=None, lens=None, lse=None, w=None) == 0


def evict(L, ws=fake(20), ws_bytes=1 << 30, **over):  # noqa: F811
    a = dict(N=3, cols=5, pages=10, page=4, row=320, first=1, recent=2, table=fake(1), lens=fake(2), keep=fake(3),
             w=fake(4), cache=fake(5), out=fake(6))
    a.update(over)
    return L.gdn_mla_evict(*[a[n] for n in ("N", "cols", "pages", "page", "row", "first", "recent", "table", "lens",
                                            "keep", "w", "cache", "out")], ws, ws_bytes, None)


def test_eviction_rejects_bad_arguments(L):  # noqa: F811
    for over, code in ((dict(N=-1), EINVAL), (dict(cols=0), EINVAL), (dict(pages=0), EINVAL), (dict(page=0), EINVAL),
                       (dict(row=0), EINVAL), (dict(row=24), EINVAL), (dict(row=2320), EUNSUPPORTED),
                       (dict(first=-1), EINVAL), (dict(recent=-1), EINVAL), (dict(cols=1 << 30), EINVAL),
                       (dict(pages=1 << 30), EINVAL), (dict(N=1 << 22, cols=256), EINVAL)):
        assert evict(L, **over) == code, over
    for n in ("table", "lens", "keep", "w", "cache", "out"):
        assert evict(L, **{n: None}) == EINVAL, n
    assert evict(L, out=fake(2)) == EINVAL and evict(L, cache=fake(4)) == EINVAL and evict(L, cache=off(5, 8)) == EINVAL
    need = L.gdn_mla_evict_workspace_size(3, 5, 4, 320)
    assert need > 0 and L.gdn_mla_evict_workspace_size(3, 5, 4, 24) == 0
    assert evict(L, ws=None) == EWORKSPACE and evict(L, ws_bytes=need - 1) == EWORKSPACE and evict(L, ws=off(20, 16)) == EINVAL
    assert evict(L, N=0, table=None, lens=None, keep=None, w=None, cache=None, out=None, ws=None, ws_bytes=0) == 0


def test_eviction_rejects_tables_that_hold_nearly_2_31_rows(L):  # noqa: F811
    """Such a sequence's chunks of 8192 rows cannot be counted in int32 (the last one's end passes it)."""
    for cols, page in ((2 ** 31 - 2048, 1), ((2 ** 31 - 4096) // 64, 64), ((2 ** 31 - 8128) // 64, 64)):
        assert L.gdn_mla_evict_workspace_size(1, cols, page, 16) == 0, (cols, page)
        assert evict(L, N=1, cols=cols, pages=10, page=page, row=16, ws_bytes=1 << 40) == EINVAL, (cols, page)
        assert b"table" in L.gdn_last_error_detail()
    assert L.gdn_mla_evict_workspace_size(1, (2 ** 31 - 8192) // 64, 64, 16) > 0


def trim(L, **over):  # noqa: F811
    a = dict(N=3, cols=5, F=10, page=4, lens=fake(1), new=fake(2), table=fake(3), stack=fake(4), free=fake(5), out=fake(6))
    a.update(over)
    return L.gdn_page_trim(*[a[n] for n in ("N", "cols", "F", "page", "lens", "new", "table", "stack", "free", "out")], None)


def test_page_trim_rejects_bad_arguments(L):  # noqa: F811
    for over in (dict(N=-1), dict(cols=0), dict(F=0), dict(page=0), dict(N=1 << 20, cols=1 << 11)):
        assert trim(L, **over) == EINVAL, over
    for n in ("lens", "new", "table", "stack", "free", "out"):
        assert trim(L, **{n: None}) == EINVAL, n
    assert trim(L, stack=fake(3)) == EINVAL and trim(L, out=fake(1)) == EINVAL and trim(L, lens=off(1, 1)) == EINVAL


def verify(L, ws=fake(20), ws_bytes=1 << 30, **over):  # noqa: F811
    a = dict(N=3, S=2, V=100, dtype=1, z=fake(1), draft=fake(2), lens=None, zq=fake(3), temp=None, u=fake(4), acc=fake(5),
             tok=fake(6), lp=fake(7))
    a.update(over)
    return L.gdn_draft_verify(*[a[n] for n in ("N", "S", "V", "dtype", "z", "draft", "lens", "zq", "temp", "u", "acc",
                                               "tok", "lp")], ws, ws_bytes, None)


def test_verification_rejects_bad_arguments(L):  # noqa: F811
    for over in (dict(N=-1), dict(S=-1), dict(V=0), dict(dtype=2), dict(N=1 << 16, V=1 << 14), dict(V=(1 << 30) + 1, N=1, S=0),
                 dict(S=2 ** 31 - 1, N=1, V=1)):
        assert verify(L, **over) == EINVAL, over
        assert L.gdn_draft_verify_workspace_size(over.get("N", 3), over.get("S", 2), over.get("V", 100),
                                                 over.get("dtype", 1)) == 0
    for n in ("z", "draft", "u", "acc", "tok"):
        assert verify(L, **{n: None}) == EINVAL, n
    assert verify(L, tok=fake(1)) == EINVAL and verify(L, lp=fake(6)) == EINVAL and verify(L, u=off(4, 2)) == EINVAL
    need = L.gdn_draft_verify_workspace_size(3, 2, 100, 1)
    assert verify(L, ws=None) == EWORKSPACE and verify(L, ws_bytes=need - 1) == EWORKSPACE
    assert verify(L, ws=off(20, 16)) == EINVAL and verify(L, acc=fake(20)) == EINVAL
    assert verify(L, N=0, z=None, draft=None, zq=None, u=None, acc=None, tok=None, lp=None, ws=None, ws_bytes=0) == 0


def commit(L, **over):  # noqa: F811
    a = dict(N=3, S=2, H=4, dk=16, dv=16, dtype=1, flags=0, k=fake(1), v=fake(2), g=fake(3), beta=fake(4), A=fake(5),
             counts=fake(6), hin=fake(7), hout=fake(8))
    a.update(over)
    return L.gdn_step_commit(*[a[n] for n in ("N", "S", "H", "dk", "dv", "dtype", "flags", "k", "v", "g", "beta", "A",
                                              "counts", "hin", "hout")], None)


def test_verification_takes_vocabularies_up_to_a_limit(L):  # noqa: F811
    for dtype in (0, 1):
        assert L.gdn_draft_verify_workspace_size(1, 0, 2 ** 26, dtype) > 0
        assert L.gdn_draft_verify_workspace_size(1, 0, 2 ** 26 + 1, dtype) == 0
        assert L.gdn_draft_verify_workspace_size(31, 0, 2 ** 26, dtype) > 0
        assert L.gdn_draft_verify_workspace_size(33, 0, 2 ** 26, dtype) == 0  # (2^31 elements and more)


def test_commit_rejects_bad_arguments(L):  # noqa: F811
    for over in (dict(N=-1), dict(S=-1), dict(H=0), dict(dk=0), dict(dk=129), dict(dv=129), dict(dtype=3), dict(flags=8),
                 dict(N=1 << 20, H=64, dk=128, dv=128)):
        assert commit(L, **over) == EINVAL, over
    for n in ("k", "v", "g", "beta", "A", "counts", "hout"):
        assert commit(L, **{n: None}) == EINVAL, n
    assert commit(L, hout=off(7, 16)) == EINVAL and b"overlaps" in L.gdn_last_error_detail()
    assert commit(L, hout=fake(1)) == EINVAL and commit(L, k=off(1, 2)) == EINVAL
    assert commit(L, N=0, k=None, v=None, g=None, beta=None, A=None, counts=None, hin=None, hout=None) == 0
    assert commit(L, S=0, k=None, v=None, g=None, beta=None, A=None, counts=None, hout=fake(7)) == 0  # in place: nothing to do


def test_commit_rejects_more_states_than_a_launch_has_threads_for(L):  # noqa: F811
    """A wave takes 64 columns of a state, a launch has fewer than 2^32 threads."""
    far = dict(k=fake(1), v=fake(20), g=fake(40), beta=fake(60), A=fake(80), counts=fake(100), hin=fake(120), hout=fake(140))
    for N, H, dk, dv in ((1 << 26, 1, 1, 1), (1 << 27, 1, 1, 1), (1 << 20, 64, 1, 1), ((1 << 26) - 3, 1, 1, 1), (1 << 22, 16, 5, 6),
                         (1 << 26, 1, 1, 31), (1 << 25, 2, 31, 1)):
        assert commit(L, N=N, S=1, H=H, dk=dk, dv=dv, **far) == EINVAL, (N, H, dk, dv)
        assert b"launch" in L.gdn_last_error_detail()


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z, i = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.draft_verify(z(2, 3, 10), i(2, 2), z(2, 3))
    with pytest.raises(ValueError):
        gdn.draft_verify(z(2, 10), i(2, 2), z(2, 3))
    with pytest.raises(ValueError):
        gdn.draft_verify(z(2, 0, 10), i(2, 2), z(2, 3))
    with pytest.raises(ValueError):
        gdn.step_commit(z(2, 3, 4), z(2, 3, 4, 5), None, None, None, None)
    with pytest.raises(ValueError):
        gdn.step_commit(z(2, 3, 1, 4), z(2, 3, 1, 5), None, None, None, None)
    with pytest.raises(ValueError):
        gdn.page_trim(i(2), i(2), i(2), i(4), i(1), 16)
    with pytest.raises(ValueError):
        gdn.page_trim(i(2), i(2), i(2, 3), i(4), i(1), 2 ** 31)
    with pytest.raises(ValueError):
        gdn.mla_evict(z(3, 4), z(3, 4), i(2, 3), i(2), i(2))
    with pytest.raises(ValueError):
        gdn.mla_evict(None, z(3, 4, 8), i(2, 3), i(2), i(2))
    with pytest.raises(ValueError):
        gdn.mla_weights(z(2, 3), z(3, 4, 8), i(2, 3), i(2), z(2, 3), z(3, 4), scale=1.0)
    with pytest.raises(ValueError):
        gdn.mla_step_shared(z(2, 1, 16), z(3, 4, 16), i(2, 3), i(2), 16, i(3), i(1), i(2), scale=1.0)
