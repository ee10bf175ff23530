"""Serving beside the plain decode step: prefixes that a batch shares, drafts
and what follows from them, and caches that may not grow. The binding of the
gdn_mla_step_shared, gdn_mla_weights, gdn_mla_evict, gdn_page_trim,
gdn_draft_verify and gdn_step_commit entry points of include/gdn.h, which
define the operations. As in the package's other calls, tensors are contiguous
HIP device tensors, every step runs in the library's kernels on the current
stream of the tensors' device, and nothing synchronises."""
from __future__ import annotations

import ctypes

import torch

from . import MlaStepShape, _bytes, _check, _dtype_code, _flags, lib
from .latent import _int32, _need, _on, _p, _stream, _tensors


def _space(workspace, need, dev):
    _need(workspace, "workspace", torch.uint8, None, dev)
    return _bytes(need, dev) if workspace is None or workspace.numel() < need else workspace


def _paged(q, cache, block_table, lens, dl, scale):
    """Shape of a call over the paged cache, and the leading dimensions of q ([N, S, H] or [N, H])."""
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be [N, S, H, d] or [N, H, d]")
    _tensors(cache=cache, block_table=block_table, lens=lens)
    if cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("cache must be [pages, page_size, d], block_table [N, max_pages]")
    _int32(q=q.numel(), dl=dl, pages=cache.shape[0], page_size=cache.shape[1], max_pages=block_table.shape[1])
    lead, d, dev = tuple(q.shape[:-1]), q.shape[-1], q.device
    N, H, S = lead[0], lead[-1], lead[1] if len(lead) == 3 else 1
    _need(q, "q", q.dtype)
    _need(cache, "cache", q.dtype, tuple(cache.shape[:2]) + (d,), dev)
    _need(block_table, "block_table", torch.int32, (N, block_table.shape[1]), dev)
    _need(lens, "lens", torch.int32, (N,), dev)
    return MlaStepShape(N, S, H, dl, d - dl, _dtype_code(q), cache.shape[0], cache.shape[1], block_table.shape[1],
                        scale), lead


def mla_step_shared(q, cache, block_table, lens, dl, prefix_table, prefix_lens, starts, *, scale, o=None, lse=None,
                    workspace=None):
    """mla_step for sequences that share long prefixes: sequences starts[g] ..
    starts[g + 1] - 1 see the prefix_lens[g] cached rows of prefix_table[g]
    before their own. q, cache, block_table, lens as in mla_step (lens counts
    own rows only, the new tokens' included); prefix_table [G, prefix_pages],
    prefix_lens [G], starts [G + 1], all int32. page_plan's positions of the new
    tokens lack the prefix's length: add it before rows and queries are turned by
    them. Returns (o [..., dl], lse)."""
    s, lead = _paged(q, cache, block_table, lens, dl, scale)
    _tensors(prefix_table=prefix_table, prefix_lens=prefix_lens, starts=starts)
    if prefix_table.dim() != 2:
        raise ValueError("prefix_table must be [G, prefix_pages]")
    (G, cols), dev = prefix_table.shape, q.device
    _int32(G=G, prefix_pages=cols)
    _need(prefix_table, "prefix_table", torch.int32, (G, cols), dev)
    _need(prefix_lens, "prefix_lens", torch.int32, (G,), dev)
    _need(starts, "starts", torch.int32, (G + 1,), dev)
    L = lib()
    workspace = _space(workspace, int(L.gdn_mla_step_shared_workspace_size(ctypes.byref(s), G, cols)), dev)
    if o is None:
        o = torch.empty(lead + (max(int(dl), 0),), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, lead + (dl,), dev)
    if lse is None:
        lse = torch.empty(lead, dtype=torch.float32, device=dev)
    _need(lse, "lse", torch.float32, lead, dev)
    with _on(dev):
        st = L.gdn_mla_step_shared(ctypes.byref(s), G, cols, _p(q), _p(cache), _p(block_table), _p(lens),
                                   _p(prefix_table), _p(prefix_lens), _p(starts), _p(o), _p(lse), _p(workspace),
                                   workspace.numel(), _stream(dev))
    _check("gdn_mla_step_shared", st)
    return o, lse


def mla_weights(q, cache, block_table, lens, lse, weights, known=None, *, scale, decay=1.0):
    """Attention weight of every cached row of the sequences, added to weights
    [pages, page_size] fp32 in place: rows at positions below known [N] (by
    default lens - S: the new tokens' rows begin anew) keep decay times what
    they had. q, cache, block_table, lens as in mla_step, lse its result.
    Returns weights."""
    # (a row is one vector here: how it splits into latent and rotary part does not matter)
    d = q.shape[-1] if isinstance(q, torch.Tensor) and q.dim() else 0
    dl = min(512, d // 16 * 16)
    s, lead = _paged(q, cache, block_table, lens, dl, scale)
    dev = q.device
    _tensors(lse=lse, weights=weights)
    _need(lse, "lse", torch.float32, lead, dev)
    _need(weights, "weights", torch.float32, tuple(cache.shape[:2]), dev)
    _need(known, "known", torch.int32, (s.N,), dev)
    with _on(dev):
        st = lib().gdn_mla_weights(ctypes.byref(s), decay, _p(q), _p(cache), _p(block_table), _p(lens), _p(lse),
                                   _p(known), _p(weights), _stream(dev))
    _check("gdn_mla_weights", st)
    return weights


def mla_evict(weights, cache, block_table, lens, keep, *, first=0, recent=0, lens_out=None, workspace=None):
    """Drops the cached rows of least weight: sequence n keeps keep[n] rows, the
    first `first`, the last `recent` and those of the highest weights, moved to
    the front of its pages in their order, in cache [pages, page_size, d] and
    weights [pages, page_size] alike. block_table [N, max_pages], lens, keep
    [N] int32. Sequences that share a page with another must not be evicted.
    Kept rows stay turned as they are, and page_plan's positions of later tokens
    lack the rows dropped: add lens less the result, from every eviction, before
    rows and queries are turned by them. Returns the new lengths (page_trim gives
    the pages back)."""
    _tensors(weights=weights, cache=cache, block_table=block_table, lens=lens, keep=keep)
    if cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("cache must be [pages, page_size, d], block_table [N, max_pages]")
    (pages, page, d), (N, cols), dev = cache.shape, block_table.shape, cache.device
    row = d * cache.element_size()
    _int32(pages=pages, page_size=page, N=N, max_pages=cols, row_bytes=row, first=first, recent=recent)
    _dtype_code(cache)
    _need(cache, "cache", cache.dtype)
    _need(weights, "weights", torch.float32, (pages, page), dev)
    i32 = torch.int32
    _need(block_table, "block_table", i32, (N, cols), dev)
    _need(lens, "lens", i32, (N,), dev)
    _need(keep, "keep", i32, (N,), dev)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    _need(lens_out, "lens_out", i32, (N,), dev)
    L = lib()
    workspace = _space(workspace, int(L.gdn_mla_evict_workspace_size(N, cols, page, row)), dev)
    with _on(dev):
        st = L.gdn_mla_evict(N, cols, pages, page, row, first, recent, _p(block_table), _p(lens), _p(keep),
                             _p(weights), _p(cache), _p(lens_out), _p(workspace), workspace.numel(), _stream(dev))
    _check("gdn_mla_evict", st)
    return lens_out


def page_trim(lens, new_lens, block_table, free_pages, n_free, page_size, *, n_free_out=None):
    """Pages behind sequences that became shorter (rejected drafts, evicted
    rows) back on the stack of free pages, without leaving the GPU: block_table
    [N, max_pages], lens and new_lens [N], free_pages [n_pages] (updated in
    place), n_free [1], all int32; table entries below 0 are no pages and are
    left out. Returns the number of free pages afterwards
    [1] (n_free_out=n_free updates it in place)."""
    _tensors(lens=lens, new_lens=new_lens, block_table=block_table, free_pages=free_pages, n_free=n_free)
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [N, max_pages], free_pages [n_pages]")
    (N, cols), i32, dev = block_table.shape, torch.int32, block_table.device
    _int32(block_table=block_table.numel(), free_pages=free_pages.numel(), page_size=page_size)
    for t, name, shape in ((block_table, "block_table", None), (lens, "lens", (N,)), (new_lens, "new_lens", (N,)),
                           (free_pages, "free_pages", None), (n_free, "n_free", (1,)),
                           (n_free_out, "n_free_out", (1,))):
        _need(t, name, i32, shape, dev)
    if n_free_out is None:
        n_free_out = torch.empty_like(n_free)
    with _on(dev):
        st = lib().gdn_page_trim(N, cols, free_pages.numel(), page_size, _p(lens), _p(new_lens), _p(block_table),
                                 _p(free_pages), _p(n_free), _p(n_free_out), _stream(dev))
    _check("gdn_page_trim", st)
    return n_free_out


def draft_verify(logits, draft, uniforms, draft_logits=None, draft_lens=None, temperature=None, *, want_logprobs=True,
                 workspace=None):
    """Drafted tokens against the target's distributions, from given random
    numbers. logits [N, S+1, V] (row i where draft[:, i] is to stand), draft
    [N, S] int32, uniforms [N, S+1] fp32 in [0, 1), draft_logits [N, S, V] what
    the draft was drawn from (None: drafts without a distribution), draft_lens
    [N] int32 how many of them count, temperature [N] fp32 (0: greedy). Returns
    (accepted [N], tokens [N, S+1], logprobs [N, S+1] or None): the drafts
    accepted, then the token drawn, then -1."""
    _tensors(logits=logits, draft=draft, uniforms=uniforms)
    if logits.dim() != 3 or logits.shape[1] < 1:
        raise ValueError("logits must be [N, S + 1, V]")
    (N, S1, V), dev = logits.shape, logits.device
    _int32(logits=logits.numel(), N=N, S=S1, V=V)
    _need(logits, "logits", logits.dtype)
    _need(draft, "draft", torch.int32, (N, S1 - 1), dev)
    _need(uniforms, "uniforms", torch.float32, (N, S1), dev)
    _need(draft_logits, "draft_logits", logits.dtype, (N, S1 - 1, V), dev)
    _need(draft_lens, "draft_lens", torch.int32, (N,), dev)
    _need(temperature, "temperature", torch.float32, (N,), dev)
    L, code = lib(), _dtype_code(logits)
    workspace = _space(workspace, int(L.gdn_draft_verify_workspace_size(N, S1 - 1, V, code)), dev)
    accepted = torch.empty((N,), dtype=torch.int32, device=dev)
    tokens = torch.empty((N, S1), dtype=torch.int32, device=dev)
    logprobs = torch.empty((N, S1), dtype=torch.float32, device=dev) if want_logprobs else None
    with _on(dev):
        st = L.gdn_draft_verify(N, S1 - 1, V, code, _p(logits), _p(draft), _p(draft_lens), _p(draft_logits),
                                _p(temperature), _p(uniforms), _p(accepted), _p(tokens), _p(logprobs), _p(workspace),
                                workspace.numel(), _stream(dev))
    _check("gdn_draft_verify", st)
    return accepted, tokens, logprobs


def step_commit(k, v, g, beta, A_log, counts, h_in=None, h_out=None, *, additive=False, gate_logits=False,
                norm_k=False):
    """The states after the first counts[n] of S tokens (e.g. the accepted ones
    of a draft): step_tokens without its outputs. k [N,S,H,dk]; v [N,S,H,dv]; g,
    beta [N,S,H]; counts [N] int32; h_in [N,H,dk,dv] fp32 or None; h_out may be
    h_in. Returns h_out."""
    if not all(isinstance(t, torch.Tensor) and t.dim() == 4 for t in (k, v)):
        raise ValueError("k and v must be [N, S, H, d]")
    (N, S, H, dk), dv, dev, f32 = k.shape, v.shape[-1], k.device, torch.float32
    _tensors(g=g, beta=beta, A_log=A_log, counts=counts)
    _int32(k=k.numel(), v=v.numel(), state=N * H * dk * dv)
    _need(k, "k", k.dtype)
    _need(v, "v", k.dtype, (N, S, H, dv), dev)
    _need(g, "g", f32, (N, S, H), dev)
    _need(beta, "beta", f32, (N, S, H), dev)
    _need(A_log, "A_log", f32, (H,), dev)
    _need(counts, "counts", torch.int32, (N,), dev)
    _need(h_in, "h_in", f32, (N, H, dk, dv), dev)
    if h_out is None:
        h_out = torch.empty((N, H, dk, dv), dtype=f32, device=dev)
    _need(h_out, "h_out", f32, (N, H, dk, dv), dev)
    with _on(dev):
        st = lib().gdn_step_commit(N, S, H, dk, dv, _dtype_code(k), _flags(additive, gate_logits, norm_k), _p(k),
                                   _p(v), _p(g), _p(beta), _p(A_log), _p(counts), _p(h_in), _p(h_out), _stream(dev))
    _check("gdn_step_commit", st)
    return h_out
