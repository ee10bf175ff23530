"""Latent attention and its paged cache: the binding of the gdn_mla_*,
gdn_norm_rope* and gdn_page_plan entry points of include/gdn.h, which define
the operations. As in the package's other calls, tensors are contiguous HIP
device tensors, every step runs in the library's kernels on the current
stream of the tensors' device, and nothing synchronises."""
from __future__ import annotations

import contextlib
import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import MlaShape, MlaStepShape, _bytes, _check, _dtype_code, _need as _explain, lib

ROPE_NORM, ROPE_INTERLEAVED = 1, 2
_HERE = contextlib.nullcontext()


def _need(t, name, dtype=None, shape=None, device=None):
    """The package's tensor check; the usual case (all is well) in a few
    comparisons, since a decode step makes dozens of them."""
    if (t is None or (type(t) is torch.Tensor and t.is_cuda and (dtype is None or t.dtype is dtype)
                      and (shape is None or t.shape == shape) and (device is None or t.device == device)
                      and t.is_contiguous())):
        return
    _explain(t, name, dtype, shape, device)


def _tensors(**ts):
    for name, t in ts.items():
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor")


def _int32(**sizes):
    """Sizes the library takes as int32 (ctypes would cut the rest off)."""
    for name, n in sizes.items():
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError(f"{name} = {n} is too large")


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _on(dev):
    """The device a launch has to be made on, current for its time."""
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _mla_shape(q, k, v, k_rope, lens, scale):
    if not all(isinstance(t, torch.Tensor) and t.dim() == 4 for t in (q, k, v)):
        raise ValueError("q, k and v must be [B, T, heads, d] tensors")
    B, Tq, H, D = q.shape
    _, Tk, Hk, dn = k.shape
    dr, dv, dev = D - dn, v.shape[-1], q.device
    _int32(q=q.numel(), k=k.numel(), v=v.numel())
    if D < 1 or dr < 0 or (dr > 0) != (k_rope is not None):
        raise ValueError("the last dimension of q must be that of k, plus that of k_rope when it is given")
    Hr = 0
    if k_rope is not None:
        if not isinstance(k_rope, torch.Tensor) or k_rope.dim() != 4:
            raise ValueError("k_rope must be [B, T, heads, dr]")
        Hr = k_rope.shape[2]
        _int32(k_rope=k_rope.numel())
    _need(q, "q", q.dtype, (B, Tq, H, D))
    _need(k, "k", q.dtype, (B, Tk, Hk, dn), dev)
    _need(v, "v", q.dtype, (B, Tk, Hk, dv), dev)
    _need(k_rope, "k_rope", q.dtype, (B, Tk, Hr, dr), dev)
    _need(lens, "lens", torch.int32, (B,), dev)
    return MlaShape(B, Tq, Tk, H, Hk, Hr, dn, dr, dv, _dtype_code(q), D ** -0.5 if scale is None else scale)


def mla_fwd(q, k, v, k_rope=None, lens=None, *, scale=None, want_lse=True, o=None, lse=None):
    """Causal attention of expanded heads. q [B,Tq,H,dn+dr], k [B,Tk,Hk,dn],
    v [B,Tk,Hk,dv], k_rope [B,Tk,Hr,dr] or None; the queries are the last Tq
    of the Tk positions. lens [B] int32: keys of each (right-padded) sequence.
    scale: (dn + dr) ** -0.5 by default. Returns (o, lse or None)."""
    s = _mla_shape(q, k, v, k_rope, lens, scale)
    dev = q.device
    if o is None:
        o = torch.empty((s.B, s.Tq, s.H, s.dv), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, (s.B, s.Tq, s.H, s.dv), dev)
    if lse is None and want_lse:
        lse = torch.empty((s.B, s.Tq, s.H), dtype=torch.float32, device=dev)
    _need(lse, "lse", torch.float32, (s.B, s.Tq, s.H), dev)
    with _on(dev):
        st = lib().gdn_mla_fwd(ctypes.byref(s), _p(q), _p(k), _p(k_rope), _p(v), _p(lens), _p(o), _p(lse),
                               _stream(dev))
    _check("gdn_mla_fwd", st)
    return o, lse


def mla_bwd(q, k, v, o, lse, do, k_rope=None, lens=None, *, scale=None, workspace=None, out=None):
    """Backward of mla_fwd: the gradients of sum(do * o), a dict with dq, dk,
    dv and dk_rope (None without k_rope). The arguments are the forward's, o
    and lse its results."""
    s = _mla_shape(q, k, v, k_rope, lens, scale)
    dev = q.device
    _need(o, "o", q.dtype, (s.B, s.Tq, s.H, s.dv), dev)
    _need(do, "do", q.dtype, (s.B, s.Tq, s.H, s.dv), dev)
    _need(lse, "lse", torch.float32, (s.B, s.Tq, s.H), dev)
    if lse is None or o is None or do is None:
        raise ValueError("o, lse and do are required")
    r = {} if out is None else out
    for name, like in (("dq", q), ("dk", k), ("dv", v), ("dk_rope", k_rope)):
        if r.get(name) is None:
            r[name] = None if like is None else torch.empty_like(like)
        elif like is None:
            raise ValueError("dk_rope without k_rope")
        else:
            _need(r[name], name, q.dtype, like.shape, dev)
    L = lib()
    need = int(L.gdn_mla_bwd_workspace_size(ctypes.byref(s)))
    _need(workspace, "workspace", torch.uint8, None, dev)
    if workspace is None or workspace.numel() < need:
        workspace = _bytes(need, dev)
    with _on(dev):
        st = L.gdn_mla_bwd(ctypes.byref(s), _p(q), _p(k), _p(k_rope), _p(v), _p(lens), _p(o), _p(lse), _p(do),
                           _p(r["dq"]), _p(r["dk"]), _p(r["dk_rope"]), _p(r["dv"]), _p(workspace),
                           workspace.numel(), _stream(dev))
    _check("gdn_mla_bwd", st)
    return r


class LatentAttention(torch.autograd.Function):
    """Autograd wrapper of mla_fwd and mla_bwd; returns o."""

    @staticmethod
    def forward(ctx, q, k, v, k_rope=None, lens=None, scale=None):
        o, lse = mla_fwd(q, k, v, k_rope, lens, scale=scale)
        ctx.save_for_backward(q, k, v, k_rope, lens, o, lse)
        ctx.scale = scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, k_rope, lens, o, lse = ctx.saved_tensors
        r = mla_bwd(q, k, v, o, lse, do.contiguous(), k_rope, lens, scale=ctx.scale)
        return r["dq"], r["dk"], r["dv"], r["dk_rope"], None, None


def mla_step(q, cache, block_table, lens, dl, *, scale, o=None, lse=None, workspace=None):
    """New tokens against their cached rows. q [N,S,H,dl+dr] (or [N,H,dl+dr]
    for one token each), cache [pages,page_size,dl+dr], block_table
    [N,max_pages] int32, lens [N] int32 (the new tokens included; their rows
    are in the cache already). Returns (o [..., dl], lse)."""
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
    s = MlaStepShape(N, S, H, dl, d - dl, _dtype_code(q), cache.shape[0], cache.shape[1], block_table.shape[1], scale)
    L = lib()
    need = int(L.gdn_mla_step_workspace_size(ctypes.byref(s)))
    _need(workspace, "workspace", torch.uint8, None, dev)
    if workspace is None or workspace.numel() < need:
        workspace = _bytes(need, dev)
    if o is None:
        o = torch.empty(lead + (max(int(dl), 0),), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, lead + (dl,), dev)
    if lse is None:
        lse = torch.empty(lead, dtype=torch.float32, device=dev)
    _need(lse, "lse", torch.float32, lead, dev)
    with _on(dev):
        st = L.gdn_mla_step(ctypes.byref(s), _p(q), _p(cache), _p(block_table), _p(lens), _p(o), _p(lse),
                            _p(workspace), workspace.numel(), _stream(dev))
    _check("gdn_mla_step", st)
    return o, lse


def _rope_args(x, weight, positions, freqs, norm, interleaved):
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be [..., H, d]")
    dev, lead, d = x.device, tuple(x.shape[:-2]), x.shape[-1]
    _int32(x=x.numel())
    _need(x, "x", x.dtype)
    if weight is not None and not norm:
        raise ValueError("weight needs norm=True")
    _need(weight, "weight", torch.float32, (d,), dev)
    r = 0
    if freqs is not None:
        if positions is None:
            raise ValueError("freqs need positions")
        r = 2 * freqs.numel()
        _int32(r=r)
        _need(freqs, "freqs", torch.float64, (r // 2,), dev)
        _need(positions, "positions", torch.int32, lead, dev)
    M = 1
    for n in lead:
        M *= n
    flags = (ROPE_NORM if norm else 0) | (ROPE_INTERLEAVED if interleaved else 0)
    return M, x.shape[-2], d, r, _dtype_code(x), flags, dev


def norm_rope(x, weight=None, positions=None, freqs=None, *, norm=True, eps=1e-6, interleaved=False, y=None):
    """Every head's row of x [..., H, d] RMS-normalised (times weight [d]
    fp32), its last 2 * len(freqs) columns turned by positions [...] int32 *
    freqs (fp64). norm=False: the rotation alone. y may be x."""
    M, H, d, r, dt, flags, dev = _rope_args(x, weight, positions, freqs, norm, interleaved)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", x.dtype, x.shape, dev)
    with _on(dev):
        st = lib().gdn_norm_rope(M, H, d, r, dt, flags, eps, _p(x), _p(weight), _p(positions), _p(freqs), _p(y),
                                 _stream(dev))
    _check("gdn_norm_rope", st)
    return y


def norm_rope_bwd(dy, x, weight=None, positions=None, freqs=None, *, norm=True, eps=1e-6, interleaved=False,
                  want_dw=None, workspace=None):
    """Backward of norm_rope: a dict with dx and dw (None unless want_dw, by
    default when weight is given). x is not read without norm."""
    M, H, d, r, dt, flags, dev = _rope_args(dy, weight, positions, freqs, norm, interleaved)
    if norm and x is None:
        raise ValueError("x is required with norm=True")
    _need(x, "x", dy.dtype, dy.shape, dev)
    dx = torch.empty_like(dy)
    dw = None
    if weight is not None if want_dw is None else want_dw:
        dw = torch.empty((d,), dtype=torch.float32, device=dev)
    L = lib()
    need = int(L.gdn_norm_rope_bwd_workspace_size(M, H, d)) if dw is not None else 0
    _need(workspace, "workspace", torch.uint8, None, dev)
    if workspace is None or workspace.numel() < need:
        workspace = _bytes(need, dev)
    with _on(dev):
        st = L.gdn_norm_rope_bwd(M, H, d, r, dt, flags, eps, _p(dy), _p(x), _p(weight), _p(positions), _p(freqs),
                                 _p(dx), _p(dw), _p(workspace), workspace.numel(), _stream(dev))
    _check("gdn_norm_rope_bwd", st)
    return {"dx": dx, "dw": dw}


class NormRope(torch.autograd.Function):
    """Autograd wrapper of norm_rope: gradients for x and weight."""

    @staticmethod
    def forward(ctx, x, weight=None, positions=None, freqs=None, norm=True, eps=1e-6, interleaved=False):
        ctx.save_for_backward(x if norm else None, weight, positions, freqs)
        ctx.how = dict(norm=norm, eps=eps, interleaved=interleaved)
        return norm_rope(x, weight, positions, freqs, norm=norm, eps=eps, interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, positions, freqs = ctx.saved_tensors
        r = norm_rope_bwd(dy.contiguous(), x, weight, positions, freqs, want_dw=weight is not None
                          and ctx.needs_input_grad[1], **ctx.how)
        return r["dx"], r["dw"], None, None, None, None, None


def mla_write(c, k_rope, slots, cache, weight=None, positions=None, freqs=None, *, norm=True, eps=1e-6,
              interleaved=False):
    """New tokens' rows into the paged cache [pages, page_size, dl+dr], in
    place: row slots[i] = [norm(c[i]) * weight | k_rope[i] turned by
    positions[i] * freqs]. c [n,dl], k_rope [n,dr] or None, slots [n] int32
    (outside the cache: skipped; no slot twice). Returns cache."""
    _tensors(c=c, slots=slots, cache=cache)
    if c.dim() != 2 or cache.dim() != 3:
        raise ValueError("c must be [n, dl], cache [pages, page_size, dl + dr]")
    n, dl = c.shape
    _int32(c=c.numel(), d=cache.shape[2])
    dr, dev = cache.shape[2] - dl, c.device
    if dr < 0 or (dr > 0) != (k_rope is not None):
        raise ValueError("the last dimension of cache must be that of c, plus that of k_rope when it is given")
    if weight is not None and not norm:
        raise ValueError("weight needs norm=True")
    _need(c, "c", c.dtype)
    _need(k_rope, "k_rope", c.dtype, (n, dr), dev)
    _need(cache, "cache", c.dtype, None, dev)
    _need(slots, "slots", torch.int32, (n,), dev)
    _need(weight, "weight", torch.float32, (dl,), dev)
    if freqs is not None:
        if positions is None:
            raise ValueError("freqs need positions")
        _need(freqs, "freqs", torch.float64, (dr // 2,), dev)
        _need(positions, "positions", torch.int32, (n,), dev)
    flags = (ROPE_NORM if norm else 0) | (ROPE_INTERLEAVED if interleaved else 0)
    with _on(dev):
        st = lib().gdn_mla_write(n, dl, dr, _dtype_code(c), flags, eps, _p(c), _p(k_rope), _p(weight), _p(positions),
                                 _p(freqs), _p(slots), _p(cache), cache.shape[0] * cache.shape[1], _stream(dev))
    _check("gdn_mla_write", st)
    return cache


def page_plan(lens, new_lens, block_table, free_pages, n_free, page_size, max_tokens, *, lens_out=None,
              n_free_out=None):
    """Pages, slots and positions of the next step's tokens, without leaving
    the GPU. lens, new_lens [N], block_table [N, max_pages], free_pages
    [n_pages], n_free [1], all int32; block_table and free_pages are updated
    in place, new_lens[i] < 0 ends sequence i. Returns a dict with starts
    [N + 1], granted [N], lens [N], n_free [1], slots and positions
    [max_tokens], block_table and free_pages. lens_out=lens and
    n_free_out=n_free update those in place too. positions count the rows that
    a sequence holds, without a shared prefix's and those an eviction dropped."""
    _tensors(lens=lens, new_lens=new_lens, block_table=block_table, free_pages=free_pages, n_free=n_free)
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [N, max_pages], free_pages [n_pages]")
    N, cols = block_table.shape
    _int32(block_table=block_table.numel(), free_pages=free_pages.numel(), page_size=page_size, max_tokens=max_tokens)
    i32, dev = torch.int32, block_table.device
    for t, name, shape in ((block_table, "block_table", (N, cols)), (lens, "lens", (N,)),
                           (new_lens, "new_lens", (N,)), (free_pages, "free_pages", None), (n_free, "n_free", (1,)),
                           (lens_out, "lens_out", (N,)), (n_free_out, "n_free_out", (1,))):
        _need(t, name, i32, shape, dev)
    if max_tokens < 0:
        raise ValueError("max_tokens must be >= 0")
    cap = int(max_tokens)
    # one allocation for what the call makes
    granted, starts, slots, positions, lens_new, n_free_new = torch.empty(
        3 * N + 2 * cap + 2, dtype=i32, device=dev).split([N, N + 1, cap, cap, N, 1])
    lens_out = lens_new if lens_out is None else lens_out
    n_free_out = n_free_new if n_free_out is None else n_free_out
    with _on(dev):
        st = lib().gdn_page_plan(N, cols, free_pages.numel(), page_size, cap, _p(lens), _p(new_lens),
                                 _p(block_table), _p(free_pages), _p(n_free), _p(lens_out), _p(n_free_out),
                                 _p(granted), _p(starts), _p(slots), _p(positions), _stream(dev))
    _check("gdn_page_plan", st)
    return {"starts": starts, "granted": granted, "lens": lens_out, "n_free": n_free_out, "slots": slots,
            "positions": positions, "block_table": block_table, "free_pages": free_pages}
