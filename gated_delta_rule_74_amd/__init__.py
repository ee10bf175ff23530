"""Gated delta rule on MI355X (gfx950): thin Python binding over libgdn.so.

Every step of the computation runs in the library's HIP kernels; this module
only checks tensor properties, allocates outputs and workspaces with PyTorch
and passes raw pointers plus the current HIP stream through the C ABI
declared in include/gdn.h. There is no fallback: if libgdn.so is missing the
calls raise.

    o, hT, ctx = fwd(q, k, v, g, beta, A_log, h0=None, save_context=True)
    grads      = bwd(q, k, v, g, beta, A_log, do, h0=None, dhT=None, context=ctx)
    o, h      = step(q, k, v, g, beta, A_log, h_in, h_out=None)
    o, h      = step_tokens(q, k, v, g, beta, A_log, h_in)     # [N, S, H, *] tokens
    o, hT     = GatedDeltaRule.apply(q, k, v, g, beta, A_log, h0, additive, gate_logits, norm_k, D)
    o, hT, ctx = fwd_noalloc(q, k, v, g, beta, A_log, h0, o=o)   # no device allocation

Layer edges (fused into the kernels, off by default): norm_k=True
L2-normalises every key row where it is loaded (dk comes back with respect to
the raw keys); D [H] fp32 adds the skip term o_t += D[h] v_t (bwd returns dD).

The latent-attention layers of the hybrid stack, and their paged cache
(latent.py):

    o, lse    = mla_fwd(q, k, v, k_rope, lens)                 # expanded heads, causal
    grads     = mla_bwd(q, k, v, o, lse, do, k_rope, lens)
    o         = LatentAttention.apply(q, k, v, k_rope, lens, scale)
    y         = norm_rope(x, weight, positions, freqs)         # per-head norm and rotation
    plan      = page_plan(lens, new_lens, block_table, free_pages, n_free, page_size, max_tokens)
    cache     = mla_write(c, k_rope, plan["slots"], cache, weight, plan["positions"], freqs)
    o, lse    = mla_step(q, cache, block_table, plan["lens"], dl, scale=scale)

Serving beside the plain step (serving.py): prefixes that a batch shares,
drafts, and caches that may not grow:

    o, lse    = mla_step_shared(q, cache, block_table, lens, dl, prefix_table, prefix_lens, starts, scale=scale)
    accepted, tokens, logprobs = draft_verify(logits, draft, uniforms, draft_logits)
    h         = step_commit(k, v, g, beta, A_log, counts, h_in)  # the state after the accepted tokens
    n_free    = page_trim(lens, new_lens, block_table, free_pages, n_free, page_size)
    weights   = mla_weights(q, cache, block_table, lens, lse, weights, scale=scale)
    lens      = mla_evict(weights, cache, block_table, lens, keep, first=4, recent=64)
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = ["fwd", "fwd_noalloc", "bwd", "step", "step_tokens", "GatedDeltaRule", "GdnError", "lib", "EXPORTS",
           "LIB_PATH", "context_size", "context_states", "fwd_workspace_size", "bwd_workspace_size",
           "LaunchTimer", "NOALLOC_SCRATCH_BYTES", "mla_fwd", "mla_bwd", "LatentAttention", "mla_step", "norm_rope",
           "norm_rope_bwd", "NormRope", "mla_write", "page_plan", "mla_step_shared", "mla_weights", "mla_evict", "page_trim",
           "draft_verify", "step_commit"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")
EXPORTS = ["gdn_fwd", "gdn_bwd", "gdn_step", "gdn_step_tokens", "gdn_fwd_workspace_size", "gdn_bwd_workspace_size",
           "gdn_fwd_context_size", "gdn_time_launches", "gdn_launch_kind", "gdn_status_string",
           "gdn_last_error_detail", "gdn_fwd_noalloc", "gdn_mla_fwd", "gdn_mla_bwd", "gdn_mla_bwd_workspace_size",
           "gdn_mla_step", "gdn_mla_step_workspace_size", "gdn_norm_rope", "gdn_norm_rope_bwd",
           "gdn_norm_rope_bwd_workspace_size", "gdn_mla_write", "gdn_page_plan", "gdn_mla_step_shared",
           "gdn_mla_step_shared_workspace_size", "gdn_mla_weights", "gdn_mla_evict", "gdn_mla_evict_workspace_size",
           "gdn_page_trim", "gdn_draft_verify", "gdn_draft_verify_workspace_size", "gdn_step_commit"]

GDN_F32, GDN_BF16 = 0, 1
NOALLOC_SCRATCH_BYTES = 64 << 20  # GDN_NOALLOC_SCRATCH_BYTES of include/gdn.h
GDN_FLAG_ADDITIVE = 1
GDN_FLAG_GATE_LOGITS = 2
GDN_FLAG_L2NORM_K = 4
_lib = None


class GdnError(RuntimeError):
    def __init__(self, func, status, detail):
        super().__init__(f"{func} failed with status {status}: {detail}")
        self.status = status
        self.detail = detail


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class MlaShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Tq", "Tk", "H", "Hk", "Hr", "dn", "dr", "dv", "dtype")] + [
        ("scale", ctypes.c_float)]


class MlaStepShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "S", "H", "dl", "dr", "dtype", "pages", "page_size",
                                              "max_pages")] + [("scale", ctypes.c_float)]


def lib():
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gated_delta_rule_74_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, S, Z = ctypes.c_void_p, ctypes.POINTER(Shape), ctypes.c_size_t
        I32, U32 = ctypes.c_int32, ctypes.c_uint32
        L.gdn_fwd.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]
        L.gdn_fwd_noalloc.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P]
        L.gdn_bwd.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]
        L.gdn_step.argtypes = [I32, I32, I32, I32, I32, U32, P, P, P, P, P, P, P, P, P, P, P]
        L.gdn_step_tokens.argtypes = [I32, I32, I32, I32, I32, I32, U32, P, P, P, P, P, P, P, P, P, P, P]
        for f in (L.gdn_fwd, L.gdn_fwd_noalloc, L.gdn_bwd, L.gdn_step, L.gdn_step_tokens):
            f.restype = ctypes.c_int
        for f in (L.gdn_fwd_workspace_size, L.gdn_bwd_workspace_size, L.gdn_fwd_context_size):
            f.argtypes = [S]
            f.restype = Z
        I64, F = ctypes.c_int64, ctypes.c_float
        A, D = ctypes.POINTER(MlaShape), ctypes.POINTER(MlaStepShape)
        L.gdn_mla_fwd.argtypes = [A, P, P, P, P, P, P, P, P]
        L.gdn_mla_bwd.argtypes = [A, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]
        L.gdn_mla_step.argtypes = [D, P, P, P, P, P, P, P, Z, P]
        L.gdn_norm_rope.argtypes = [I64, I32, I32, I32, I32, U32, F, P, P, P, P, P, P]
        L.gdn_norm_rope_bwd.argtypes = [I64, I32, I32, I32, I32, U32, F, P, P, P, P, P, P, P, P, Z, P]
        L.gdn_mla_write.argtypes = [I64, I32, I32, I32, U32, F, P, P, P, P, P, P, P, I64, P]
        L.gdn_page_plan.argtypes = [I32, I32, I32, I32, I32] + [P] * 12
        L.gdn_mla_step_shared.argtypes = [D, I32, I32] + [P] * 10 + [Z, P]
        L.gdn_mla_weights.argtypes = [D, F] + [P] * 8
        L.gdn_mla_evict.argtypes = [I32] * 7 + [P] * 7 + [Z, P]
        L.gdn_page_trim.argtypes = [I32] * 4 + [P] * 7
        L.gdn_draft_verify.argtypes = [I32] * 4 + [P] * 10 + [Z, P]
        L.gdn_step_commit.argtypes = [I32] * 6 + [U32] + [P] * 9
        for f in (L.gdn_mla_fwd, L.gdn_mla_bwd, L.gdn_mla_step, L.gdn_norm_rope, L.gdn_norm_rope_bwd,
                  L.gdn_mla_write, L.gdn_page_plan, L.gdn_mla_step_shared, L.gdn_mla_weights, L.gdn_mla_evict,
                  L.gdn_page_trim, L.gdn_draft_verify, L.gdn_step_commit):
            f.restype = ctypes.c_int
        L.gdn_mla_bwd_workspace_size.argtypes = [A]
        L.gdn_mla_step_workspace_size.argtypes = [D]
        L.gdn_norm_rope_bwd_workspace_size.argtypes = [I64, I32, I32]
        L.gdn_mla_step_shared_workspace_size.argtypes = [D, I32, I32]
        L.gdn_mla_evict_workspace_size.argtypes = [I32] * 4
        L.gdn_draft_verify_workspace_size.argtypes = [I32] * 4
        for f in (L.gdn_mla_bwd_workspace_size, L.gdn_mla_step_workspace_size, L.gdn_norm_rope_bwd_workspace_size,
                  L.gdn_mla_step_shared_workspace_size, L.gdn_mla_evict_workspace_size,
                  L.gdn_draft_verify_workspace_size):
            f.restype = Z
        L.gdn_time_launches.argtypes = [P, I32]
        L.gdn_time_launches.restype = I32
        L.gdn_launch_kind.argtypes = [I32]
        L.gdn_launch_kind.restype = I32
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_last_error_detail.argtypes = []
        L.gdn_last_error_detail.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(func, status):
    if status != 0:
        raise GdnError(func, status, lib().gdn_last_error_detail().decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t, name, dtype=None, shape=None, device=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a HIP device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _flags(additive, gate_logits, norm_k=False):
    return ((GDN_FLAG_ADDITIVE if additive else 0) | (GDN_FLAG_GATE_LOGITS if gate_logits else 0)
            | (GDN_FLAG_L2NORM_K if norm_k else 0))


def _shape(q, v, additive, gate_logits=False, norm_k=False):
    B, T, H, dk = q.shape
    return Shape(B, T, H, dk, v.shape[-1], _dtype_code(q), 64, _flags(additive, gate_logits, norm_k))


def _check_seq(q, k, v, g, beta, A_log, h0=None, D=None):
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, dk]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _need(q, "q", q.dtype, (B, T, H, dk))
    _need(k, "k", q.dtype, (B, T, H, dk), dev)
    _need(v, "v", q.dtype, (B, T, H, dv), dev)
    _need(g, "g", torch.float32, (B, T, H), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(h0, "h0", torch.float32, (B, H, dk, dv), dev)
    _need(D, "D", torch.float32, (H,), dev)
    return B, T, H, dk, dv


def context_size(q, v, additive=False):
    s = _shape(q, v, additive)
    return int(lib().gdn_fwd_context_size(ctypes.byref(s)))


def fwd_workspace_size(q, v, additive=False):
    s = _shape(q, v, additive)
    return int(lib().gdn_fwd_workspace_size(ctypes.byref(s)))


def _bytes(n, dev):
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=dev)


def context_states(context, q, v):
    """View of the chunk-start states inside a forward context:
    [B, H, ceil(T/64), dk, dv] in the dtype of q (for inspection/tests; the
    context stores each state transposed, so the view is not contiguous)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    NC = (T + 63) // 64
    n = B * H * NC * dk * dv * q.element_size()
    return context[:n].view(q.dtype).view(B, H, NC, dv, dk).transpose(-1, -2)


def bwd_workspace_size(q, v, additive=False):
    s = _shape(q, v, additive)
    return int(lib().gdn_bwd_workspace_size(ctypes.byref(s)))


def fwd(q, k, v, g, beta, A_log, h0=None, *, additive=False, gate_logits=False, norm_k=False, D=None,
        save_context=False, want_hT=True, want_o=True, o=None, hT=None, context=None, workspace=None):
    """Chunked forward. Returns (o or None, hT or None, context or None); the
    context (a byte tensor) lets bwd() skip recomputing the forward.
    gate_logits: g and beta are logits (the kernels apply the sigmoid).
    norm_k: keys L2-normalised per token; D [H]: skip term o += D[h] v.
    want_o=False: a state-only pass (e.g. a prefill for decoding)."""
    B, T, H, dk, dv = _check_seq(q, k, v, g, beta, A_log, h0, D)
    s = _shape(q, v, additive, gate_logits, norm_k)
    dev = q.device
    if o is None and want_o:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, (B, T, H, dv), dev)
    if hT is None and want_hT:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    _need(hT, "hT", torch.float32, (B, H, dk, dv), dev)
    L = lib()
    if context is None and save_context:
        context = _bytes(L.gdn_fwd_context_size(ctypes.byref(s)), dev)
    _need(context, "context", torch.uint8, None, dev)
    if context is not None and context.numel() < L.gdn_fwd_context_size(ctypes.byref(s)):
        raise ValueError("context is smaller than gdn_fwd_context_size()")
    need = int(L.gdn_fwd_workspace_size(ctypes.byref(s)))
    if workspace is None or workspace.numel() < need:
        workspace = _bytes(need, dev)
    st = L.gdn_fwd(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(A_log), _p(D), _p(h0),
                   _p(o), _p(hT), _p(context), _p(workspace), workspace.numel(), _stream(dev))
    _check("gdn_fwd", st)
    return o, hT, context


def fwd_noalloc(q, k, v, g, beta, A_log, h0=None, *, o, hT=None, context=None, additive=False,
                gate_logits=False, norm_k=False, D=None):
    """The forward through gdn_fwd_noalloc: the library takes its workspace
    from a static device array, so the call allocates nothing. Every output
    is the caller's (o may be None only for a state-only pass, given
    explicitly as o=None). Returns (o, hT, context)."""
    B, T, H, dk, dv = _check_seq(q, k, v, g, beta, A_log, h0, D)
    s = _shape(q, v, additive, gate_logits, norm_k)
    dev = q.device
    _need(o, "o", q.dtype, (B, T, H, dv), dev)
    _need(hT, "hT", torch.float32, (B, H, dk, dv), dev)
    _need(context, "context", torch.uint8, None, dev)
    L = lib()
    if context is not None and context.numel() < L.gdn_fwd_context_size(ctypes.byref(s)):
        raise ValueError("context is smaller than gdn_fwd_context_size()")
    st = L.gdn_fwd_noalloc(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(A_log), _p(D),
                           _p(h0), _p(o), _p(hT), _p(context), _stream(dev))
    _check("gdn_fwd_noalloc", st)
    return o, hT, context


def bwd(q, k, v, g, beta, A_log, do, h0=None, dhT=None, *, context=None, additive=False,
        gate_logits=False, norm_k=False, D=None, want_dD=None, want_dh0=True, want_hT=False, workspace=None,
        out=None):
    """Backward of sum(do * o) + sum(dhT * hT). Returns a dict with dq, dk,
    dv, dg, dbeta, dA_log, dD (when want_dD, by default when D is given),
    dh0 (or None) and hT (when want_hT); with gate_logits, dg and dbeta are
    with respect to the logits; with norm_k, dk is with respect to the raw
    keys. norm_k and D must be those of the forward."""
    B, T, H, dk, dv = _check_seq(q, k, v, g, beta, A_log, h0, D)
    dev = q.device
    _need(do, "do", q.dtype, (B, T, H, dv), dev)
    _need(dhT, "dhT", torch.float32, (B, H, dk, dv), dev)
    _need(context, "context", torch.uint8, None, dev)
    s = _shape(q, v, additive, gate_logits, norm_k)
    L = lib()
    if context is not None and context.numel() < L.gdn_fwd_context_size(ctypes.byref(s)):
        raise ValueError("context is smaller than gdn_fwd_context_size()")
    need = int(L.gdn_bwd_workspace_size(ctypes.byref(s)))
    if workspace is None or workspace.numel() < need:
        workspace = _bytes(need, dev)
    r = out if out is not None else {}
    r.setdefault("dq", torch.empty_like(q))
    r.setdefault("dk", torch.empty_like(k))
    r.setdefault("dv", torch.empty_like(v))
    r.setdefault("dg", torch.empty_like(g))
    r.setdefault("dbeta", torch.empty_like(beta))
    r.setdefault("dA_log", torch.empty_like(A_log))
    if want_dD is None:
        want_dD = D is not None
    if want_dD:
        r.setdefault("dD", torch.empty((H,), dtype=torch.float32, device=dev))
    else:
        r["dD"] = None
    if want_dh0:
        r.setdefault("dh0", torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev))
    else:
        r["dh0"] = None
    if want_hT:
        r.setdefault("hT", torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev))
    else:
        r["hT"] = None
    st = L.gdn_bwd(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(A_log), _p(D), _p(h0),
                   _p(context), _p(do), _p(dhT), _p(r["dq"]), _p(r["dk"]), _p(r["dv"]),
                   _p(r["dg"]), _p(r["dbeta"]), _p(r["dA_log"]), _p(r["dD"]), _p(r["dh0"]), _p(r["hT"]),
                   _p(workspace), workspace.numel(), _stream(dev))
    _check("gdn_bwd", st)
    return r


def step(q, k, v, g, beta, A_log, h_in=None, h_out=None, *, additive=False, gate_logits=False, norm_k=False,
         D=None, o=None):
    """One decode token per sequence. q, k [N,H,dk]; v [N,H,dv]; g, beta
    [N,H]; h_in [N,H,dk,dv] fp32 or None. h_out may be h_in (in place).
    Returns (o, h_out)."""
    if q.dim() != 3:
        raise ValueError("q must be [N, H, dk]")
    N, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _need(q, "q", q.dtype, (N, H, dk))
    _need(k, "k", q.dtype, (N, H, dk), dev)
    _need(v, "v", q.dtype, (N, H, dv), dev)
    _need(g, "g", torch.float32, (N, H), dev)
    _need(beta, "beta", torch.float32, (N, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(h_in, "h_in", torch.float32, (N, H, dk, dv), dev)
    _need(D, "D", torch.float32, (H,), dev)
    if h_out is None:
        h_out = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    _need(h_out, "h_out", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, (N, H, dv), dev)
    st = lib().gdn_step(N, H, dk, dv, _dtype_code(q), _flags(additive, gate_logits, norm_k), _p(q),
                        _p(k), _p(v), _p(g), _p(beta), _p(A_log), _p(D), _p(h_in), _p(h_out), _p(o),
                        _stream(dev))
    _check("gdn_step", st)
    return o, h_out


def step_tokens(q, k, v, g, beta, A_log, h_in=None, h_out=None, *, additive=False, gate_logits=False,
                norm_k=False, D=None, o=None):
    """S consecutive decode tokens per sequence from a carried state (e.g. the
    draft tokens of a multi-token prediction). q, k [N,S,H,dk]; v [N,S,H,dv];
    g, beta [N,S,H]; h_in [N,H,dk,dv] fp32 or None; h_out may be h_in.
    Returns (o [N,S,H,dv], h_out)."""
    if q.dim() != 4:
        raise ValueError("q must be [N, S, H, dk]")
    N, S, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _need(q, "q", q.dtype, (N, S, H, dk))
    _need(k, "k", q.dtype, (N, S, H, dk), dev)
    _need(v, "v", q.dtype, (N, S, H, dv), dev)
    _need(g, "g", torch.float32, (N, S, H), dev)
    _need(beta, "beta", torch.float32, (N, S, H), dev)
    _need(A_log, "A_log", torch.float32, (H,), dev)
    _need(h_in, "h_in", torch.float32, (N, H, dk, dv), dev)
    _need(D, "D", torch.float32, (H,), dev)
    if h_out is None:
        h_out = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    _need(h_out, "h_out", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty((N, S, H, dv), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, (N, S, H, dv), dev)
    st = lib().gdn_step_tokens(N, S, H, dk, dv, _dtype_code(q), _flags(additive, gate_logits, norm_k),
                               _p(q), _p(k), _p(v), _p(g), _p(beta), _p(A_log), _p(D), _p(h_in),
                               _p(h_out), _p(o), _stream(dev))
    _check("gdn_step_tokens", st)
    return o, h_out


class LaunchTimer:
    """Brackets every kernel the library launches (from this thread) with
    HIP events, for per-kernel timings: `with LaunchTimer(n) as t: ...` then
    t.durations_ms() gives one duration per launch, in launch order."""

    def __init__(self, max_launches):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * max_launches)]
        for e in self.events:  # torch creates the HIP event on first record
            e.record()
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * len(self.events))(
            *[ctypes.c_void_p(e.cuda_event) for e in self.events])
        self.count = 0

    def __enter__(self):
        lib().gdn_time_launches(self._arr, len(self.events))
        return self

    def __exit__(self, *exc):
        self.count = int(lib().gdn_time_launches(None, 0))
        return False

    def durations_ms(self):
        torch.cuda.synchronize()
        n = min(self.count, len(self.events) // 2)
        return [self.events[2 * i].elapsed_time(self.events[2 * i + 1]) for i in range(n)]

    KINDS = ("fwd_prep", "fwd_chain", "bwd_chain", "bwd_local", "dA_reduce", "step", "fwd_scan", "bwd_scan",
             "mla_fwd", "mla_bwd_q", "mla_bwd_k", "mla_rope_sum", "mla_step", "mla_join", "norm_rope",
             "norm_rope_bwd", "norm_sum", "mla_write", "page_plan", "page_fill", "mla_prefix", "mla_weights",
             "evict_choose", "evict_move", "page_trim", "verify_sums", "verify_decide", "verify_left", "verify_draw", "step_commit")

    def kinds(self):
        """Kernel name of every bracketed launch, in launch order."""
        n = min(self.count, len(self.events) // 2)
        return [self.KINDS[lib().gdn_launch_kind(i)] for i in range(n)]


class GatedDeltaRule(torch.autograd.Function):
    """Autograd wrapper: forward saves its context (chunk-start states and
    per-chunk key blocks), backward reads it instead of recomputing."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, A_log, h0=None, additive=False, gate_logits=False, norm_k=False, D=None):
        o, hT, cs = fwd(q, k, v, g, beta, A_log, h0, additive=additive, gate_logits=gate_logits, norm_k=norm_k,
                        D=D, save_context=True)
        ctx.save_for_backward(q, k, v, g, beta, A_log, h0, cs, D)
        ctx.additive = additive
        ctx.gate_logits = gate_logits
        ctx.norm_k = norm_k
        return o, hT

    @staticmethod
    def backward(ctx, do, dhT):
        q, k, v, g, beta, A_log, h0, cs, D = ctx.saved_tensors
        if do is None:
            do = torch.zeros(q.shape[:3] + (v.shape[-1],), dtype=q.dtype, device=q.device)
        r = bwd(q, k, v, g, beta, A_log, do.contiguous(), h0,
                None if dhT is None else dhT.contiguous(), context=cs,
                additive=ctx.additive, gate_logits=ctx.gate_logits, norm_k=ctx.norm_k, D=D,
                want_dD=D is not None and ctx.needs_input_grad[10], want_dh0=h0 is not None)
        return (r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], r["dA_log"], r["dh0"], None, None, None,
                r["dD"])


from .latent import (LatentAttention, NormRope, mla_bwd, mla_fwd, mla_step, mla_write, norm_rope,  # noqa: E402
                     norm_rope_bwd, page_plan)
from .serving import (draft_verify, mla_evict, mla_step_shared, mla_weights, page_trim, step_commit)  # noqa: E402
