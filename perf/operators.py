"""Workloads of the latent-attention and paged-cache operators.

Each case is one call (for training: forward and backward) of an operator of
the package on inputs made from a seed:

  train   mla_fwd + mla_bwd       causal attention of expanded heads with a shared rotary key
  step    mla_step                new tokens against a paged latent cache (absorbed form)
  norm    norm_rope (+ backward)  per-head RMS norm and rotation of the last columns in one pass
  write   mla_write               latent norm, key rotation and scatter into the paged cache
  plan    page_plan               block tables, slots and positions from request lengths

With `own` false, run() computes them in elementary torch operations in
32 bits (angles in 64), rounded once at the end. exact() computes the
definition in 64 bits, head by head or sequence by sequence.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
THETA = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    """The measured cases."""
    return [
        # the layer of the repository's main workload (dim 896, 16 heads of 56) with a 32-wide rotary part
        dict(name="train layer bf16", op="train", B=8, T=4096, past=0, H=16, Hk=16, Hr=1, dn=56, dr=32, dv=56,
             dtype="bf16", ragged=False),
        # one long document, wide heads, keys and values shared by four query heads each
        dict(name="train long shared bf16", op="train", B=1, T=16384, past=0, H=16, Hk=4, Hr=1, dn=128, dr=64, dv=128,
             dtype="bf16", ragged=False),
        # a small padded batch in full precision, an empty sequence in it, a part of the keys from an earlier chunk
        dict(name="train padded fp32", op="train", B=5, T=331, past=70, H=4, Hk=2, Hr=2, dn=16, dr=16, dv=16,
             dtype="fp32", ragged=True),
        # a full serving batch: one new token for each sequence, lengths from a few tokens to the context
        dict(name="step serve bf16", op="step", N=256, S=1, H=16, dl=128, dr=32, page=64, most=4096, dtype="bf16"),
        # one sequence with a long context and a wide latent: the work has to be split along the cache
        dict(name="step long bf16", op="step", N=1, S=1, H=16, dl=512, dr=64, page=64, most=131072, dtype="bf16"),
        # a draft of three tokens verified at once, short pages, full precision
        dict(name="step draft fp32", op="step", N=48, S=3, H=8, dl=256, dr=64, page=16, most=1500, dtype="fp32"),
        # queries of the layer above, forward and backward
        dict(name="norm train bf16", op="norm", B=8, T=4096, H=16, d=88, r=32, inter=False, grad=True, dtype="bf16"),
        # queries of a small decode batch
        dict(name="norm step fp32", op="norm", B=33, T=1, H=16, d=88, r=32, inter=True, grad=False, dtype="fp32"),
        # the latents of a long prompt batch into the cache
        dict(name="write prompt bf16", op="write", n=32768, dl=512, dr=64, page=64, dtype="bf16"),
        # the latents of one decode step of the serving batch
        dict(name="write step bf16", op="write", n=256, dl=128, dr=32, page=64, dtype="bf16"),
        # one token for each sequence of the serving batch
        dict(name="plan step", op="plan", N=256, most=1, page=64, context=4096, cap=256),
        # prompts of all lengths admitted together, finished sequences released
        dict(name="plan prompts", op="plan", N=1024, most=1024, page=16, context=4096, cap=524288),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["train", "train", "step", "step", "norm", "write", "plan"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "train":
        T = _log(rng, 1, 4096)
        H = rng.choice([1, 2, 4, 8, 16])
        Hk = rng.choice([h for h in (1, 2, 4, 8, 16) if H % h == 0])
        Hr = rng.choice([h for h in (1, 2, 4, 8, 16) if Hk % h == 0])
        B = max(1, min(_log(rng, 1, 16), int(1.5e9 // (H * T * T))))
        return dict(op=op, B=B, T=T, past=rng.choice([0, 0, rng.randrange(0, 300)]), H=H, Hk=Hk, Hr=Hr,
                    dn=8 * rng.randrange(1, 17), dr=8 * rng.randrange(0, 9), dv=8 * rng.randrange(1, 17),
                    dtype=dtype, ragged=rng.random() < 0.5)
    if op == "step":
        most = _log(rng, 1, 65536)
        N = max(1, min(_log(rng, 1, 300), 1000000 // most))
        return dict(op=op, N=N, S=rng.choice([1, 1, 2, 3, 4, 7]), H=rng.choice([1, 2, 4, 8, 16, 24, 32]),
                    dl=16 * rng.randrange(2, 33), dr=8 * rng.randrange(0, 9), page=rng.choice([1, 16, 24, 64, 128]),
                    most=most, dtype=dtype)
    if op == "norm":
        d = rng.randrange(2, 257) if rng.random() < 0.3 else 8 * rng.randrange(1, 65)
        r = min(d - d % 2, 2 * rng.randrange(0, 33))
        T = _log(rng, 1, 8192)
        return dict(op=op, B=rng.randrange(1, 5), T=T, H=rng.choice([1, 3, 4, 8, 16]), d=d, r=r,
                    inter=rng.random() < 0.5, grad=rng.random() < 0.6, dtype=dtype)
    if op == "write":
        return dict(op=op, n=_log(rng, 1, 32768), dl=8 * rng.randrange(1, 65), dr=8 * rng.randrange(0, 9),
                    page=rng.choice([1, 16, 24, 64]), dtype=dtype)
    N = _log(rng, 1, 4096)
    most = _log(rng, 1, max(1, 500000 // N))
    return dict(op=op, N=N, most=most, page=rng.choice([1, 16, 24, 64]), context=most + _log(rng, 16, 4096),
                cap=N * most)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _freqs(r):
    return THETA ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r) if r else None


def _spread(n, top):
    """n lengths from 0 (1 when there are fewer than three) to top, evenly spread."""
    lo = 0 if n >= 3 else min(1, top)
    return [top if n == 1 else lo + (top - lo) * i // (n - 1) for i in range(n)]


def _shuffled(values, g):
    v = torch.tensor(values, dtype=torch.int32, device=DEV)
    return v[torch.randperm(len(values), generator=g, device=DEV)].contiguous()


def prepare(case, seed):
    """The inputs of a case."""
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "train":
        ty = TYPES[case["dtype"]]
        B, T, H, Tk = case["B"], case["T"], case["H"], case["T"] + case["past"]
        s["scale"] = (case["dn"] + case["dr"]) ** -0.5
        s["q"] = _randn(g, (B, T, H, case["dn"] + case["dr"]), ty)
        s["k"] = _randn(g, (B, Tk, case["Hk"], case["dn"]), ty)
        s["kr"] = _randn(g, (B, Tk, case["Hr"], case["dr"]), ty) if case["dr"] else None
        s["v"] = _randn(g, (B, Tk, case["Hk"], case["dv"]), ty)
        s["do"] = _randn(g, (B, T, H, case["dv"]), ty)
        s["lens"] = _shuffled(_spread(B, Tk), g) if case["ragged"] else None
    elif op == "step":
        ty = TYPES[case["dtype"]]
        N, page, d = case["N"], case["page"], case["dl"] + case["dr"]
        cols = -(-case["most"] // page)
        lens = _spread(N, case["most"])
        used = sum(-(-x // page) for x in lens)
        pages = max(1, used) + 1
        s["lens"] = _shuffled(lens, g)
        s["scale"] = d ** -0.5
        s["q"] = _randn(g, (N, case["S"], case["H"], d), ty)
        s["cache"] = _randn(g, (pages, page, d), ty)
        need = (s["lens"] + page - 1) // page
        first = torch.cumsum(need, 0) - need
        at = first[:, None] + torch.arange(cols, device=DEV)[None, :]
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        inside = torch.arange(cols, device=DEV)[None, :] < need[:, None]
        s["table"] = torch.where(inside, order[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
        # rows that no sequence holds keep what uninitialised memory may hold
        rows = torch.ones(pages * page, dtype=torch.bool, device=DEV)
        pos = torch.arange(cols * page, device=DEV)[None, :]
        slot = s["table"].long().repeat_interleave(page, 1) * page + pos % page
        rows[slot[pos < s["lens"][:, None]]] = False
        s["cache"].view(pages * page, d)[rows] = float("nan")
    elif op == "norm":
        ty = TYPES[case["dtype"]]
        B, T, H, d = case["B"], case["T"], case["H"], case["d"]
        s["x"] = _randn(g, (B, T, H, d), ty)
        s["w"] = 1 + 0.1 * _randn(g, (d,))
        s["freqs"] = _freqs(case["r"])
        start = torch.randint(0, 100000, (B, 1), generator=g, device=DEV)
        s["pos"] = (start + torch.arange(T, device=DEV)[None, :]).to(torch.int32)
        s["dy"] = _randn(g, (B, T, H, d), ty) if case["grad"] else None
    elif op == "write":
        ty = TYPES[case["dtype"]]
        n, page = case["n"], case["page"]
        pages = -(-n // page) + 3
        s["c"] = _randn(g, (n, case["dl"]), ty)
        s["kr"] = _randn(g, (n, case["dr"]), ty) if case["dr"] else None
        s["w"] = 1 + 0.1 * _randn(g, (case["dl"],))
        s["freqs"] = _freqs(case["dr"])
        s["pos"] = torch.randint(0, 100000, (n,), generator=g, device=DEV).to(torch.int32)
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32)
        s["slots"] = torch.where(torch.rand(n, generator=g, device=DEV) < 0.02, -1, slots).to(torch.int32)
        s["cache"] = _randn(g, (pages, page, case["dl"] + case["dr"]), ty)
    else:
        N, page, most = case["N"], case["page"], case["most"]
        cols = -(-case["context"] // page)
        lens = torch.randint(0, case["context"] - most + 1, (N,), generator=g, device=DEV)
        new = torch.randint(1, most + 1, (N,), generator=g, device=DEV)
        if most > 1:  # some wait, some have ended
            kind = torch.rand(N, generator=g, device=DEV)
            new = torch.where(kind < 0.1, 0, torch.where(kind < 0.2, -1, new))
        held = (lens + page - 1) // page
        pages = N * cols
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = order.view(N, cols).clone()
        col = torch.arange(cols, device=DEV)[None, :]
        inside = col < held[:, None]
        s["table"] = torch.where(inside, table, -1).contiguous()
        # the free pages as a stack: enough for nine in ten of the pages asked for
        asked = torch.where(new > 0, (lens + new + page - 1) // page - held, 0).sum()
        free = table[~inside]
        s["stack"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        s["stack"][:free.numel()] = free
        s["n_free"] = torch.minimum((asked * 9 + 9) // 10, torch.tensor(free.numel(), device=DEV)).to(
            torch.int32).view(1)
        s["lens"], s["new"] = lens.to(torch.int32), new.to(torch.int32)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    """One pass through the case's operator."""
    return (_own if own else _plain)[state["op"]](state)


def _gdn():
    import gated_delta_rule_74_amd as gdn

    return gdn


def _own_train(s):
    gdn = _gdn()
    o, lse = gdn.mla_fwd(s["q"], s["k"], s["v"], s["kr"], s["lens"], scale=s["scale"])
    r = gdn.mla_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], s["kr"], s["lens"], scale=s["scale"])
    return {"o": o, "lse": lse, "dq": r["dq"], "dk": r["dk"], "dv": r["dv"], "dkr": r["dk_rope"]}


def _own_step(s):
    o, lse = _gdn().mla_step(s["q"], s["cache"], s["table"], s["lens"], s["dl"], scale=s["scale"])
    return {"o": o, "lse": lse}


def _own_norm(s):
    gdn = _gdn()
    y = gdn.norm_rope(s["x"], s["w"], s["pos"], s["freqs"], eps=EPS, interleaved=s["inter"])
    if s["dy"] is None:
        return {"y": y}
    r = gdn.norm_rope_bwd(s["dy"], s["x"], s["w"], s["pos"], s["freqs"], eps=EPS, interleaved=s["inter"])
    return {"y": y, "dx": r["dx"], "dw": r["dw"]}


def _own_write(s):
    return {"cache": _gdn().mla_write(s["c"], s["kr"], s["slots"], s["cache"], s["w"], s["pos"], s["freqs"], eps=EPS)}


def _own_plan(s):
    return _gdn().page_plan(s["lens"], s["new"], s["table"], s["stack"], s["n_free"], s["page"], s["cap"])


# the plain forms

def _heads_first(t, H):
    """[B, T, h, d] in 32 bits as [B, H, T, d], shared heads repeated."""
    t = t.float()
    return t.repeat_interleave(H // t.shape[2], 2).transpose(1, 2).contiguous()


def _seen(B, T, Tk, lens, device):
    """Which keys each query sees, [B or 1, 1, T, Tk]."""
    at = torch.arange(T, device=device)[:, None] + (Tk - T)
    key = torch.arange(Tk, device=device)[None, :]
    seen = (key <= at)[None, None]
    if lens is not None:
        n = lens.long().clamp(0, Tk)[:, None, None, None]
        seen = seen & (key[None, None] < n) & (at[None, None] < n)
    return seen


def _plain_train(s):
    q, do = (s[n].float().transpose(1, 2).contiguous() for n in ("q", "do"))
    B, H, T, _ = q.shape
    k, v, Tk = _heads_first(s["k"], H), _heads_first(s["v"], H), s["k"].shape[1]
    dn = k.shape[-1]
    if s["kr"] is not None:
        k = torch.cat([k, _heads_first(s["kr"], H)], -1)
    seen = _seen(B, T, Tk, s["lens"], q.device)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"]).masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)
    p = p.div_(torch.where(l == 0, 1.0, l))
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2).contiguous()).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)

    def shared(t, h):  # [B, H, Tk, d] -> [B, Tk, h, d], summed over the heads that share one
        return t.view(B, h, H // h, Tk, t.shape[-1]).sum(2).transpose(1, 2).contiguous()

    ty, back = s["q"].dtype, lambda t: t.transpose(1, 2).to(s["q"].dtype).contiguous()  # noqa: E731
    return {"o": back(o), "lse": lse.transpose(1, 2).contiguous(), "dq": back(dq),
            "dk": shared(dk[..., :dn], s["k"].shape[2]).to(ty), "dv": shared(dv, s["v"].shape[2]).to(ty),
            "dkr": None if s["kr"] is None else shared(dk[..., dn:], s["kr"].shape[2]).to(ty)}


def _plain_step(s):
    q, cache, table, lens, dl = s["q"], s["cache"], s["table"], s["lens"], s["dl"]
    N, S, H, d = q.shape
    page, cap = cache.shape[1], table.shape[1] * cache.shape[1]
    pos = torch.arange(cap, device=q.device)
    n = lens.long().clamp(0, cap)[:, None]
    slot = table.long().repeat_interleave(page, 1) * page + pos % page
    held = pos[None, :] < n
    rows = cache.view(-1, d)[torch.where(held, slot, 0)].float()
    rows = rows.masked_fill_(~held[..., None], 0.0)  # [N, cap, d]
    at = n - S + torch.arange(S, device=q.device)[None, :]
    seen = (pos[None, None, :] <= at[..., None])[:, :, None, :]
    qf = q.float().view(N, S * H, d)
    p = torch.matmul(qf, rows.transpose(1, 2).contiguous()).view(N, S, H, cap).mul_(s["scale"])
    p = p.masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(N, S * H, cap), rows[..., :dl].contiguous()).view(N, S, H, dl) / torch.where(l == 0, 1.0, l)
    return {"o": o.to(q.dtype), "lse": (m + l.log()).squeeze(-1)}


def _cos_sin(pos, freqs):
    a = pos.double()[..., None] * freqs
    return a.cos().float(), a.sin().float()


def _pairs(x, inter):
    r = x.shape[-1]
    return (x[..., 0::2], x[..., 1::2]) if inter else (x[..., : r // 2], x[..., r // 2:])


def _join(a, b, inter):
    return torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)


def _turn(x, pos, freqs, inter, back=False):
    """The last columns of [..., H, d] turned by their angles (back: by the negative ones)."""
    if freqs is None:
        return x
    r = 2 * freqs.numel()
    cos, sin = (t[..., None, :] for t in _cos_sin(pos, freqs))
    sin = -sin if back else sin
    a, b = _pairs(x[..., x.shape[-1] - r:], inter)
    return torch.cat([x[..., : x.shape[-1] - r], _join(a * cos - b * sin, b * cos + a * sin, inter)], -1)


def _plain_norm(s):
    x = s["x"].float()
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    hat = x * inv
    y = _turn(hat * s["w"], s["pos"], s["freqs"], s["inter"]).to(s["x"].dtype)
    if s["dy"] is None:
        return {"y": y}
    dz = _turn(s["dy"].float(), s["pos"], s["freqs"], s["inter"], back=True)
    dw = (dz * hat).flatten(0, -2).double().sum(0).float()
    dh = dz * s["w"]
    dx = inv * (dh - hat * (dh * hat).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(s["x"].dtype), "dw": dw}


def _plain_write(s):
    c = s["c"].float()
    row = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["w"]
    if s["kr"] is not None:
        row = torch.cat([row, _turn(s["kr"].float()[:, None, :], s["pos"], s["freqs"], False)[:, 0]], -1)
    flat = s["cache"].view(-1, row.shape[-1])
    go = s["slots"] >= 0
    flat[s["slots"][go].long()] = row.to(flat.dtype)[go]
    return {"cache": s["cache"]}


def _plain_plan(s):
    lens, new, table, stack, page, cap = s["lens"].long(), s["new"].long(), s["table"], s["stack"], s["page"], s["cap"]
    N, cols = table.shape
    dev, F = lens.device, stack.numel()
    held = (lens + page - 1) // page
    gone = new < 0
    # pages of the sequences that ended go back, in order, on top of the stack
    back = torch.where(gone, held, 0)
    back_end = torch.cumsum(back, 0)
    i = torch.arange(N * cols, device=dev)
    who = torch.searchsorted(back_end, i, right=True).clamp(max=N - 1)
    page_id = table[who, (i - (back_end - back)[who]).clamp(0, cols - 1)]
    n_free = s["n_free"].long()
    to = torch.where(i < back_end[-1], n_free + i, F)
    wide = torch.cat([stack, stack.new_zeros(1)]).scatter_(0, to.clamp(max=F), page_id)
    stack.copy_(wide[:F])
    top = n_free + back_end[-1]
    # who gets what it asks for
    ask = torch.where(gone, 0, new)
    need = torch.where(ask > 0, (lens + ask + page - 1) // page - held, 0)
    fits = (lens + ask + page - 1) // page <= cols
    need_f, ask_f = torch.where(fits, need, 0), torch.where(fits, ask, 0)
    need_end, ask_end = torch.cumsum(need_f, 0), torch.cumsum(ask_f, 0)
    yes = fits & (ask_end <= cap) & ((need_f == 0) | (need_end <= top))
    granted = torch.where(yes, ask_f, 0)
    ends = torch.cumsum(granted, 0)
    starts = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    used = torch.where(yes, need_f, 0)
    used_end = torch.cumsum(used, 0)
    # their new pages, from the top of the stack down
    i = torch.arange(min(F, cap // page + 2 * N), device=dev)
    who = torch.searchsorted(used_end, i, right=True).clamp(max=N - 1)
    col = held[who] + i - (used_end - used)[who]
    at = torch.where(i < used_end[-1], who * cols + col, N * cols)
    ids = stack[(top - 1 - i).clamp(0, F - 1)]
    flat = torch.cat([table.view(-1), table.new_zeros(1)]).scatter_(0, at, ids)
    table.copy_(flat[:-1].view(N, cols))
    # where each new token goes
    t = torch.arange(cap, device=dev)
    who = torch.searchsorted(ends, t, right=True).clamp(max=N - 1)
    pos = lens[who] + t - (ends - granted)[who]
    live = t < ends[-1]
    slot = table[who, (pos // page).clamp(0, cols - 1)].long() * page + pos % page
    return {"starts": starts, "granted": granted.to(torch.int32),
            "lens": torch.where(gone, 0, lens + granted).to(torch.int32), "n_free": (top - used_end[-1]).to(torch.int32),
            "slots": torch.where(live, slot, -1).to(torch.int32), "positions": torch.where(live, pos, 0).to(torch.int32),
            "block_table": table, "free_pages": stack}


_plain = {"train": _plain_train, "step": _plain_step, "norm": _plain_norm, "write": _plain_write, "plan": _plain_plan}
_own = {"train": _own_train, "step": _own_step, "norm": _own_norm, "write": _own_write, "plan": _own_plan}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    """Bytes read and written once and operations of one pass."""
    op = case["op"]
    if op == "plan":
        N = case["N"]
        tokens = N * (case["most"] + 1) / 2 * (0.8 if case["most"] > 1 else 1)
        return {"bytes": 4 * (5 * N + 2 * case["cap"] + 2 * tokens / case["page"]), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "train":
        B, T, H, Tk = case["B"], case["T"], case["H"], case["T"] + case["past"]
        D, dv = case["dn"] + case["dr"], case["dv"]
        rows = B * T * H * (2 * D + 2 * dv) + 2 * B * Tk * (case["Hk"] * (case["dn"] + dv) + case["Hr"] * case["dr"])
        pairs = 0
        for n in _spread(B, Tk) if case["ragged"] else [Tk] * B:
            live = max(0, n - case["past"])  # queries at positions past .. n - 1
            pairs += live * case["past"] + live * (live + 1) // 2
        return {"bytes": e * rows + 4 * B * T * H, "flops": 2 * H * pairs * (4 * D + 3 * dv)}
    if op == "step":
        tokens, d = sum(_spread(case["N"], case["most"])), case["dl"] + case["dr"]
        rows = case["N"] * case["S"] * case["H"]
        return {"bytes": e * (tokens * d + rows * (d + case["dl"])) + 4 * rows + 4 * tokens / case["page"],
                "flops": 2 * tokens * case["S"] * case["H"] * (d + case["dl"])}
    if op == "norm":
        n = case["B"] * case["T"] * case["H"] * case["d"]
        return {"bytes": e * n * (5 if case["grad"] else 2) + 4 * case["B"] * case["T"], "flops": n * (20 if case["grad"] else 7)}
    n, d = case["n"], case["dl"] + case["dr"]
    return {"bytes": n * (2 * e * d + 8), "flops": 6 * n * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits (None: whole numbers only)."""
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    return {"train": _exact_train, "step": _exact_step, "norm": _exact_norm, "write": _exact_write}[op](s)


def _softmax_rows(z, ok):
    """exp(z - max) normalised over the allowed columns and the log of the sum; zero rows where none is."""
    z = torch.where(ok, z, torch.full_like(z, -math.inf))
    some = ok.any(-1, keepdim=True)
    top = torch.where(some, z.max(-1, keepdim=True).values, torch.zeros_like(z[..., :1]))
    w = torch.exp(z - top)
    total = w.sum(-1, keepdim=True)
    prob = torch.where(some, w / total, torch.zeros_like(w))
    return prob, torch.where(some, top + total.log(), torch.full_like(top, -math.inf))[..., 0]


def _exact_train(s):
    B, T, H, D = s["q"].shape
    Tk, Hk, dn, dv = s["k"].shape[1], s["k"].shape[2], s["k"].shape[3], s["v"].shape[3]
    out = {"o": torch.zeros(B, T, H, dv), "lse": torch.full((B, T, H), -math.inf), "dq": torch.zeros(B, T, H, D),
           "dk": torch.zeros(B, Tk, Hk, dn), "dv": torch.zeros(B, Tk, Hk, dv),
           "dkr": None if s["kr"] is None else torch.zeros(B, Tk, s["kr"].shape[2], D - dn)}
    out = {n: None if t is None else t.to(DEV, torch.float64) for n, t in out.items()}
    lens = [Tk] * B if s["lens"] is None else s["lens"].tolist()
    for b in range(B):
        n = max(0, min(Tk, lens[b]))
        live = max(0, n - (Tk - T))  # the first `live` queries stand before the end
        if live == 0:
            continue
        at = torch.arange(live, device=DEV)[:, None] + (Tk - T)
        ok = torch.arange(n, device=DEV)[None, :] <= at
        for h in range(H):
            hk = h * Hk // H
            q, do = s["q"][b, :live, h].double(), s["do"][b, :live, h].double()
            k, v = s["k"][b, :n, hk].double(), s["v"][b, :n, hk].double()
            if s["kr"] is not None:
                hr = h * s["kr"].shape[2] // H
                k = torch.cat([k, s["kr"][b, :n, hr].double()], 1)
            prob, lse = _softmax_rows(q @ k.T * s["scale"], ok)
            o = prob @ v
            out["o"][b, :live, h], out["lse"][b, :live, h] = o, lse
            out["dv"][b, :n, hk] += prob.T @ do
            dz = prob * (do @ v.T - (o * do).sum(1, keepdim=True)) * s["scale"]
            out["dq"][b, :live, h] = dz @ k
            dk = dz.T @ q
            out["dk"][b, :n, hk] += dk[:, :dn]
            if s["kr"] is not None:
                out["dkr"][b, :n, hr] += dk[:, dn:]
    return out


def _exact_step(s):
    N, S, H, d = s["q"].shape
    page, dl = s["page"], s["dl"]
    o = torch.zeros(N, S, H, dl, dtype=torch.float64, device=DEV)
    lse = torch.full((N, S, H), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        rows = s["cache"][s["table"][i, : -(-n // page)].long()].reshape(-1, d)[:n].double()
        last = torch.arange(S, device=DEV) + n - S
        ok = torch.arange(n, device=DEV)[None, None, :] <= last[:, None, None]
        z = (s["q"][i].double().reshape(S * H, d) @ rows.T).view(S, H, n) * s["scale"]
        prob, lse[i] = _softmax_rows(z, ok.expand(S, H, n))
        o[i] = (prob.reshape(S * H, n) @ rows[:, :dl]).view(S, H, dl)
    return {"o": o, "lse": lse}


def _as_complex(x, inter):
    a, b = _pairs(x, inter)
    return torch.complex(a.contiguous(), b.contiguous())


def _rotated(x, pos, freqs, inter, sign=1.0):
    """The last columns as complex numbers times exp(i angle), in 64 bits."""
    if freqs is None:
        return x
    r = 2 * freqs.numel()
    ang = sign * pos.double()[..., None, None] * freqs
    z = _as_complex(x[..., x.shape[-1] - r:], inter) * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([x[..., : x.shape[-1] - r], _join(z.real, z.imag, inter)], -1)


def _exact_norm(s):
    x, w = s["x"].double(), s["w"].double()
    rms = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    y = _rotated(x / rms * w, s["pos"], s["freqs"], s["inter"])
    if s["dy"] is None:
        return {"y": y}
    dz = _rotated(s["dy"].double(), s["pos"], s["freqs"], s["inter"], -1.0)
    dot = (dz * w * x).sum(-1, keepdim=True)
    dx = dz * w / rms - x * dot / (x.shape[-1] * rms ** 3)
    return {"y": y, "dx": dx, "dw": (dz * x / rms).reshape(-1, x.shape[-1]).sum(0)}


def _exact_write(s):
    c = s["c"].double()
    row = c / (c.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["w"].double()
    if s["kr"] is not None:
        row = torch.cat([row, _rotated(s["kr"].double()[:, None], s["pos"], s["freqs"], False)[:, 0]], -1)
    cache = s["cache"].double()
    flat = cache.view(-1, row.shape[-1])
    go = s["slots"] >= 0
    flat[s["slots"][go].long()] = row[go]
    return {"cache": cache}
