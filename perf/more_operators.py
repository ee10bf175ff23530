"""Workloads of the serving operators beside the plain decode step.

Each case is one pass through an operator of the package on inputs made from a
seed:

  shared   mla_step_shared        new tokens against a paged latent cache whose sequences share long prefixes
  verify   draft_verify           drafted tokens against the target's distributions, from given random numbers
  commit   step_commit            the recurrent state after the accepted tokens
  weights  mla_weights            attention weight added up for every cached row
  evict    mla_evict + page_trim  the rows of least weight dropped, the rest moved up, whole pages given back
  trim     page_trim              pages behind shortened sequences given back

With `own` false, run() computes them in elementary torch operations, in 32
bits and rounded once at the end, and in 64 bits where whole numbers hang on
the sums. exact() computes the definition in 64 bits, sequence by sequence.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    """The measured cases."""
    return [
        # a serving batch behind one long system prompt: one new token for each sequence, answers of up to 1024 rows
        dict(name="shared serve bf16", op="shared", N=256, S=1, H=16, dl=128, dr=32, page=64, G=1, prefix=16384,
             most=1024, dtype="bf16"),
        # drafts of three tokens, four groups with documents of their own, a wide latent
        dict(name="shared groups bf16", op="shared", N=48, S=3, H=16, dl=512, dr=64, page=64, G=4, prefix=8191,
             most=700, dtype="bf16"),
        # a few sequences with short prefixes, full precision: latency counts
        dict(name="shared small fp32", op="shared", N=5, S=1, H=8, dl=64, dr=16, page=16, G=2, prefix=700, most=90,
             dtype="fp32"),
        # a depth-2 draft of the serving batch, tokenizer of 64 k and 256 bytes, sampled and greedy sequences together
        dict(name="verify serve bf16", op="verify", N=256, S=2, V=65792, q=True, ragged=True, dtype="bf16"),
        # a few sequences, drafts without a distribution (looked up), an odd vocabulary
        dict(name="verify lookup fp32", op="verify", N=3, S=4, V=32001, q=False, ragged=False, dtype="fp32"),
        # the states of one layer of the serving batch after its drafts were verified
        dict(name="commit serve bf16", op="commit", N=256, S=3, H=16, dk=56, dv=56, dtype="bf16"),
        # longer drafts of a small batch in full precision
        dict(name="commit small fp32", op="commit", N=33, S=7, H=8, dk=64, dv=64, dtype="fp32"),
        # every step of the serving batch
        dict(name="weights serve bf16", op="weights", N=256, S=1, H=16, dl=128, dr=32, page=64, most=4096, fresh=False,
             dtype="bf16"),
        # the last 32 tokens of prompts, which weigh all rows before them for the first time
        dict(name="weights window fp32", op="weights", N=12, S=32, H=8, dl=256, dr=64, page=16, most=2000, fresh=True,
             dtype="fp32"),
        # the serving batch cut down to half the context
        dict(name="evict serve bf16", op="evict", N=256, dl=128, dr=32, page=64, most=4096, keep=2048, first=4,
             recent=64, dtype="bf16"),
        # one long context halved
        dict(name="evict long bf16", op="evict", N=1, dl=512, dr=64, page=64, most=131072, keep=65536, first=16,
             recent=1024, dtype="bf16"),
        # the serving batch after its drafts were verified
        dict(name="trim serve", op="trim", N=256, page=16, most=4096, drop=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["shared", "shared", "verify", "verify", "commit", "weights", "evict", "evict", "trim"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    latent = dict(dl=16 * rng.randrange(2, 33), dr=8 * rng.randrange(0, 9), page=rng.choice([1, 16, 24, 64, 128]))
    if op == "shared":
        S, H = rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 4, 8, 16, 24])
        prefix = _log(rng, 1, 32768)
        room = 4e10 if dtype == "bf16" else 5e9
        N = max(1, min(_log(rng, 1, 300), int(room // (S * H * prefix * 4 * latent["dl"]))))
        return dict(op=op, N=N, S=S, H=H, **latent, G=rng.randrange(1, min(N, 6) + 1), prefix=prefix,
                    most=min(_log(rng, 1, 1500), max(1, 200000 // N)), dtype=dtype)
    if op == "verify":
        V, S = _log(rng, 50, 150000), rng.randrange(1, 9)
        return dict(op=op, N=max(1, min(_log(rng, 1, 300), 50000000 // (V * (2 * S + 1)))), S=S, V=V,
                    q=rng.random() < 0.7, ragged=rng.random() < 0.5, dtype=dtype)
    if op == "commit":
        top = 128 if dtype == "bf16" else 64
        return dict(op=op, N=_log(rng, 1, 256), S=rng.randrange(1, 9), H=rng.choice([1, 3, 8, 16]),
                    dk=rng.randrange(8, top + 1), dv=rng.randrange(8, top + 1), dtype=dtype)
    most = _log(rng, 1, 65536)
    N = max(1, min(_log(rng, 1, 300), 500000 // most))
    if op == "weights":
        fresh = rng.random() < 0.3
        return dict(op=op, N=N, S=rng.choice([8, 17, 32]) if fresh else rng.choice([1, 1, 2, 3]),
                    H=rng.choice([1, 4, 8, 16, 24]), **latent, most=most, fresh=fresh, dtype=dtype)
    if op == "evict":
        keep = rng.randrange(0, most + 1)
        return dict(op=op, N=N, **latent, most=most, keep=keep, first=rng.choice([0, 4]),
                    recent=rng.choice([0, 1, 64]), dtype=dtype)
    return dict(op=op, N=_log(rng, 1, 2048), page=rng.choice([1, 16, 24, 64]), most=_log(rng, 1, 4096),
                drop=_log(rng, 1, 4096))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _rand(g, shape):
    return torch.rand(shape, generator=g, device=DEV)


def _spread(n, top):
    """n lengths from 0 (1 when there are fewer than three) to top, evenly spread."""
    lo = 0 if n >= 3 else min(1, top)
    return [top if n == 1 else lo + (top - lo) * i // (n - 1) for i in range(n)]


def _shuffled(values, g):
    v = torch.tensor(values, dtype=torch.int32, device=DEV)
    return v[torch.randperm(len(values), generator=g, device=DEV)].contiguous()


def _tables(lens, page, cols, order, at):
    """Block table of sequences of these lengths, their pages order[at:] one after the other; the first one unused."""
    need = (lens + page - 1) // page
    ends = torch.cumsum(need, 0) + at
    where = (ends - need)[:, None] + torch.arange(cols, device=DEV)[None, :]
    inside = torch.arange(cols, device=DEV)[None, :] < need[:, None]
    table = torch.where(inside, order[where.clamp(max=order.numel() - 1)], -1)
    return table.to(torch.int32).contiguous(), int(ends[-1])


def _held(table, lens, page):
    """Slots of the rows that sequences hold."""
    pos = torch.arange(table.shape[1] * page, device=DEV)
    slot = table.long().repeat_interleave(page, 1) * page + pos % page
    return slot[pos[None, :] < lens[:, None]]


def _cache(g, pages, page, d, ty, used):
    """A pool of rows; those that no sequence holds keep what uninitialised memory may hold."""
    cache = _randn(g, (pages, page, d), ty)
    free = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    for slots in used:
        free[slots] = False
    cache.view(pages * page, d)[free] = float("nan")
    return cache


def _groups(n, g):
    """Group g of `g` holds a share of n sequences that grows with its number."""
    total = g * (g + 1) // 2
    return [n * (i * (i + 1) // 2) // total for i in range(g + 1)]


def prepare(case, seed):
    """The inputs of a case."""
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op in ("shared", "weights", "evict"):
        ty, N, page, d = TYPES[case["dtype"]], case["N"], case["page"], case["dl"] + case["dr"]
        cols = -(-case["most"] // page)
        lens = _spread(N, case["most"])
        s["lens"], s["scale"] = _shuffled(lens, g), d ** -0.5
        own_pages = sum(-(-x // page) for x in lens)
    if op == "shared":
        G = case["G"]
        # prefixes from half to all of the longest
        plens = [case["prefix"] - case["prefix"] * i // (2 * G) for i in range(G)]
        pages = own_pages + sum(-(-x // page) for x in plens) + 1
        order = torch.randperm(pages, generator=g, device=DEV)
        s["prefix_lens"] = _shuffled(plens, g)
        s["table"], at = _tables(s["lens"], page, cols, order, 0)
        s["prefix_table"], _ = _tables(s["prefix_lens"], page, -(-case["prefix"] // page), order, at)
        s["starts"] = torch.tensor(_groups(N, G), dtype=torch.int32, device=DEV)
        s["q"] = _randn(g, (N, case["S"], case["H"], d), ty)
        s["cache"] = _cache(g, pages, page, d, ty, [_held(s["table"], s["lens"], page),
                                                    _held(s["prefix_table"], s["prefix_lens"], page)])
    elif op == "weights":
        pages = own_pages + 1
        order = torch.randperm(pages, generator=g, device=DEV)
        s["table"], _ = _tables(s["lens"], page, cols, order, 0)
        s["q"] = _randn(g, (N, case["S"], case["H"], d), ty)
        s["cache"] = _cache(g, pages, page, d, ty, [_held(s["table"], s["lens"], page)])
        # the step's own statistics
        z, seen, _ = _own_scores(s, torch.float64)
        s["lse"] = torch.logsumexp(z, -1).to(torch.float32)
        del z, seen
        s["weights"] = _rand(g, (pages, page))
        s["known"] = torch.zeros_like(s["lens"]) if case["fresh"] else None
        s["decay"] = 1.0 if case["fresh"] else 0.95
    elif op == "evict":
        # pages of the pool: those in use, and twenty free ones
        pages = own_pages + 20
        order = torch.randperm(pages, generator=g, device=DEV)
        s["table"], at = _tables(s["lens"], page, cols, order, 0)
        slots = _held(s["table"], s["lens"], page)
        s["cache"] = _cache(g, pages, page, d, ty, [slots])
        # attention weights: a few rows have most of it, some none at all
        w = torch.exp(3 * _randn(g, (pages * page,))) * (_rand(g, (pages * page,)) > 0.1)
        s["weights"] = w.view(pages, page).contiguous()
        s["keep"] = torch.full((N,), case["keep"], dtype=torch.int32, device=DEV)
        s["stack"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        s["stack"][:pages - at] = order[at:].to(torch.int32)
        s["n_free"] = torch.tensor([pages - at], dtype=torch.int32, device=DEV)
    elif op == "trim":
        N, page = case["N"], case["page"]
        s["lens"] = torch.randint(0, case["most"] + 1, (N,), generator=g, device=DEV).to(torch.int32)
        gone = torch.randint(0, case["drop"] + 1, (N,), generator=g, device=DEV).to(torch.int32)
        s["new_lens"] = (s["lens"] - gone).clamp(min=0)
        pages = N * -(-case["most"] // page) + 20
        order = torch.randperm(pages, generator=g, device=DEV)
        s["table"], at = _tables(s["lens"], page, -(-case["most"] // page), order, 0)
        s["stack"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        s["stack"][:pages - at] = order[at:].to(torch.int32)
        s["n_free"] = torch.tensor([pages - at], dtype=torch.int32, device=DEV)
    elif op == "verify":
        ty, N, S, V = TYPES[case["dtype"]], case["N"], case["S"], case["V"]
        z = 2.5 * _randn(g, (N, S + 1, V))
        s["logits"] = z.to(ty)
        # one sequence in eight is greedy, the others are sampled at temperatures around one
        t = 0.6 + 0.8 * _rand(g, (N,))
        s["temperature"] = torch.where(_rand(g, (N,)) < 0.125, 0.0, t).contiguous()
        # the draft's head is the target's, a little off
        zq = (z[:, :S] + 0.7 * _randn(g, (N, S, V))).to(ty)
        # its tokens, drawn from its distribution
        heat = s["temperature"][:, None, None]
        noise = -torch.log(-torch.log(_rand(g, (N, S, V)).clamp(1e-20, 1 - 1e-7)))
        s["draft"] = (zq.float() + heat * noise).argmax(-1).to(torch.int32)
        s["draft_logits"] = zq.contiguous() if case["q"] else None
        s["draft_lens"] = (torch.randint(0, S + 1, (N,), generator=g, device=DEV).to(torch.int32) if case["ragged"]
                           else None)
        s["uniforms"] = _rand(g, (N, S + 1))
    else:
        ty, N, S, H, dk, dv = TYPES[case["dtype"]], *(case[n] for n in ("N", "S", "H", "dk", "dv"))
        k = _randn(g, (N, S, H, dk))
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(ty)
        s["v"] = _randn(g, (N, S, H, dv), ty)
        s["g"], s["beta"] = _rand(g, (N, S, H)), _rand(g, (N, S, H))
        s["A_log"] = _randn(g, (H,))
        s["counts"] = torch.randint(0, S + 1, (N,), generator=g, device=DEV).to(torch.int32)
        s["h"] = _randn(g, (N, H, dk, dv))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    """One pass through the case's operator."""
    return (_own if own else _plain)[state["op"]](state)


def _gdn():
    import gated_delta_rule_74_amd as gdn

    return gdn


def _own_shared(s):
    o, lse = _gdn().mla_step_shared(s["q"], s["cache"], s["table"], s["lens"], s["dl"], s["prefix_table"],
                                    s["prefix_lens"], s["starts"], scale=s["scale"])
    return {"o": o, "lse": lse}


def _own_verify(s):
    accepted, tokens, logprobs = _gdn().draft_verify(s["logits"], s["draft"], s["uniforms"], s["draft_logits"],
                                                     s["draft_lens"], s["temperature"])
    return {"accepted": accepted, "tokens": tokens, "logprobs": logprobs}


def _own_commit(s):
    return {"h": _gdn().step_commit(s["k"], s["v"], s["g"], s["beta"], s["A_log"], s["counts"], s["h"])}


def _own_weights(s):
    return {"weights": _gdn().mla_weights(s["q"], s["cache"], s["table"], s["lens"], s["lse"], s["weights"],
                                          s["known"], scale=s["scale"], decay=s["decay"])}


def _own_evict(s):
    gdn = _gdn()
    lens = gdn.mla_evict(s["weights"], s["cache"], s["table"], s["lens"], s["keep"], first=s["first"],
                         recent=s["recent"])
    n_free = gdn.page_trim(s["lens"], lens, s["table"], s["stack"], s["n_free"], s["page"])
    return {"weights": s["weights"], "cache": s["cache"], "lens": lens, "free_pages": s["stack"], "n_free": n_free}


def _own_trim(s):
    n_free = _gdn().page_trim(s["lens"], s["new_lens"], s["table"], s["stack"], s["n_free"], s["page"])
    return {"free_pages": s["stack"], "n_free": n_free}


# the plain forms

def _own_scores(s, ty):
    """Scores of every token against its sequence's rows [N, S, H, cap] (-inf where it sees none), which it sees, the rows."""
    q, cache, table, page = s["q"], s["cache"], s["table"], s["page"]
    N, S, H, d = q.shape
    cap = table.shape[1] * page
    pos = torch.arange(cap, device=q.device)
    n = s["lens"].long().clamp(0, cap)[:, None]
    slot = table.long().repeat_interleave(page, 1) * page + pos % page
    held = pos[None, :] < n
    rows = cache.view(-1, d)[torch.where(held, slot, 0)].to(ty)
    rows = rows.masked_fill_(~held[..., None], 0.0)  # [N, cap, d]
    at = n - S + torch.arange(S, device=q.device)[None, :]
    seen = (pos[None, None, :] <= at[..., None])[:, :, None, :]
    z = torch.matmul(q.to(ty).view(N, S * H, d), rows.transpose(1, 2).contiguous()).view(N, S, H, cap)
    return z.mul_(s["scale"]).masked_fill_(~seen, -math.inf), seen, rows


def _plain_shared(s):
    q, dl = s["q"], s["dl"]
    N, S, H, d = q.shape
    z, seen, rows = _own_scores(s, torch.float32)
    m = z.amax(-1, keepdim=True)
    # a token before position 0 is none: it sees no prefix either
    real = (s["lens"][:, None] - S + torch.arange(S, device=q.device)[None, :] >= 0)[:, :, None, None]
    starts, flat = s["starts"].tolist(), s["cache"].view(-1, d)
    prefix = []
    for i, (lo, hi) in enumerate(zip(starts, starts[1:])):
        r = flat[_held(s["prefix_table"][i:i + 1], s["prefix_lens"][i:i + 1], s["page"])].float()
        zp = torch.matmul(q[lo:hi].float().reshape(-1, d), r.t().contiguous()).mul_(s["scale"]).view(hi - lo, S, H, len(r))
        zp = zp.masked_fill_(~real[lo:hi], -math.inf)
        if zp.numel():
            m[lo:hi] = torch.maximum(m[lo:hi], zp.amax(-1, keepdim=True))
        prefix.append((lo, hi, zp, r))
    m = torch.where(m == -math.inf, 0.0, m)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(N, S * H, -1), rows[..., :dl].contiguous()).view(N, S, H, dl)
    for lo, hi, zp, r in prefix:
        p = zp.sub_(m[lo:hi]).exp_()
        l[lo:hi] += p.sum(-1, keepdim=True)
        o[lo:hi] += torch.matmul(p.view((hi - lo) * S * H, len(r)), r[:, :dl].contiguous()).view(hi - lo, S, H, dl)
    o = o / torch.where(l == 0, 1.0, l)
    return {"o": o.to(q.dtype), "lse": (m + l.log()).squeeze(-1)}


def _plain_verify(s):
    z, draft, u, zq = s["logits"], s["draft"].long(), s["uniforms"].double(), s["draft_logits"]
    N, S1, V = z.shape
    S, dev = S1 - 1, z.device
    L = torch.full((N,), S, device=dev) if s["draft_lens"] is None else s["draft_lens"].long()
    heat = s["temperature"].double()
    greedy = heat <= 0
    t = torch.where(greedy, 1.0, heat)[:, None, None]
    p = torch.softmax(z.double() / t, -1)
    q = None if zq is None else torch.softmax(zq.double() / t, -1)
    best = z.float().argmax(-1)
    px = p[:, :S].gather(2, draft[..., None])[..., 0]
    qx = torch.ones_like(px) if q is None else q.gather(2, draft[..., None])[..., 0]
    good = torch.where(greedy[:, None], draft == best[:, :S], u[:, :S] * qx < px)
    good = good & (torch.arange(S, device=dev)[None, :] < L[:, None])
    accepted = torch.cumprod(good.long(), 1).sum(1)
    row = torch.arange(N, device=dev)
    left = p[row, accepted]
    lost = accepted < L
    at = accepted.clamp(max=max(S - 1, 0))
    if q is None:
        less = torch.zeros_like(left).scatter_(1, draft[row, at][:, None], math.inf)
    else:
        less = q[row, at]
    left = torch.where(lost[:, None], (left - less).clamp(min=0.0), left)
    c = torch.cumsum(left, 1)
    drawn = torch.searchsorted(c, u[:, S:] * c[:, -1:], right=True)[:, 0].clamp(max=V - 1)
    drawn = torch.where(greedy, best[row, accepted], drawn)
    i = torch.arange(S1, device=dev)[None, :]
    tokens = torch.where(i < accepted[:, None], torch.cat([draft, draft[:, :1]], 1),
                         torch.where(i == accepted[:, None], drawn[:, None], -1))
    lp = p.log_().gather(2, tokens.clamp(min=0)[..., None])[..., 0]
    return {"accepted": accepted.to(torch.int32), "tokens": tokens.to(torch.int32),
            "logprobs": torch.where(tokens >= 0, lp, 0.0).float()}


def _plain_commit(s):
    h = s["h"].clone()
    A = -s["A_log"].exp()
    for t in range(s["S"]):
        k, v, beta = s["k"][:, t].float(), s["v"][:, t].float(), s["beta"][:, t, :, None]
        alpha = (s["g"][:, t] * A).exp()[..., None]
        u = (k[..., None] * h).sum(-2)
        w = beta * (v - alpha * u)
        new = alpha[..., None] * h + k[..., None] * w[..., None, :]
        h = torch.where((t < s["counts"])[:, None, None, None], new, h)
    return {"h": h}


def _plain_weights(s):
    N, S = s["q"].shape[:2]
    z, seen, _ = _own_scores(s, torch.float32)
    lse = s["lse"][..., None]
    w = torch.where(seen & (lse != -math.inf), z.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_(), 0.0).sum((1, 2))
    page, pos = s["page"], torch.arange(z.shape[-1], device=z.device)
    known = (s["lens"] - S if s["known"] is None else s["known"]).long()
    inside = pos[None, :] < s["lens"][:, None]
    slot = (s["table"].long().repeat_interleave(page, 1) * page + pos % page)[inside]
    flat = s["weights"].view(-1)
    old = torch.where((pos[None, :] < known[:, None])[inside], flat[slot] * s["decay"], 0.0)
    flat[slot] = old + w[inside]
    return {"weights": s["weights"]}


def _plain_trim_into(s, new):
    lens, table, stack, page = s["lens"].long(), s["table"], s["stack"], s["page"]
    held, left = (lens + page - 1) // page, (new.long().clamp(min=0).minimum(lens) + page - 1) // page
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    back = table[(col >= left[:, None]) & (col < held[:, None])]  # in order of the sequences and columns
    n = s["n_free"].long()
    at = n + torch.arange(back.numel(), device=table.device)
    stack[at] = back
    return (n + back.numel()).to(torch.int32)


def _plain_trim(s):
    n_free = _plain_trim_into(s, s["new_lens"])
    return {"free_pages": s["stack"], "n_free": n_free}


def _plain_evict(s):
    page, table, lens = s["page"], s["table"], s["lens"].long()
    pos = torch.arange(table.shape[1] * page, device=table.device)[None, :]
    slot = table.long().repeat_interleave(page, 1) * page + pos % page
    inside = pos < lens[:, None]
    keep = s["keep"].long().clamp(min=0).minimum(lens)
    first = keep.clamp(max=s["first"])
    recent = (keep - first).clamp(max=s["recent"])
    flat_w, flat_c = s["weights"].view(-1), s["cache"].view(-1, s["cache"].shape[-1])
    w = flat_w[torch.where(inside, slot, 0)]
    sure = (pos < first[:, None]) | (pos >= (lens - recent)[:, None])
    w = torch.where(inside, torch.where(sure, math.inf, w), -1.0)
    rank = torch.sort(w, dim=1, descending=True, stable=True).indices.argsort(1)
    stay = inside & (rank < keep[:, None])
    to = torch.cumsum(stay, 1) - 1
    src = slot[stay]
    dst = slot.gather(1, to.clamp(min=0))[stay]
    flat_w[dst] = flat_w[src]
    flat_c[dst] = flat_c[src]
    lens = keep.to(torch.int32)
    n_free = _plain_trim_into(s, lens)
    return {"weights": s["weights"], "cache": s["cache"], "lens": lens, "free_pages": s["stack"], "n_free": n_free}


_plain = {"shared": _plain_shared, "verify": _plain_verify, "commit": _plain_commit, "weights": _plain_weights,
          "evict": _plain_evict, "trim": _plain_trim}
_own = {"shared": _own_shared, "verify": _own_verify, "commit": _own_commit, "weights": _own_weights,
        "evict": _own_evict, "trim": _own_trim}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    """Bytes read and written once and operations of one pass."""
    op = case["op"]
    if op == "trim":
        return {"bytes": 4 * (2 * case["N"] + 2 * case["N"] * min(case["drop"], case["most"]) / 2 / case["page"]),
                "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "verify":  # every row up to the end of each draft, about twelve operations for an exponential and its sum
        rows = case["N"] * ((case["S"] / 2 if case["ragged"] else case["S"]) * (2 if case["q"] else 1) + 1)
        return {"bytes": e * rows * case["V"], "flops": 12 * rows * case["V"]}
    if op == "commit":
        N, S, H, dk, dv = (case[n] for n in ("N", "S", "H", "dk", "dv"))
        return {"bytes": N * H * (8 * dk * dv + S / 2 * (e * (dk + dv) + 8)), "flops": N * H * S / 2 * 5 * dk * dv}
    d, tokens = case["dl"] + case["dr"], sum(_spread(case["N"], case["most"]))
    if op == "shared":
        M, G = case["N"] * case["S"] * case["H"], case["G"]
        plens = [case["prefix"] - case["prefix"] * i // (2 * G) for i in range(G)]
        per = _groups(case["N"], G)
        pairs = tokens * case["S"] * case["H"] + sum(  # (which length goes to which group is drawn: their mean)
            sum(plens) / G * (hi - lo) * case["S"] * case["H"] for lo, hi in zip(per, per[1:]))
        return {"bytes": e * ((tokens + sum(plens)) * d + M * (d + case["dl"])) + 4 * M,
                "flops": 2 * pairs * (d + case["dl"])}
    if op == "weights":
        M = case["N"] * case["S"] * case["H"]
        return {"bytes": e * (tokens * d + M * d) + 4 * (2 - case["fresh"]) * tokens + 4 * M,
                "flops": 2 * tokens * case["S"] * case["H"] * d}
    kept = sum(min(x, case["keep"]) for x in _spread(case["N"], case["most"]) if x > case["keep"])
    return {"bytes": 2 * kept * (e * d + 4) + 4 * tokens, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits (None: whole numbers only)."""
    op = case["op"]
    if op == "trim":
        return None
    s = prepare(case, seed)
    return {"shared": _exact_shared, "verify": _exact_verify, "commit": _exact_commit, "weights": _exact_weights, "evict": _exact_evict}[op](s)


def _rows_of(table, n, page):
    """Slots of the first n rows of one sequence."""
    pages = table[: -(-n // page)].long()
    return (pages[:, None] * page + torch.arange(page, device=table.device)[None, :]).reshape(-1)[:n]


def _exact_shared(s):
    N, S, H, d = s["q"].shape
    dl, page, flat = s["dl"], s["page"], s["cache"].view(-1, d)
    o = torch.zeros(N, S, H, dl, dtype=torch.float64, device=DEV)
    lse = torch.full((N, S, H), -math.inf, dtype=torch.float64, device=DEV)
    starts, plens = s["starts"].tolist(), s["prefix_lens"].tolist()
    group = {n: g for g in range(len(plens)) for n in range(starts[g], starts[g + 1])}
    fronts = [flat[_rows_of(s["prefix_table"][g], plens[g], page)].double() for g in range(len(plens))]
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        own_rows = flat[_rows_of(s["table"][i], n, page)].double()
        front = fronts[group[i]] if i in group else own_rows[:0]
        rows = torch.cat([front, own_rows])
        for t in range(S):
            end = n - S + t + 1  # own rows this token sees
            if end < 1:
                continue
            r = rows[: len(front) + end]
            w = torch.softmax(s["q"][i, t].double() @ r.T * s["scale"], -1)
            o[i, t] = w @ r[:, :dl]
            lse[i, t] = torch.logsumexp(s["q"][i, t].double() @ r.T * s["scale"], -1)
    return {"o": o, "lse": lse}


def _exact_verify(s):
    """The log-probabilities of the tokens that a loop over the sequences accepts and draws."""
    N, S1, V = s["logits"].shape
    out = torch.zeros(N, S1, dtype=torch.float64, device=DEV)
    for n in range(N):
        heat = float(s["temperature"][n])
        t = heat if heat > 0 else 1.0
        length = S1 - 1 if s["draft_lens"] is None else int(s["draft_lens"][n])
        logp = torch.log_softmax(s["logits"][n].double() / t, -1)
        u, taken = s["uniforms"][n].double(), 0
        while taken < length:
            x = int(s["draft"][n, taken])
            logq = None if s["draft_logits"] is None else torch.log_softmax(s["draft_logits"][n, taken].double() / t, -1)
            if heat <= 0:
                fine = x == int(logp[taken].argmax())
            else:
                fine = bool(u[taken].log() + (0.0 if logq is None else logq[x]) < logp[taken, x])
            if not fine:
                break
            out[n, taken] = logp[taken, x]
            taken += 1
        p = logp[taken].exp()
        if taken < length:
            p = p.clone()
            if logq is None:
                p[x] = 0.0
            else:
                p = (p - logq.exp()).relu()
        if heat <= 0:
            x = int(logp[taken].argmax())
        else:
            ends = p.cumsum(0)
            x = int((ends <= u[-1] * ends[-1]).sum().clamp(max=V - 1))
        out[n, taken] = logp[taken, x]
    return {"accepted": None, "tokens": None, "logprobs": out}


def _exact_commit(s):
    h = s["h"].double()
    a = -torch.exp(s["A_log"].double())
    eye = torch.eye(h.shape[2], dtype=torch.float64, device=DEV)
    for i, c in enumerate(s["counts"].tolist()):
        for t in range(c):
            k, v, b = s["k"][i, t].double(), s["v"][i, t].double(), s["beta"][i, t].double()[:, None, None]
            keep = torch.exp(s["g"][i, t].double() * a)[:, None, None] * (eye - b * k[:, :, None] * k[:, None, :])
            h[i] = keep @ h[i] + b * k[:, :, None] * v[:, None, :]
    return {"h": h}


def _exact_weights(s):
    N, S, H, d = s["q"].shape
    out = s["weights"].double().view(-1)
    flat = s["cache"].view(-1, d)
    for i, n in enumerate(s["lens"].tolist()):
        slots = _rows_of(s["table"][i], n, s["page"])
        z = s["q"][i].double().reshape(S * H, d) @ flat[slots].double().T * s["scale"]
        last = torch.arange(S, device=DEV).repeat_interleave(H) + n - S
        ok = (torch.arange(n, device=DEV)[None, :] <= last[:, None])
        w = torch.where(ok, torch.exp(z - s["lse"][i].double().reshape(-1, 1)), 0.0).sum(0)
        known = max(n - S, 0) if s["known"] is None else int(s["known"][i])
        old = out[slots] * float(s["decay"])
        old[known:] = 0.0
        out[slots] = old + w
    return {"weights": out.view(s["weights"].shape)}


def _exact_evict(s):
    weights, cache = s["weights"].double().view(-1), s["cache"].double().view(-1, s["cache"].shape[-1])
    for i, n in enumerate(s["lens"].tolist()):
        k = max(0, min(n, int(s["keep"][i])))
        if k == n:
            continue
        a = min(k, s["first"])
        b = min(k - a, s["recent"])
        slots = _rows_of(s["table"][i], n, s["page"])
        w = weights[slots[a:n - b]]
        best = torch.argsort(-w, stable=True)[: k - a - b] + a
        stay = torch.cat([torch.arange(a, device=DEV), best.sort().values, torch.arange(n - b, n, device=DEV)])
        weights[slots[:k]], cache[slots[:k]] = weights[slots[stay]], cache[slots[stay]]
    return {"weights": weights.view(s["weights"].shape), "cache": cache.view(s["cache"].shape), "lens": None,
            "free_pages": None, "n_free": None}
