"""Cases for the 8-bit cache and for scored decode attention: keys and values
quantised on their way into the sharded paged cache, read back out of it, and
attended there by one query per request; and decode attention whose scores are
capped, biased by distance, or limited to a window, a prefix and a document,
over the 16-bit, 32-bit and 8-bit caches.

``run`` computes each operator in its plain form, elementary torch operations
in 32 bits rounded once, or, with ``own`` set, through the package's calls.
Token x of a request lives in virtual block x // (bs*dcp); inside the virtual
block runs of ``il`` tokens go round the ranks, and each rank fills its page of
``bs`` tokens in order.  An 8-bit page holds e4m3 numbers and, for each head, a
scale of its keys and one of its values.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    plain = dict(cap=0.0, window=0, prefix=0, alibi=False, docs=False, sink=False)
    return [
        # a decode step's new tokens, each into the middle of a page
        dict(name="append_step", op="append", dtype="bf16", B=32, T=1, ctx=65536, Hkv=8, d=128,
             dcp=8, bs=16, il=1, fused=True, mix=1),
        # a chunk of four prompts
        dict(name="append_prompt", op="append", dtype="bf16", B=4, T=2048, ctx=9001, Hkv=8, d=128,
             dcp=8, bs=16, il=1, fused=True, mix=2),
        # ragged runs of 32-bit keys and values, three ranks, 64-wide heads, large pages
        dict(name="append_ragged", op="append", dtype="f32", B=16, T=37, ctx=777, Hkv=2, d=64,
             dcp=3, bs=64, il=4, fused=False, mix=3),
        # a short context read back for a chunk of its prompt
        dict(name="gather_short", op="gather", dtype="f32", B=1, T=1500, Hkv=8, d=128, dcp=2,
             bs=16, il=1, mix=4),
        # the contexts of eight requests, for prefill attention
        dict(name="gather_chunk", op="gather", dtype="bf16", B=8, T=8192, Hkv=8, d=128, dcp=8,
             bs=16, il=1, mix=5),
        # one user's short chat over the 8-bit cache: the latency of a call
        dict(plain, name="q8_one", op="q8", dtype="bf16", B=1, ctx=1500, even=True, Hq=32, Hkv=8,
             d=128, dcp=2, bs=16, il=1, mix=6),
        # a serving batch with mixed contexts
        dict(plain, name="q8_b32", op="q8", dtype="bf16", B=32, ctx=65536, even=False, Hq=32,
             Hkv=8, d=128, dcp=8, bs=16, il=1, mix=7),
        # one long document beside a short request, capped scores and a sink
        dict(plain, name="q8_tail", op="q8", dtype="bf16", B=2, ctx=524288, even=False, Hq=32,
             Hkv=8, d=128, dcp=8, bs=64, il=1, mix=8, cap=30.0, sink=True),
        # a window with the first tokens kept, over capped scores: a 16-bit cache
        dict(plain, name="scored_window", op="scored", dtype="bf16", B=32, ctx=65536, even=False,
             Hq=32, Hkv=8, d=128, dcp=8, bs=16, il=1, mix=9, cap=50.0, window=4096, prefix=4),
        # biased by distance over whole contexts, one query head for each key/value head
        dict(plain, name="scored_bias", op="scored", dtype="bf16", B=16, ctx=16384, even=False,
             Hq=8, Hkv=8, d=128, dcp=4, bs=32, il=1, mix=10, alibi=True),
        # packed documents, one shared key/value head, 64-wide heads, three ranks, odd lengths
        dict(plain, name="scored_docs", op="scored", dtype="bf16", B=16, ctx=9001, even=False,
             Hq=16, Hkv=1, d=64, dcp=3, bs=32, il=4, mix=11, docs=True, alibi=True, cap=20.0),
        # the 32-bit cache
        dict(plain, name="scored_f32", op="scored", dtype="f32", B=2, ctx=3001, even=False, Hq=8,
             Hkv=2, d=64, dcp=2, bs=16, il=1, mix=12, cap=30.0, alibi=True, window=2000, sink=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], dict(bytes=0.0, flops=0.0))
        m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    op = rng.choice(["append", "append", "gather", "q8", "q8", "q8", "scored", "scored", "scored"])
    bs = rng.choice([16, 32, 64])
    f32 = rng.random() < 0.2
    c = dict(op=op, dtype="f32" if f32 else "bf16", dcp=rng.choice([1, 2, 3, 4, 8]), bs=bs,
             il=rng.choice([1, 4, 16, bs]), d=rng.choice([64, 128, 128]), mix=rng.randrange(1 << 20))
    if op == "append":
        c.update(B=_log(rng, 1, 32), T=_log(rng, 1, 2048), ctx=_log(rng, 1, 65536),
                 Hkv=rng.choice([1, 2, 8, 8]), fused=rng.random() < 0.5)
        shrink = ("T", "B")
    elif op == "gather":
        c.update(B=_log(rng, 1, 8), T=_log(rng, 1, 8192), Hkv=rng.choice([1, 2, 8, 8]))
        shrink = ("T", "B")
    else:
        Hq, Hkv = rng.choice([(32, 8), (32, 8), (16, 2), (8, 2), (16, 1), (8, 8)])
        c.update(B=_log(rng, 1, 4 if f32 else 32), ctx=_log(rng, 1, 8192 if f32 else 65536),
                 even=rng.random() < 0.2, Hq=Hq, Hkv=Hkv, sink=rng.random() < 0.3,
                 cap=rng.choice([0.0, 0.0, 20.0, 50.0]), alibi=rng.random() < 0.3,
                 docs=rng.random() < 0.25, window=_log(rng, 1, 8192) if rng.random() < 0.4 else 0)
        c["prefix"] = rng.choice([0, 1, 4, 100]) if c["window"] else 0
        shrink = ("ctx", "B")
        if f32:
            most[op] = {k: v / 64 for k, v in most[op].items()}
    while any(work(c)[k] > most[op][k] for k in ("bytes", "flops")):
        k = max(shrink, key=c.get)
        c[k] = max(1, c[k] * 2 // 3)
    return c


def _lens(c):
    """Contexts of the requests: the first is the longest."""
    r = random.Random(c["mix"])
    if c["even"]:
        return [c["ctx"]] * c["B"]
    return [c["ctx"]] + [_log(r, max(1, c["ctx"] // 16), c["ctx"]) for _ in range(c["B"] - 1)]


def _seen(c):
    """Of each request: its length, the first token of its last document, the first token of the
    window, and the tokens from the document's start that are seen anyhow."""
    r, out = random.Random(c["mix"] + 1), []
    for n in _lens(c):
        lo = r.randrange(0, n) if c["docs"] else 0
        w = max(lo, n - c["window"]) if c["window"] else lo
        out.append((n, lo, w, min(lo + c["prefix"], w)))
    return out


def _runs(c):
    """Cached and new tokens of each request of an append."""
    r = random.Random(c["mix"])
    T = [c["T"]] + [r.randint(max(1, c["T"] // 2), c["T"]) for _ in range(c["B"] - 1)]
    return [c["ctx"]] + [r.randrange(0, c["ctx"] + 1) for _ in range(c["B"] - 1)], T


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        N, row = sum(_runs(c)[1]), c["Hkv"] * c["d"]
        return dict(bytes=float(2 * N * row * (es + 1) + 8 * N * c["Hkv"] / c["bs"] + 8 * c["B"]),
                    flops=0.0)
    if c["op"] == "gather":
        N, row = c["B"] * c["T"], c["Hkv"] * c["d"]
        return dict(bytes=float(2 * N * row * (es + 1) + 8 * N * c["Hkv"] / c["bs"] + 12 * N),
                    flops=0.0)
    seen = sum(n - w + p - lo for n, lo, w, p in _seen(c))
    row = 2 * c["Hkv"] * c["d"] * (1 if c["op"] == "q8" else es)
    scales = 8 * seen * c["Hkv"] / c["bs"] if c["op"] == "q8" else 0
    return dict(bytes=float(seen * row + scales + c["B"] * c["Hq"] * (2 * c["d"] * es + 4)),
                flops=float(4 * c["Hq"] * c["d"] * seen))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _place(x, c):
    """Rank, virtual block and place in the rank's page of tokens x."""
    vbs = c["bs"] * c["dcp"]
    vb, off = x // vbs, x % vbs
    run = off // c["il"]
    return run % c["dcp"], vb, run // c["dcp"] * c["il"] + off % c["il"]


def _two_to(e):
    """2**e by its bits: a power may be off by a step, and ties go by it."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, dtype, g):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


def _tables(lens, c, g, spare=3):
    """Block tables [dcp, B, VB] over randomly placed pages of each rank, and the pages' number."""
    vbs = c["bs"] * c["dcp"]
    n = torch.tensor([-(-L // vbs) for L in lens], device="cuda")
    VB, nb = int(n.max()), int(n.sum()) + spare
    used = torch.arange(VB, device="cuda") < n[:, None]
    bt = torch.full((c["dcp"], len(lens), VB), -1, dtype=torch.int32, device="cuda")
    perm = torch.argsort(torch.rand((c["dcp"], nb), device="cuda", generator=g), 1)
    bt[:, used] = perm[:, :nb - spare].to(torch.int32)
    return bt, nb


def _cache8(c, nb, g):
    """Pools of quantised normal numbers, whose pages are of unlike sizes, and the pages' scales."""
    shape = (c["dcp"], nb, c["Hkv"], c["bs"], c["d"])
    k, v = ((_normal(shape, torch.bfloat16, g) * 64).to(E4M3) for _ in range(2))
    sc = torch.zeros((c["dcp"], nb, c["Hkv"], 4), device="cuda")
    up = torch.randint(-1, 2, (c["dcp"], nb, c["Hkv"], 2), device="cuda", generator=g)
    sc[..., :2] = _two_to(up - 6)
    return dict(k=k, v=v, sc=sc)


def _prepare_append(c, g):
    ctx, T = _runs(c)
    N, H, d = sum(T), c["Hkv"], c["d"]
    bt, nb = _tables([x + t for x, t in zip(ctx, T)], c, g)
    # a token now and then is several times the others, as in real layers
    big = torch.where(torch.rand((N, 1, 1), device="cuda", generator=g) < 0.05, 6.0, 1.0)
    if c["fused"]:  # the output of one projection; k and v are views of it
        qkv = (_normal((N, 4 * H + 2 * H, d), torch.float32, g) * big).to(DT[c["dtype"]])
        _, k, v = qkv.split([4 * H, H, H], 1)
    else:
        k, v = ((_normal((N, H, d), torch.float32, g) * big).to(DT[c["dtype"]]) for _ in range(2))
    s = _cache8(c, nb, g)
    return dict(kp=s["k"], vp=s["v"], sc=s["sc"], bt=bt, nb=nb, new_k=k, new_v=v,
                start=torch.tensor([0] + T).cumsum(0).to("cuda", torch.int32),
                ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"))


def _prepare_gather(c, g):
    bt, nb = _tables([c["T"]] * c["B"], c, g)
    t = torch.arange(c["B"] * c["T"], device="cuda")
    return dict(_cache8(c, nb, g), bt=bt, nb=nb, req=(t // c["T"]).to(torch.int32), pos=t % c["T"])


def _prepare_decode(c, g):
    lens, dt = _lens(c), DT[c["dtype"]]
    bt, nb = _tables(lens, c, g)
    if c["op"] == "q8":
        s = _cache8(c, nb, g)
    else:
        shape = (c["dcp"], nb, c["Hkv"], c["bs"], c["d"])
        s = dict(k=_normal(shape, dt, g), v=_normal(shape, dt, g))
    first = torch.tensor([lo for _, lo, _, _ in _seen(c)], dtype=torch.int32, device="cuda")
    slopes = 2.0 ** (-8.0 * torch.arange(1, c["Hq"] + 1, device="cuda") / c["Hq"])
    return dict(s, q=_normal((c["B"], c["Hq"], c["d"]), dt, g), bt=bt, nb=nb, longest=max(lens),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                first=first if c["docs"] else None, slopes=slopes if c["alibi"] else None,
                sink=_normal((c["Hq"],), torch.float32, g) if c["sink"] else None,
                scale=c["d"] ** -0.5)


def prepare(case, seed):
    g = _gen(seed)
    s = {"append": _prepare_append, "gather": _prepare_gather, "q8": _prepare_decode,
         "scored": _prepare_decode}[case["op"]](case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _handles(s):
    """The layout, the cache and the score form that a program makes once and keeps."""
    if "lib" not in s:
        import context_paged_decode_gb300 as dcp

        c = s["case"]
        s["layout"] = dcp.Layout(c["dcp"], c["bs"], c["il"])
        if c["op"] == "append":
            s["kv"] = dcp.PagedKV8(list(s["kp"]), list(s["vp"]), list(s["sc"]), s["bt"], s["nb"])
        elif c["op"] == "scored":
            s["kv"] = dcp.PagedKV(list(s["k"]), list(s["v"]), s["bt"], s["nb"])
        else:
            s["kv"] = dcp.PagedKV8(list(s["k"]), list(s["v"]), list(s["sc"]), s["bt"], s["nb"])
        if c["op"] in ("q8", "scored"):
            s["form"] = dcp.Scores(cap=c["cap"], window=c["window"], prefix=c["prefix"],
                                   slopes=s["slopes"], first=s["first"])
        s["lib"] = dcp
    return s["lib"], s["layout"]


def _own_append(s):
    dcp, L = _handles(s)
    dcp.q8_append_gqa(L, s["new_k"], s["new_v"], s["kv"], s["start"], s["ctx"])
    return s["kp"], s["vp"], s["sc"]


def _own_gather(s):
    dcp, L = _handles(s)
    return dcp.q8_gather_gqa(L, s["kv"], s["req"], s["pos"], dtype=DT[s["case"]["dtype"]])


def _own_q8(s):
    dcp, L = _handles(s)
    return dcp.q8_decode_gqa(L, s["q"], s["kv"], s["lens"], s["scale"], scores=s["form"],
                             sink=s["sink"])


def _own_scored(s):
    dcp, L = _handles(s)
    return dcp.scored_decode_gqa(L, s["q"], s["kv"], s["lens"], s["scale"], s["form"],
                                 sink=s["sink"])


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _to8(x):
    """The bytes of x in e4m3."""
    return x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _rows(pool, *at):
    """Entries of a pool in 32 bits."""
    if pool.dtype == E4M3:
        return pool.view(torch.uint8)[at].view(E4M3).float()
    return pool[at].float()


def _need(top):
    """The smallest power of two, 2^-60 at least, by which entries up to `top` fit into e4m3."""
    m, e = torch.frexp(top)
    e = torch.where(top == 0, -60, e - 9 + (m > 0.875))
    return _two_to(e.clamp(min=-60))


def _written(x, pool, sc, which, pid, rank, page, loc):
    """Rows x [N, H, d] into the pages of one pool, and the pages' scales."""
    dcp, nb, H = pool.shape[:3]
    x = x.float()
    size = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)                     # [N, H]
    top = torch.zeros((dcp * nb, H), device="cuda")
    top.scatter_reduce_(0, pid[:, None].expand(-1, H), size, "amax")
    low = torch.full((dcp * nb,), pool.shape[3], device="cuda", dtype=torch.int64)
    low.scatter_reduce_(0, pid, loc, "amin")
    old = sc[..., which].reshape(dcp * nb, H)[pid]                              # [N, H]
    old = torch.where((low[pid] > 0)[:, None] & old.isfinite() & (old > 0), old, 0.0)
    new = torch.maximum(old, _need(top[pid]))
    # the other places of a page whose scale grows
    more = torch.where((old > 0) & (new > old), old / new, 1.0)
    held = pool.view(torch.uint8)
    held[rank, page] = _to8(_rows(pool, rank, page) * more[..., None, None])
    held[rank, page, :, loc] = _to8(x / new[..., None])
    sc[rank, page, :, which] = new


def _plain_append(s):
    c = s["case"]
    t = torch.arange(s["new_k"].shape[0], device="cuda")
    req = torch.searchsorted(s["start"].long(), t, right=True) - 1
    rank, vb, loc = _place(s["ctx"][req].long() + t - s["start"][req], c)
    page = s["bt"][rank, req, vb].long()
    pid = rank * s["nb"] + page
    _written(s["new_k"], s["kp"], s["sc"], 0, pid, rank, page, loc)
    _written(s["new_v"], s["vp"], s["sc"], 1, pid, rank, page, loc)
    return s["kp"], s["vp"], s["sc"]


def _plain_gather(s):
    c = s["case"]
    rank, vb, loc = _place(s["pos"], c)
    page = s["bt"][rank, s["req"].long(), vb].long()
    sc = s["sc"][rank, page]
    return tuple((_rows(p, rank, page, slice(None), loc) * sc[..., i, None]).to(DT[c["dtype"]])
                 for i, p in enumerate((s["k"], s["v"])))


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    x = torch.arange(s["longest"], device="cuda")
    rank, vb, loc = _place(x, c)
    page = s["bt"][rank, :, vb].t().long().clamp(min=0)                         # [B, L]
    k = _rows(s["k"], rank, page, slice(None), loc)                             # [B, L, Hkv, d]
    v = _rows(s["v"], rank, page, slice(None), loc)
    if c["op"] == "q8":
        sc = s["sc"][rank, page]
        k, v = k * sc[..., 0, None], v * sc[..., 1, None]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    e = (q @ k.permute(0, 2, 3, 1) * s["scale"]).view(B, Hq, -1)
    if c["cap"]:
        e = c["cap"] * torch.tanh(e / c["cap"])
    n = s["lens"].long()[:, None]
    if s["slopes"] is not None:
        e = e - s["slopes"][:, None] * (n - 1 - x).float()[:, None]
    lo = s["first"].long()[:, None] if s["first"] is not None else torch.zeros_like(n)
    w = torch.maximum(lo, n - c["window"]) if c["window"] else lo
    seen = (x < n) & (x >= lo) & ((x >= w) | (x < lo + c["prefix"]))            # [B, L]
    e = e.masked_fill(~seen[:, None], -math.inf)
    top = e.amax(-1, keepdim=True)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"][:, None])
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(e - top)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][:, None] - top)
    o = p.view(B, Hkv, Hq // Hkv, -1) @ v.transpose(1, 2)
    o = o.view(B, Hq, d) / torch.where(total == 0, 1.0, total)
    return o.to(s["q"].dtype), (top + torch.log(total)).squeeze(-1)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "gather": _own_gather, "q8": _own_q8,
                "scored": _own_scored}[op](state)
    return {"append": _plain_append, "gather": _plain_gather, "q8": _plain_decode,
            "scored": _plain_decode}[op](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, request by request and page by page
# ---------------------------------------------------------------------------

def _two_to_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest8(y):
    """The e4m3 numbers nearest to y, ties to even, as 64-bit numbers."""
    y = y.clamp(-448.0, 448.0)
    step = _two_to_64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(y / step) * step


def _pages_of(c, s, b, n):
    """Request b's pages on each rank in order, and the token of each place in them."""
    slots = torch.arange(c["bs"], device="cuda")
    for r in range(c["dcp"]):
        pages = s["bt"][r, b][s["bt"][r, b] >= 0].long()
        block = torch.arange(pages.numel(), device="cuda")[:, None] * c["bs"] * c["dcp"]
        yield r, pages, block + (slots // c["il"] * c["dcp"] + r) * c["il"] + slots % c["il"]


def _exact_append(c, s):
    ctx, T = _runs(c)
    kp, vp, sc = s["kp"].double(), s["vp"].double(), s["sc"].double()
    at = 0
    for b, (n, t) in enumerate(zip(ctx, T)):
        for r, pages, x in _pages_of(c, s, b, n + t):
            fresh = (x >= n) & (x < n + t)                                       # [pages, bs]
            hit = fresh.any(1)
            ids, mine, tok = pages[hit], fresh[hit], (x[hit] - n).clamp(0, t - 1) + at
            for pool, rows, i in ((kp, s["new_k"], 0), (vp, s["new_v"], 1)):
                y = rows[tok].double().transpose(1, 2)                           # [P, H, bs, d]
                top = torch.where(mine[:, None, :, None], y.abs(), 0.0).amax((2, 3))
                up = (torch.arange(-60, 121, device="cuda")[:, None, None])
                fits = _two_to_64(up) * 448.0 >= top
                up = up[fits.to(torch.int8).argmax(0), 0, 0]
                held = torch.where(mine[:, :1], 0.0, sc[r, ids, :, i])
                new = torch.maximum(held, _two_to_64(up))
                kept = pool[r, ids]
                grown = ((held > 0) & (new > held))[..., None, None]
                kept = torch.where(grown, _nearest8(kept * (held / new)[..., None, None]), kept)
                pool[r, ids] = torch.where(mine[:, None, :, None],
                                           _nearest8(y / new[..., None, None]), kept)
                sc[r, ids, :, i] = new
        at += t
    return kp, vp, sc


def _context(c, s, b, n):
    """Keys and values of request b in 64 bits, [Hkv, n, d]."""
    k = torch.zeros((c["Hkv"], n, c["d"]), dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    for r, pages, x in _pages_of(c, s, b, n):
        keep = x.flatten() < n
        for name, to, i in (("k", k, 0), ("v", v, 1)):
            rows = _rows(s[name], r, pages).double()
            if "sc" in s:
                rows = rows * s["sc"][r, pages, :, i, None, None].double()
            rows = rows.transpose(0, 1).reshape(c["Hkv"], -1, c["d"])
            to[:, x.flatten()[keep]] = rows[:, keep]
    return k, v


def _exact_gather(c, s):
    ks, vs = zip(*(_context(c, s, b, c["T"]) for b in range(c["B"])))
    return tuple(torch.cat(x, 1).transpose(0, 1).contiguous() for x in (ks, vs))


def _exact_decode(c, s):
    o = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], c["Hq"]), dtype=torch.float64, device="cuda")
    for b, (n, lo, w, p) in enumerate(_seen(c)):
        k, v = _context(c, s, b, n)
        x = torch.cat([torch.arange(lo, p), torch.arange(w, n)]).cuda()
        for h in range(c["Hq"]):
            g = h * c["Hkv"] // c["Hq"]
            e = k[g, x] @ s["q"][b, h].double() * c["d"] ** -0.5
            if c["cap"]:
                e = c["cap"] * torch.tanh(e / c["cap"])
            if c["alibi"]:
                e = e - s["slopes"][h].double() * (n - 1 - x)
            if c["sink"]:
                e = torch.cat([e, s["sink"][h].double().view(1)])
            lse[b, h] = torch.logsumexp(e, 0)
            o[b, h] = torch.exp(e - lse[b, h])[:x.numel()] @ v[g, x]
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "q8": _exact_decode,
            "scored": _exact_decode}[case["op"]](case, s)
