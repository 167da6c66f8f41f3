"""Cases for the cache-side operators of a serving step: attention of drafted
token trees over the sharded paged cache, rotary positions on the way into the
cache, the life of the cache's pages, and keeping the accepted drafted tokens.

``run`` computes each operator in its plain form, elementary torch operations
in 32 bits rounded once, or, with ``own`` set, through the package's calls.
Token x of a request lives in virtual block x // (bs*dcp); inside the virtual
block runs of ``il`` tokens go round the ranks, and each rank fills its page of
``bs`` tokens in order.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user, a short chat, eight drafted tokens: the latency of a call
        dict(name="tree_one", op="tree", dtype="bf16", B=1, T=8, ctx=1500, Hq=32, Hkv=8, d=128,
             dcp=2, bs=16, il=1, sink=False, mix=1),
        # a serving batch with mixed contexts and sixteen drafted tokens a request
        dict(name="tree_b32", op="tree", dtype="bf16", B=32, T=16, ctx=65536, Hq=32, Hkv=8, d=128,
             dcp=8, bs=16, il=1, sink=False, mix=2),
        # wide trees over long documents: 256 query rows for each key/value head
        dict(name="tree_wide", op="tree", dtype="bf16", B=8, T=64, ctx=65536, Hq=32, Hkv=8, d=128,
             dcp=8, bs=64, il=1, sink=False, mix=3),
        # one shared key/value head, 64-wide heads, three ranks, odd lengths, a sink
        dict(name="tree_mqa", op="tree", dtype="bf16", B=16, T=5, ctx=9001, Hq=16, Hkv=1, d=64,
             dcp=3, bs=32, il=4, sink=True, mix=4),
        # the 32-bit cache
        dict(name="tree_f32", op="tree", dtype="f32", B=2, T=11, ctx=3001, Hq=8, Hkv=2, d=64,
             dcp=2, bs=16, il=1, sink=True, mix=5),
        # the drafted tokens of a decode step: 32 requests, 8 tokens each
        dict(name="rope_step", op="rope", dtype="bf16", T=256, Hq=32, Hkv=8, d=128, rot=128,
             axes=1, pairs="halves", dcp=8, bs=16, il=1, far=131072),
        # a prompt chunk with images and video: three axes, read out of one fused projection
        dict(name="rope_prompt", op="rope", dtype="bf16", T=8192, Hq=32, Hkv=8, d=128, rot=128,
             axes=3, pairs="halves", dcp=8, bs=16, il=1, far=131072),
        # latent rows: 64 rotated entries behind 512 others, adjacent pairs, odd token count
        dict(name="rope_latent", op="rope", dtype="bf16", T=1025, Hq=128, Hkv=0, d=576, rot=64,
             axes=1, pairs="adjacent", dcp=8, bs=64, il=1, far=262144),
        # a few samples of one prompt: free the old ones, fork, copy the open pages, grow
        dict(name="pages_few", op="pages", dtype="bf16", parents=2, fan=2, ctx=1000, grow=9, H=8,
             d=128, pools=2, dcp=2, bs=16, il=1, shared=False, mix=6),
        # many samples over long prompts
        dict(name="pages_many", op="pages", dtype="bf16", parents=16, fan=8, ctx=32001, grow=200,
             H=8, d=128, pools=2, dcp=8, bs=16, il=1, shared=False, mix=7),
        # the accepted tokens of a step, keys and values of four layers
        dict(name="compact_step", op="compact", dtype="bf16", B=32, T=16, keep=5, ctx=1500, H=8,
             d=128, pools=8, dcp=8, bs=16, il=1, mix=8),
        # the same over latent rows of sixteen layers, wide trees
        dict(name="compact_latent", op="compact", dtype="bf16", B=64, T=64, keep=9, ctx=777, H=1,
             d=576, pools=16, dcp=8, bs=64, il=64, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], dict(bytes=0.0, flops=0.0))
        m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    op = rng.choice(["tree", "tree", "tree", "rope", "rope", "pages", "compact"])
    bs = rng.choice([16, 32, 64])
    base = dict(op=op, dcp=rng.choice([1, 2, 3, 4, 8]), bs=bs, il=rng.choice([1, 4, 16, bs]))
    if op == "tree":
        f32 = rng.random() < 0.2
        Hq, Hkv = rng.choice([(32, 8), (32, 8), (16, 2), (8, 2), (16, 1), (8, 8)])
        c = dict(base, dtype="f32" if f32 else "bf16", Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128, 128]),
                 B=_log(rng, 1, 4 if f32 else 32), T=_log(rng, 1, 16 if f32 else 64),
                 ctx=_log(rng, 1, 8192 if f32 else 65536), sink=rng.random() < 0.3,
                 mix=rng.randrange(1 << 20))
        if f32:
            most[op] = {k: v / 64 for k, v in most[op].items()}
        while any(work(c)[k] > most[op][k] for k in ("bytes", "flops")):
            c["ctx"] = max(1, c["ctx"] * 2 // 3)
        return c
    if op == "rope":
        if rng.random() < 0.35:
            return dict(base, dtype="bf16", T=_log(rng, 1, 1025), Hq=rng.choice([16, 64, 128]),
                        Hkv=0, d=576, rot=64, axes=rng.choice([1, 3]), pairs="adjacent",
                        far=_log(rng, 4096, 1048576))
        d = rng.choice([64, 128, 128])
        Hq, Hkv = rng.choice([(32, 8), (16, 2), (8, 8)])
        f32 = rng.random() < 0.25
        return dict(base, dtype="f32" if f32 else "bf16", T=_log(rng, 1, 4096 if f32 else 8192),
                    Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]),
                    axes=rng.choice([1, 3, 4]), pairs=rng.choice(["halves", "halves", "adjacent"]),
                    far=_log(rng, 4096, 1048576))
    if op == "pages":
        c = dict(base, dtype="bf16", parents=_log(rng, 1, 16), fan=_log(rng, 1, 8),
                 ctx=_log(rng, 1, 32001), grow=rng.randrange(1, 201), H=rng.choice([1, 2, 8]),
                 d=128, pools=2, shared=rng.random() < 0.3, mix=rng.randrange(1 << 20))
    else:
        latent = rng.random() < 0.4
        T = _log(rng, 2, 64)
        c = dict(base, dtype="bf16", B=_log(rng, 1, 48), T=T, keep=rng.randrange(1, min(9, T) + 1),
                 ctx=_log(rng, 1, 1500), H=1 if latent else rng.choice([2, 8]),
                 d=576 if latent else 128, pools=_log(rng, 1, 8), mix=rng.randrange(1 << 20))
    while work(c)["bytes"] > most[op]["bytes"]:
        k = max(("parents", "fan", "pools") if op == "pages" else ("B", "pools"), key=c.get)
        c[k] = max(1, c[k] // 2)
    return c


def _tree_sizes(c):
    """Cached and drafted tokens of each request: the first has the most of both."""
    r = random.Random(c["mix"])
    ctx = [c["ctx"]] + [_log(r, max(1, c["ctx"] // 16), c["ctx"]) for _ in range(c["B"] - 1)]
    T = [c["T"]] + [r.randint(max(1, c["T"] // 2), c["T"]) for _ in range(c["B"] - 1)]
    return ctx, T


def _parent_lens(c):
    r = random.Random(c["mix"])
    return [max(1, c["ctx"] - r.randrange(0, max(1, c["ctx"] // 8))) for _ in range(c["parents"])]


def _kept(c):
    """For each request the accepted nodes, in order: node 0, then nodes that lie
    behind the kept prefix (so a second pass over the same cache changes nothing)."""
    r = random.Random(c["mix"])
    paths = []
    for _ in range(c["B"]):
        n = r.randint(1, min(c["keep"], max(1, (c["T"] + 1) // 2)))
        paths.append([0] + sorted(r.sample(range(n, c["T"]), n - 1)))
    ctx = [max(1, c["ctx"] - r.randrange(0, max(1, c["ctx"] // 4))) for _ in range(c["B"])]
    return ctx, paths


def _local(L, r, c):
    """Tokens of [0, L) that rank r holds."""
    vbs, turn = c["bs"] * c["dcp"], c["il"] * c["dcp"]
    full, rem = L // vbs, L % vbs
    return full * c["bs"] + rem // turn * c["il"] + min(max(rem % turn - r * c["il"], 0), c["il"])


def _open_pages(L, c):
    """Ranks whose last page of a length is not full, and of these the ones that hold a token."""
    vbs = c["bs"] * c["dcp"]
    if L % vbs == 0:
        return 0, 0
    if c["shared"]:
        return 1, c["dcp"]
    n = [_local(L, r, c) - L // vbs * c["bs"] for r in range(c["dcp"])]
    return sum(x < c["bs"] for x in n), sum(0 < x < c["bs"] for x in n)


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "tree":
        ctx, T = _tree_sizes(c)
        N, L = sum(T), sum(ctx) + sum(T)
        return dict(bytes=float(2 * L * c["Hkv"] * c["d"] * es + 2 * N * c["Hq"] * c["d"] * es
                                + N * (c["Hq"] * 4 + 8)),
                    flops=float(sum(4 * c["Hq"] * c["d"] * t * (x + t) for x, t in zip(ctx, T))))
    if c["op"] == "rope":
        heads = c["Hq"] + (2 * c["Hkv"] if c["Hkv"] else 1)
        turned = c["Hq"] + (c["Hkv"] or 1)
        return dict(bytes=float(2 * c["T"] * heads * c["d"] * es
                                + c["T"] * 8 * (c["axes"] + c["dcp"])),
                    flops=float(c["T"] * turned * c["rot"] * 3))
    if c["op"] == "pages":
        vbs, lens = c["bs"] * c["dcp"], _parent_lens(c)
        tables = 1 if c["shared"] else c["dcp"]
        entries = sum(c["fan"] * -(-(L + c["grow"]) // vbs) for L in lens) * tables
        copies = sum(c["fan"] * _open_pages(L, c)[1] for L in lens)
        page = c["H"] * c["bs"] * c["d"] * es
        # each table entry and count is read and written once as it is taken and once as it goes
        return dict(bytes=float(entries * 32 + copies * 2 * page * c["pools"]), flops=0.0)
    ctx, paths = _kept(c)
    moved = sum(sum(p != i for i, p in enumerate(q)) for q in paths)
    return dict(bytes=float(2 * moved * c["H"] * c["d"] * es * c["pools"] + 8 * sum(map(len, paths))
                            + 8 * c["B"]), flops=0.0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _place(x, c):
    """Rank, virtual block and place in the rank's page of tokens x."""
    vbs = c["bs"] * c["dcp"]
    vb, off = x // vbs, x % vbs
    run = off // c["il"]
    return run % c["dcp"], vb, run // c["dcp"] * c["il"] + off % c["il"]


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


def _prepare_tree(c, g):
    ctx, T = _tree_sizes(c)
    dt, N = DT[c["dtype"]], sum(T)
    bt, nb = _tables([x + t for x, t in zip(ctx, T)], c, g)
    shape = (c["dcp"], nb, c["Hkv"], c["bs"], c["d"])
    start = torch.tensor([0] + T).cumsum(0)
    node = torch.cat([torch.arange(t) for t in T]).tolist()
    r, mask = random.Random(int(torch.randint(1 << 40, (1,), device="cuda", generator=g))), []
    for j in node:  # a node sees itself and what its parent, an earlier node, sees
        first = len(mask) - j
        up = r.randrange(max(0, j - 4), j) if j else 0
        mask.append((mask[first + up] if j else 0) | 1 << j)
    mask = [m - (1 << 64) if m >> 63 else m for m in mask]
    return dict(q=_normal((N, c["Hq"], c["d"]), dt, g), k=_normal(shape, dt, g),
                v=_normal(shape, dt, g), bt=bt, nb=nb, start=start.to("cuda", torch.int32),
                ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                mask=torch.tensor(mask, dtype=torch.int64, device="cuda"),
                sink=_normal((c["Hq"],), torch.float32, g) if c["sink"] else None,
                scale=c["d"] ** -0.5, longest=max(x + t for x, t in zip(ctx, T)), T=max(T))


def _prepare_rope(c, g):
    dt, T, d = DT[c["dtype"]], c["T"], c["d"]
    half = c["rot"] // 2
    inv = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    pos = torch.randint(0, c["far"], (c["axes"], T), device="cuda", generator=g)
    axis = (torch.arange(half) * c["axes"] // half).to("cuda", torch.int32)
    # the tokens of up to 32 requests, each a run of positions, and their slots
    B = min(32, T)
    per = -(-T // B)
    vbs = c["bs"] * c["dcp"]
    lens = [per + vbs] * B
    bt, nb = _tables(lens, c, g)
    t = torch.arange(T, device="cuda")
    req, at = t // per, t % per + torch.randint(0, vbs, (B,), device="cuda", generator=g)[t // per]
    rank, vb, loc = _place(at, c)
    slot = torch.full((c["dcp"], T), -1, dtype=torch.int64, device="cuda")
    slot[rank, t] = bt[rank, req, vb].long() * c["bs"] + loc
    s = dict(pos=pos, inv=inv, axis=axis, slot=slot, nb=nb)
    if c["Hkv"]:
        # one fused projection's output; q, k and v are views of it
        qkv = _normal((T, c["Hq"] + 2 * c["Hkv"], d), dt, g)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
        s["kp"] = torch.zeros((c["dcp"], nb, c["Hkv"], c["bs"], d), dtype=dt, device="cuda")
        s["vp"] = torch.zeros_like(s["kp"])
    else:
        s["q"] = _normal((T, c["Hq"], d), dt, g)
        s["k"] = _normal((T, d), dt, g)
        s["kp"] = torch.zeros((c["dcp"], nb, c["bs"], d), dtype=dt, device="cuda")
    return s


def _prepare_pages(c, g):
    lens, vbs = _parent_lens(c), c["bs"] * c["dcp"]
    P, F = c["parents"], c["parents"] * c["fan"]
    if c["shared"]:
        bt, nb = _tables(lens, dict(c, dcp=1, bs=vbs), g, spare=0)
    else:
        bt, nb = _tables(lens, c, g, spare=0)
    VB = max(-(-(L + c["grow"]) // vbs) for L in lens)
    more = sum(c["fan"] * (-(-(L + c["grow"]) // vbs) - L // vbs) for L in lens)
    tables, total = bt.shape[0], (nb + more + 31) // 32 * 32
    # the parents' pages lie anywhere among all pages
    spread = torch.argsort(torch.rand((tables, total), device="cuda", generator=g), 1)
    full = torch.full((tables, P + F, VB), -1, dtype=torch.int32, device="cuda")
    held = bt >= 0
    ids = torch.gather(spread, 1, bt.clamp(min=0).long().view(tables, -1)).view(bt.shape)
    full[:, :P, :bt.shape[2]] = torch.where(held, ids.to(torch.int32), -1)
    ref = torch.zeros((tables, total), dtype=torch.int32, device="cuda")
    ref.scatter_add_(1, ids.view(tables, -1), held.to(torch.int32).view(tables, -1))
    seq = torch.zeros(P + F, dtype=torch.int32, device="cuda")
    seq[:P] = torch.tensor(lens, dtype=torch.int32)
    child = torch.arange(P, P + F, dtype=torch.int32, device="cuda")
    parent = torch.arange(F, device="cuda") % P
    return dict(bt=full, seq=seq, ref=ref, bits=_bits(ref == 0), nb=total, child=child,
                parent=parent.to(torch.int32), none=torch.zeros_like(child),
                grown=seq[parent] + c["grow"],
                pools=_normal((c["pools"], c["dcp"], total, c["H"], c["bs"], c["d"]),
                              DT[c["dtype"]], g))


def _prepare_compact(c, g):
    ctx, paths = _kept(c)
    bt, nb = _tables([x + c["T"] for x in ctx], c, g)
    path = torch.zeros((c["B"], c["keep"]), dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    return dict(bt=bt, nb=nb, ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                path=path.cuda(),
                n=torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"),
                pools=_normal((c["pools"], c["dcp"], nb, c["H"], c["bs"], c["d"]),
                              DT[c["dtype"]], g))


def prepare(case, seed):
    g = _gen(seed)
    s = {"tree": _prepare_tree, "rope": _prepare_rope, "pages": _prepare_pages,
         "compact": _prepare_compact}[case["op"]](case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _handles(s):
    """The layout and the cache handles that a program makes once and keeps."""
    if "lib" not in s:
        import context_paged_decode_gb300 as dcp

        c = s["case"]
        s["layout"] = dcp.Layout(c["dcp"], c["bs"], c["il"])
        if c["op"] == "tree":
            s["kv"] = dcp.PagedKV(list(s["k"]), list(s["v"]), s["bt"], s["nb"])
        if c["op"] in ("pages", "compact"):
            s["set"] = dcp.PoolSet([list(p) for p in s["pools"]])
        if c["op"] == "pages":
            s["pages"] = dcp.Pages(s["bt"], s["seq"], s["ref"], s["bits"], s["nb"])
        if c["op"] == "rope":
            s["kpl"], s["vpl"] = list(s["kp"]), list(s["vp"]) if "vp" in s else None
        s["lib"] = dcp
    return s["lib"], s["layout"]


def _own_tree(s):
    dcp, L = _handles(s)
    return dcp.tree_decode_gqa(L, s["q"], s["kv"], s["start"], s["ctx"], s["mask"], s["scale"],
                               s["T"], sink=s["sink"])


def _own_rope(s):
    dcp, L = _handles(s)
    adjacent = s["case"]["pairs"] == "adjacent"
    if s["case"]["Hkv"]:
        q = dcp.rope_write_gqa(L, s["q"], s["k"], s["v"], s["pos"], s["inv"], s["slot"], s["kpl"],
                               s["vpl"], s["nb"], axis=s["axis"], interleaved=adjacent)
        return q, s["kp"], s["vp"]
    q = dcp.rope_write_mla(L, s["q"], s["k"], s["pos"], s["inv"], s["slot"], s["kpl"], s["nb"],
                           axis=s["axis"], interleaved=adjacent)
    return q, s["kp"]


def _own_pages(s):
    dcp, L = _handles(s)
    dcp.pages_resize(L, s["pages"], s["child"], s["none"])
    src, dst = dcp.pages_fork(L, s["pages"], s["parent"], s["child"])
    dcp.pages_copy(L, s["set"], src, dst)
    dcp.pages_resize(L, s["pages"], s["child"], s["grown"])
    return s["bt"], s["seq"], s["ref"], s["bits"], src, dst, s["pools"]


def _own_compact(s):
    dcp, L = _handles(s)
    new = dcp.cache_compact(L, s["set"], s["bt"], s["nb"], s["ctx"], s["path"], s["n"])
    return new, s["pools"]


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_tree(s):
    c = s["case"]
    G, d, Hkv, T = c["Hq"] // c["Hkv"], c["d"], c["Hkv"], s["T"]
    B = s["ctx"].numel()
    x = torch.arange(s["longest"], device="cuda")
    rank, vb, loc = _place(x, c)
    page = s["bt"][rank, :, vb].t().long().clamp(min=0)              # [B, L]
    k = s["k"][rank, page, :, loc].float().permute(0, 2, 3, 1)       # [B, Hkv, d, L]
    v = s["v"][rank, page, :, loc].float().permute(0, 2, 1, 3)       # [B, Hkv, L, d]
    n = s["start"].diff().long()
    t = torch.arange(T, device="cuda")
    row = (s["start"][:-1, None].long() + torch.minimum(t, n[:, None] - 1))   # [B, T]
    q = s["q"][row].float().view(B, T, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, d)
    j = x - s["ctx"][:, None].long()                                 # node of a token, < 0: cached
    bit = (s["mask"][row][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
    seen = (j < 0)[:, None] | ((j < n[:, None])[:, None] & (bit == 1))         # [B, T, L]
    sc = (q @ k).view(B, Hkv, T, G, -1) * s["scale"]
    sc = sc.masked_fill(~seen[:, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, Hkv, 1, G, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - top)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (p.view(B, Hkv, T * G, -1) @ v).view(B, Hkv, T, G, d) / torch.where(total == 0, 1.0, total)
    live = t < n[:, None]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, c["Hq"], d)[live]
    return o.to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(B, T, c["Hq"])[live]


def _turned(x, s, at):
    """x [T, ..., d] in 32 bits with the entries from `at` on rotated."""
    c = s["case"]
    ang = s["pos"][s["axis"].long()].t().double() * s["inv"].double()         # [T, rot/2]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    cos, sin = (a.view(a.shape[0], *[1] * (x.dim() - 2), -1) for a in (cos, sin))
    x = x.float()
    r = x[..., at:at + c["rot"]]
    if c["pairs"] == "halves":
        a, b = r.chunk(2, -1)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., ::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :at], r, x[..., at + c["rot"]:]], -1)


def _plain_rope(s):
    c, dt = s["case"], s["q"].dtype
    at = 0 if c["Hkv"] else c["d"] - c["rot"]
    q, k = _turned(s["q"], s, at).to(dt), _turned(s["k"], s, at).to(dt)
    rank, t = s["slot"].argmax(0), torch.arange(c["T"], device="cuda")
    slot = s["slot"][rank, t]
    if c["Hkv"]:
        s["kp"][rank, slot // c["bs"], :, slot % c["bs"]] = k
        s["vp"][rank, slot // c["bs"], :, slot % c["bs"]] = s["v"]
        return q, s["kp"], s["vp"]
    s["kp"][rank, slot // c["bs"], slot % c["bs"]] = k
    return q, s["kp"]


def _bits(free):
    w = free.view(free.shape[0], -1, 32).long() << torch.arange(32, device="cuda")
    w = w.sum(-1)
    return torch.where(w >> 31 == 1, w - (1 << 32), w).to(torch.int32)


def _held(L, c, tables):
    """Tokens of [0, L) in the last, open page of each table [tables, n]."""
    vbs, turn = c["bs"] * c["dcp"], c["il"] * c["dcp"]
    rem = L % vbs
    if c["shared"]:
        return rem[None]
    r = torch.arange(tables, device="cuda")[:, None] * c["il"]
    return rem // turn * c["il"] + (rem % turn - r).clamp(0, c["il"])


def _take(s, want):
    """The lowest free pages for the wanted places [tables, n, VB] in order, one count each."""
    tables = want.shape[0]
    order = torch.sort((s["ref"] != 0).to(torch.int8), dim=1, stable=True)[1]
    k = want.view(tables, -1).cumsum(1) - 1
    ids = order.gather(1, k.clamp(min=0)).view(want.shape)
    s["ref"].scatter_add_(1, ids.view(tables, -1), want.view(tables, -1).to(torch.int32))
    return ids


def _add(ref, ids, which, by):
    t = ref.shape[0]
    add = which.expand(t, *which.shape[-2:]).to(torch.int32) * by
    ref.scatter_add_(1, ids.clamp(min=0).long().reshape(t, -1), add.reshape(t, -1))


def _plain_resize(s, req, new):
    c, bt, ref = s["case"], s["bt"], s["ref"]
    tables, vbs = bt.shape[0], c["bs"] * c["dcp"]
    rows, new = req.long(), new.long()
    old = s["seq"][rows].long()
    ov, nv = (old + vbs - 1) // vbs, (new + vbs - 1) // vbs
    vb = torch.arange(bt.shape[2], device="cuda")
    sub = bt[:, rows]
    gone = (vb >= nv[:, None]) & (vb < ov[:, None])
    _add(ref, sub, gone, -1)
    # the open page behind the kept tokens has to be the request's own
    cut = torch.minimum(old, new)
    cv, held = cut // vbs, _held(cut, c, tables)
    page = sub.gather(2, cv.clamp(max=bt.shape[2] - 1).expand(tables, -1)[..., None])[..., 0].long()
    part = (cut % vbs > 0) & (held < (vbs if c["shared"] else c["bs"]))
    again = part & (ref.gather(1, page.clamp(min=0)) > 1)
    at = again[..., None] & (vb == cv[:, None])
    want = ((vb >= ov[:, None]) & (vb < nv[:, None]))[None] | at
    ids = _take(s, want)
    _add(ref, sub, at, -1)
    bt[:, rows] = torch.where(want, ids.to(torch.int32), torch.where(gone, -1, sub))
    s["seq"][rows] = new.to(torch.int32)
    s["bits"].copy_(_bits(ref == 0))


def _plain_fork(s):
    c, bt, ref = s["case"], s["bt"], s["ref"]
    tables, vbs = bt.shape[0], c["bs"] * c["dcp"]
    rows, up = s["child"].long(), s["parent"].long()
    vb = torch.arange(bt.shape[2], device="cuda")
    old, L = s["seq"][rows].long(), s["seq"][up].long()
    _add(ref, bt[:, rows], vb < (old[:, None] + vbs - 1) // vbs, -1)
    sub = bt[:, up]
    held = _held(L, c, tables)
    opened = (L % vbs > 0) & (held < (vbs if c["shared"] else c["bs"]))       # [tables, F]
    want = opened[..., None] & (vb == (L // vbs)[:, None])
    ids = _take(s, want)
    kept = (vb < ((L + vbs - 1) // vbs)[:, None])[None] & ~want
    _add(ref, sub, kept, 1)
    bt[:, rows] = torch.where(want, ids.to(torch.int32), torch.where(kept, sub, -1))
    s["seq"][rows] = s["seq"][up]
    s["bits"].copy_(_bits(ref == 0))
    copied = want & (held > 0)[..., None]
    src = torch.where(copied, sub, -1).amax(-1)
    dst = torch.where(copied, ids.to(torch.int32), -1).amax(-1)
    return src, dst


def _plain_pages(s):
    c = s["case"]
    _plain_resize(s, s["child"], s["none"])
    src, dst = _plain_fork(s)
    a, b = (x.expand(c["dcp"], -1).long() for x in (src, dst))
    r = torch.arange(c["dcp"], device="cuda")[:, None].expand_as(a)[b >= 0]
    s["pools"][:, r, b[b >= 0]] = s["pools"][:, r, a[b >= 0]]
    _plain_resize(s, s["child"], s["grown"])
    return s["bt"], s["seq"], s["ref"], s["bits"], src, dst, s["pools"]


def _plain_compact(s):
    c = s["case"]
    i = torch.arange(c["keep"], device="cuda")
    b = torch.arange(c["B"], device="cuda")[:, None].expand(-1, c["keep"])
    live = i < s["n"][:, None]
    b, src, dst = b[live], (s["ctx"][:, None] + s["path"])[live].long(), \
        (s["ctx"][:, None] + i)[live].long()
    r0, v0, l0 = _place(src, c)
    r1, v1, l1 = _place(dst, c)
    rows = s["pools"][:, r0, s["bt"][r0, b, v0].long(), :, l0]
    s["pools"][:, r1, s["bt"][r1, b, v1].long(), :, l1] = rows
    return s["ctx"] + s["n"], s["pools"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "rope": _own_rope, "pages": _own_pages,
                "compact": _own_compact}[op](state)
    return {"tree": _plain_tree, "rope": _plain_rope, "pages": _plain_pages,
            "compact": _plain_compact}[op](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token and page by page
# ---------------------------------------------------------------------------

def _exact_tree(c, s):
    ctx, T = _tree_sizes(c)
    G, outs, lses, at = c["Hq"] // c["Hkv"], [], [], 0
    slots = torch.arange(c["bs"], device="cuda")
    for b, (n, t) in enumerate(zip(ctx, T)):
        L = n + t
        k = torch.zeros((c["Hkv"], L, c["d"]), dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        for r in range(c["dcp"]):  # each rank's pages in order, and the token of each place in them
            pages = s["bt"][r, b][s["bt"][r, b] >= 0].long()
            block = torch.arange(pages.numel(), device="cuda")[:, None] * c["bs"] * c["dcp"]
            x = (block + (slots // c["il"] * c["dcp"] + r) * c["il"] + slots % c["il"]).flatten()
            keep = x < L
            for pool, to in ((s["k"], k), (s["v"], v)):
                rows = pool[r, pages].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])
                to[:, x[keep]] = rows[:, keep].double()
        q = s["q"][at:at + t].double()
        m = s["mask"][at:at + t]
        seen = torch.ones((t, L), dtype=torch.bool, device="cuda")
        seen[:, n:] = torch.stack([(m >> j) & 1 for j in range(t)], 1) == 1
        o = torch.empty((t, c["Hq"], c["d"]), dtype=torch.float64, device="cuda")
        lse = torch.empty((t, c["Hq"]), dtype=torch.float64, device="cuda")
        for h in range(c["Hq"]):
            e = torch.where(seen, q[:, h] @ k[h // G].T * s["scale"], -math.inf)
            if s["sink"] is not None:
                e = torch.cat([e, s["sink"][h].double().expand(t, 1)], 1)
            lse[:, h] = torch.logsumexp(e, 1)
            o[:, h] = torch.softmax(e, 1)[:, :L] @ v[h // G]
        outs.append(o)
        lses.append(lse)
        at += t
    return torch.cat(outs), torch.cat(lses)


def _exact_rope(c, s):
    half, at = c["rot"] // 2, 0 if c["Hkv"] else c["d"] - c["rot"]
    turn = torch.empty((c["T"], half), dtype=torch.complex128, device="cuda")
    for i in range(half):
        ang = s["pos"][int(s["axis"][i])].double() * float(s["inv"][i])
        turn[:, i] = torch.complex(torch.cos(ang), torch.sin(ang))
    first = [at + (i if c["pairs"] == "halves" else 2 * i) for i in range(half)]
    second = [i + (half if c["pairs"] == "halves" else 1) for i in first]

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second])
        z = z * (turn if x.dim() == 2 else turn[:, None])
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def stored(pool, rows):
        flat = pool.double()
        flat = flat.transpose(2, 3).reshape(c["dcp"], -1, *rows.shape[1:]) if c["Hkv"] else \
            flat.reshape(c["dcp"], -1, c["d"])
        for r in range(c["dcp"]):
            mine = s["slot"][r] >= 0
            flat[r, s["slot"][r][mine]] = rows[mine]
        if not c["Hkv"]:
            return flat.view(pool.shape)
        return flat.view(c["dcp"], -1, c["bs"], c["Hkv"], c["d"]).transpose(2, 3).contiguous()

    if c["Hkv"]:
        return turned(s["q"]), stored(s["kp"], turned(s["k"])), stored(s["vp"], s["v"].double())
    return turned(s["q"]), stored(s["kp"], turned(s["k"]))


def _exact_pages(c, s):
    """Request by request and page by page, on the host.  Copied bytes have no other value."""
    bt, ref = s["bt"].cpu().tolist(), s["ref"].cpu().tolist()
    seq = s["seq"].cpu().tolist()
    parents, children = s["parent"].cpu().tolist(), s["child"].cpu().tolist()
    vbs, F = c["bs"] * c["dcp"], len(children)
    src = [[-1] * F for _ in bt]
    dst = [[-1] * F for _ in bt]
    for r, (rows, count) in enumerate(zip(bt, ref)):
        free = [i for i, n in enumerate(count) if n == 0]
        for f, (p, ch) in enumerate(zip(parents, children)):
            L = seq[p]
            full, open_ = divmod(L, vbs)
            rows[ch] = rows[p][:full] + [-1] * (len(rows[p]) - full)
            for page in rows[ch][:full]:
                count[page] += 1
            if open_:
                n = open_ if c["shared"] else _local(L, r, c) - full * c["bs"]
                if n == c["bs"] and not c["shared"]:
                    rows[ch][full] = rows[p][full]
                    count[rows[p][full]] += 1
                else:
                    rows[ch][full] = free.pop(0)
                    count[rows[ch][full]] += 1
                    if n:
                        src[r][f], dst[r][f] = rows[p][full], rows[ch][full]
        for p, ch in zip(parents, children):
            for v in range(-(-seq[p] // vbs), -(-(seq[p] + c["grow"]) // vbs)):
                rows[ch][v] = free.pop(0)
                count[rows[ch][v]] += 1
    for p, ch in zip(parents, children):
        seq[ch] = seq[p] + c["grow"]
    bits = [[sum((n == 0) << i for i, n in enumerate(count[w:w + 32]))
             for w in range(0, len(count), 32)] for count in ref]
    bits = [[w - (1 << 32) if w >> 31 else w for w in row] for row in bits]
    to = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return to(bt), to(seq), to(ref), to(bits), to(src), to(dst), None


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(case, s)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "pages":
        return _exact_pages(case, s)
    ctx, paths = _kept(case)
    return torch.tensor([x + len(p) for x, p in zip(ctx, paths)], dtype=torch.int32,
                        device="cuda"), None
