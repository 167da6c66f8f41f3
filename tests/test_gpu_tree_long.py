"""Drafted-tree attention where work runs on: rings that go round, accumulators that are
rescaled, units cut and joined in every way, many requests, and rows whose first parts see
nothing.  The plan of each call is worked out on the host, so that a case is known to take
the path that it is for."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.asarray(x, dtype=dtype)).cuda()


def places(n, dcp, bs, I):
    """R.place of the tokens 0 .. n - 1 as arrays."""
    x = np.arange(n)
    vb, off = np.divmod(x, bs * dcp)
    run = off // I
    return run % dcp, vb, run // dcp * I + off % I


class Case:
    """Requests of ctx cached tokens and T nodes; every row of the pools holds a number."""

    def __init__(self, lib, dtype, Hq, Hkv, d, dcp, bs, I, ctx, T, seed=0, scale=None):
        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.dims = dtype, (Hq, Hkv, d, dcp, bs, I)
        self.ctx, self.T = [int(n) for n in ctx], [int(t) for t in T]
        self.layout = lib.Layout(dcp, bs, I)
        self.bt, self.nb = R.random_tables(rng, [c + t for c, t in zip(ctx, T)], dcp, bs)
        gen = torch.Generator().manual_seed(seed)
        mk = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
        self.k, self.v = (mk(dcp, self.nb, Hkv, bs, d) for _ in range(2))
        self.start = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
        self.N = int(self.start[-1])
        self.q = mk(self.N, Hq, d)
        self.mask = []
        for t in T:   # each node sees itself and what one of the four before it sees
            own = []
            for j in range(t):
                own.append((own[rng.integers(max(0, j - 4), j)] if j else 0) | 1 << j)
            self.mask += own
        self.scale = scale or d ** -0.5

    def at(self, b, n=None):
        """(rank, page, place) of request b's tokens."""
        r, vb, loc = places(self.ctx[b] + self.T[b] if n is None else n, *self.dims[3:])
        return r, self.bt[r, b, vb], loc

    def args(self, lib, bt=None, most=None):
        kv = lib.PagedKV(list(self.k.cuda()), list(self.v.cuda()),
                         dev(self.bt if bt is None else bt), self.nb)
        m = np.array(self.mask, dtype=np.uint64).view(np.int64)
        return (self.layout, self.q.cuda(), kv, dev(self.start), dev(self.ctx),
                torch.from_numpy(m).cuda(), self.scale, most or max(max(self.T), 1))

    def seen(self, b):
        n, T, s0 = self.ctx[b], self.T[b], self.start[b]
        out = np.ones((T, n + T), dtype=bool)
        for t in range(T):
            for j in range(T):
                out[t, n + j] = (self.mask[s0 + t] >> j) & 1
        return out

    def check(self, out, lse, out_dtype, rank=None, sink=None, there=None, requests=None,
              columns=None):
        """Every row against 64 bits; `there`(b): which of b's tokens can be read."""
        Hq, Hkv, d, dcp, bs, I = self.dims
        G = Hq // Hkv
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        k, v, q = (x.float().numpy() for x in (self.k, self.v, self.q))
        for b in requests if requests is not None else range(len(self.T)):
            if self.T[b] == 0:
                continue
            r, page, loc = self.at(b)
            keep = np.ones(len(r), dtype=bool) if rank is None else r == rank
            if there is not None:
                keep &= there(b)
            kb = k[r[keep], page[keep], :, loc[keep]].astype(np.float64)   # [tokens, Hkv, d]
            vb = v[r[keep], page[keep], :, loc[keep]].astype(np.float64)
            seen, L = self.seen(b)[:, keep], int(keep.sum())
            rows = slice(self.start[b], self.start[b + 1])
            for g in range(Hkv):
                qs = q[rows, g * G:(g + 1) * G].astype(np.float64)
                for x in range(G):
                    h = g * G + x
                    o, el, wabs, size = R.attend(qs[:, x], kb[:, g], vb[:, g], seen, self.scale,
                                                 None if sink is None else float(sink[h]))
                    tol = R.attend_tol(self.dtype, out_dtype, o, wabs, size, d, L)
                    ok = np.abs(out[rows, h] - o) <= tol
                    if columns is not None:
                        ok = ok[:, columns]
                    assert ok.all(), (b, h, rank, np.argwhere(~ok)[:3])
                    empty = np.isneginf(el)
                    assert np.array_equal(np.isneginf(lse[rows, h]), empty), (b, h, rank)
                    off = np.abs(lse[rows, h][~empty] - el[~empty])
                    assert (off <= R.lse_tol(el, size, d, L)[~empty]).all(), (b, h, rank, off.max())


def plan(c, tc, per_rank=False, most=None):
    """The work of a call, as the kernels lay it out: (run, unit, first tile, tiles, whole)
    of every piece, and the number of runs."""
    Hq, Hkv, d, dcp, bs, I = c.dims
    G, most = Hq // Hkv, most or max(c.T)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if tc:
        nodes = 128 // G
        rows, chunk, tile, parts = (1 if most <= nodes else 2) * nodes * G, 16, 128, sms
        extra = 2 + (1 if per_rank else dcp)
    else:
        rows, chunk, tile = (16 if most * G <= 16 else 32) // G * G, 64, 64
        parts, extra = 2 * sms, 0
    entries = []
    for b, (n, T) in enumerate(zip(c.ctx, c.T)):
        held = np.bincount(places(n + T, dcp, bs, I)[0], minlength=dcp) if T else np.zeros(dcp, int)
        for group in ([[r] for r in range(dcp)] if per_rank else [range(dcp)]):
            chunks = sum(-(-int(held[r]) // chunk) for r in group)
            per = -(-chunks // (tile // chunk))
            entries.append((Hkv * -(-T * G // rows) if per else 0, per))
    tiles = sum(u * p for u, p in entries)
    extra = min(extra, tiles // parts)
    total = tiles + extra * sum(u for u, _ in entries)
    parts = min(parts, total)
    pieces, at, unit = [], 0, 0
    for u, per in entries:
        for _ in range(u):
            t = at
            while t < at + per:
                run = ((t + 1) * parts - 1) // total
                end = min(total * (run + 1) // parts, at + per)
                pieces.append((run, unit, t - at, end - t, t == at and end == at + per))
                t = end
            at += per + extra
            unit += 1
    return pieces, parts


# dtype, Hq, Hkv, d, dcp, bs, I, ctx, T, streams, joined by the last CTA
LONG = {
    "one-stream-merged": (BF16, 8, 8, 128, 2, 16, 1, [17000, 15500], [64, 50], 1, False),
    "two-streams-merged": (BF16, 16, 4, 64, 3, 32, 4, [14001, 13000, 14500], [64, 33, 47], 2, False),
    "one-stream-joined": (BF16, 32, 2, 64, 2, 16, 16, [1500 + 37 * (i % 17) for i in range(80)],
                          [1 + i % 8 for i in range(80)], 1, True),
    "two-streams-joined": (BF16, 16, 4, 128, 4, 16, 1, [1300 + 61 * (i % 13) for i in range(40)],
                           [64 - i % 31 for i in range(40)], 2, True),
    "one-stream-joined-wide-heads": (BF16, 16, 4, 128, 8, 64, 1,
                                     [1100 + 97 * (i % 11) for i in range(40)],
                                     [32 - i % 9 for i in range(40)], 1, True),
}


@pytest.mark.parametrize("name", LONG)
def test_rings_go_round(lib, name):
    """Runs of more tiles than the rings have slots, several units a run, units that are cut."""
    *shape, streams, joined = LONG[name]
    c = Case(lib, *shape, seed=len(name))
    Hq, Hkv, d, dcp = c.dims[:4]
    pieces, parts = plan(c, True)
    assert max(n for _, _, _, n, _ in pieces) >= 8                  # six slots at most
    assert max(np.bincount([p[0] for p in pieces])) >= 2            # several pieces in a run
    assert any(not whole for *_, whole in pieces)                   # and some are cut
    assert (max(c.T) > 128 * Hkv // Hq) == (streams == 2)
    assert (len(c.T) > 16 and len(c.T) * Hkv >= torch.cuda.get_device_properties(
        0).multi_processor_count) == joined
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sink = torch.linspace(-2, 9, Hq).cuda()
    out, lse = lib.tree_decode_gqa(*c.args(lib), sink=sink, err=err)
    c.check(out, lse, BF16, sink=sink.cpu().numpy())
    again = lib.tree_decode_gqa(*c.args(lib), sink=sink, err=err)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    out, lse = lib.tree_decode_gqa(*c.args(lib), out_dtype=F32, err=err)
    c.check(out, lse, F32)
    assert err.item() == 0


@pytest.mark.parametrize("name", ["two-streams-merged", "one-stream-joined"])
def test_rings_go_round_rank_by_rank(lib, name):
    c = Case(lib, *LONG[name][:-2], seed=3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    po, pl = lib.tree_partial_gqa(*c.args(lib), err=err)
    for r in range(c.dims[3]):
        c.check(po[r], pl[r], F32, rank=r)
    assert err.item() == 0


@pytest.mark.parametrize("streams", [1, 2])
@pytest.mark.parametrize("d", [64, 128])
def test_the_accumulator_is_rescaled(lib, streams, d):
    """Tiles whose maximum passes that of the tiles before by more than 2^8, in some rows of a
    warp and not in others, with what came before still worth a part of the result: in most
    tiles all tokens score about alike, and now and then a single one scores nine more (in
    log2 units, times a factor that each row has of its own)."""
    T = 20 * streams
    c = Case(lib, BF16, 16, 4, d, 2, 16, 1, [9000, 8800, 9100, 8700, 9050, 8900, 8950, 9011],
             [T - 1, T, T, T - 3, T, T, T - 2, T], seed=d + streams, scale=1.0)
    assert (max(c.T) > 32) == (streams == 2)
    pieces, _ = plan(c, True)
    assert max(n for _, _, _, n, _ in pieces) >= 12
    rng = np.random.default_rng(1)
    # scores: q[0] * k[0] and a little of the rest
    q, k = c.q.float() * 2.0 ** -6, c.k.float() * 2.0 ** -4
    q[..., 0] = torch.from_numpy(rng.choice([0.25, 0.5, 1.0, 1.25], q.shape[:2]).astype(np.float32))
    rises = 0
    for b in range(len(c.T)):
        r, page, loc = c.at(b)
        level = np.zeros(len(r), dtype=np.float32)
        top, x = 0.0, int(rng.integers(100, 300))
        while x < len(r):
            top += 9.0 * float(np.log(2.0))
            level[x] = top                     # the one token that is high
            rest = int(rng.integers(150, 700))
            level[x + 1:x + rest] = top - 6.0 * float(np.log(2.0)) if rng.random() < 0.5 else 0.0
            x += rest
            rises += 1
        k[torch.from_numpy(r), torch.from_numpy(page).long(), :, torch.from_numpy(loc), 0] = \
            torch.from_numpy(level)[:, None]
    c.q, c.k = q.to(BF16), k.to(BF16)
    assert rises > 100
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.tree_decode_gqa(*c.args(lib), out_dtype=F32, err=err)
    c.check(out, lse, F32)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("per_rank", [False, True])
def test_more_entries_than_the_plan_has_threads(lib, dtype, per_rank):
    """The plan goes over its entries twice when there are more than 256 (requests, or requests
    on a rank); some have no nodes and some are refused."""
    B, dcp = (70, 8) if per_rank else (530, 2)
    rng = np.random.default_rng(5)
    ctx, T = rng.integers(0, 260, B), rng.integers(0, 7, B)
    ctx[[3, B - 1]], T[[3, B - 1]] = (1900, 2100), (6, 6)
    c = Case(lib, dtype, 8, 2, 64, dcp, 16, 1, ctx, T, seed=B)
    bad = [0, 7, B // 2]
    args = list(c.args(lib))
    for b in bad:
        args[4][b] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = [b for b in range(B) if b not in bad]
    if per_rank:
        po, pl = lib.tree_partial_gqa(*args, err=err)
        for r in range(dcp):
            c.check(po[r], pl[r], F32, rank=r, requests=good)
    else:
        out, lse = lib.tree_decode_gqa(*args, err=err)
        c.check(out, lse, dtype, requests=good)
    assert err.item() == len(bad)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [3, 40])
def test_values_that_are_not_finite_in_many_short_units(lib, d, T):
    """Units of one tile, several to a run, each with an infinite and a NaN value in a node that
    one other node sees: those two rows get them, in those columns, and no others do."""
    B = 400
    rng = np.random.default_rng(d + T)
    c = Case(lib, BF16, 8, 2, d, 2, 16, 1, rng.integers(0, 40, B), [T] * B, seed=T)
    pieces, parts = plan(c, True)
    assert max(n for _, _, _, n, _ in pieces) == 1 and len(pieces) >= 4 * parts
    bad, other = T // 2, T - 1
    for b in range(B):
        s0 = c.start[b]
        for j in range(T):
            c.mask[s0 + j] &= ~(1 << bad)
        c.mask[s0 + bad] |= 1 << bad
        c.mask[s0 + other] |= 1 << bad
        r, page, loc = c.at(b)
        x = c.ctx[b] + bad
        c.v[r[x], page[x], :, loc[x], 5] = float("inf")
        c.v[r[x], page[x], :, loc[x], d - 3] = float("nan")
    finite = [i for i in range(d) if i not in (5, d - 3)]
    for _ in range(5):
        out, lse = lib.tree_decode_gqa(*c.args(lib), out_dtype=F32)
        got = out.view(B, T, 8, d)
        sees = torch.zeros(T, dtype=torch.bool, device="cuda")
        sees[[bad, other]] = True
        assert (got[:, sees][..., 5] == float("inf")).all()
        assert torch.isnan(got[:, sees][..., d - 3]).all()
        assert torch.isfinite(got[:, ~sees]).all() and torch.isfinite(got[..., finite]).all()
    c.check(out, lse, F32, columns=finite, requests=range(0, B, 7))


@pytest.mark.parametrize("most", [4, 64])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_first_parts_that_saw_nothing(lib, dtype, most):
    """A unit in many parts, of which the first have only pages that cannot be used, and scores
    near -120: a part that saw nothing sets no maximum for those behind it.  (Up to 2048 rows
    of max_tree nodes two warps join a row's parts, beyond that one.)"""
    Hq, Hkv, d, bs, n = 48, 3, 64, 16, 6000
    c = Case(lib, dtype, Hq, Hkv, d, 1, bs, 1, [n], [2], seed=most, scale=0.125)
    assert (most * Hq > 2048) == (most == 64)
    c.q = torch.ones_like(c.q)
    c.k = (-15.0 + 0.25 * c.k.float()).to(dtype)
    pieces, _ = plan(c, dtype == BF16, most=most)
    tile = 128 if dtype == BF16 else 64
    # everything before the last ten parts is gone
    gone = (max(t for _, u, t, _, _ in pieces if u == 0) - 9) * tile // bs
    assert len([p for p in pieces if p[1] == 0 and p[2] * tile < gone * bs]) > 20
    bt = c.bt.copy()
    bt[0, 0, :gone] = -1
    there = lambda b: np.arange(n + 2) >= gone * bs  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for sink in (None, torch.full((Hq,), -125.0, device="cuda")):
        out, lse = lib.tree_decode_gqa(*c.args(lib, bt, most), sink=sink, out_dtype=F32, err=err)
        c.check(out, lse, F32, there=there, sink=None if sink is None else sink.cpu().numpy())
    assert err.item() > 0
    po, pl = lib.tree_partial_gqa(*c.args(lib, bt, most))
    c.check(po[0], pl[0], F32, there=there)


@pytest.mark.parametrize("offset", [0.0, -15.0])
def test_nodes_of_many_ranks_that_see_themselves_alone(lib, offset):
    """No context, 64 nodes on 16 ranks that see only themselves, and units of six parts: most
    parts of a row saw nothing, the first ones among them."""
    c = Case(lib, F32, 33, 33, 64, 16, 16, 1, [0], [64], scale=0.125)
    c.mask = [1 << j for j in range(64)]
    c.q = torch.ones_like(c.q)
    c.k = offset + 0.25 * c.k
    pieces, _ = plan(c, False)
    assert 64 * 33 > 2048 and max(np.bincount([u for _, u, *_ in pieces])) > 4
    out, lse = lib.tree_decode_gqa(*c.args(lib))
    c.check(out, lse, F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B", [3, 40])
def test_a_workspace_aligned_to_sixteen_bytes(lib, dtype, B):
    """And to no more, with a plan made by the kernel's CTAs (3 requests) and one by itself."""
    c = Case(lib, dtype, 8, 2, 64, 2, 16, 1, [90 + b for b in range(B)],
             [1 + b % 9 for b in range(B)])
    need = lib.tree_workspace_size(c.layout, B, 9, 8, 2, 64, dtype)
    room = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    args = c.args(lib)
    want = lib.tree_decode_gqa(*args)
    c.check(*want, dtype)
    for off in (0, 16, 32, 48):
        ws = room[off:off + need]
        assert ws.data_ptr() % 64 == off
        got = lib.tree_decode_gqa(*args, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
