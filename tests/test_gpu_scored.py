"""Scored decode attention over 32-bit, 16-bit and 8-bit caches, against 64 bits.

Every place that must not count (tokens that are not seen, pages that no request
has, scales of such pages) holds NaN."""
import numpy as np
import pytest
import torch

from tests import scored_ref as S
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Problem:
    """Random requests: lens, per-request seen tokens and their keys and values, and the cache."""

    def __init__(self, lib, cache, qtype, Hq, Hkv, d, dcp, bs, I, lens, cap=0.0, window=0, prefix=0,
                 alibi=False, docs=False, sink=False, shared=False, seed=0, spread=1.0, room=0):
        rng = np.random.default_rng(seed + 1000 * d + sum(lens))
        self.lib, self.qtype, self.Hq, self.Hkv, self.d = lib, qtype, Hq, Hkv, d
        self.lens, self.cap, self.G, self.dcp, self.bs, self.I = lens, cap, Hq // Hkv, dcp, bs, I
        B = len(lens)
        self.layout = lib.Layout(dcp, bs, I)
        tables = 1 if shared else dcp
        vbs = bs * dcp
        # a table with room for more tokens: a request's tiles are cut elsewhere then
        bt, nb = R.random_tables(rng, lens, tables, bs * dcp // tables, max_vb=room // vbs)
        q = torch.from_numpy(rng.standard_normal((B, Hq, d)) * spread).to(qtype)
        self.q, self.q64 = q.cuda(), q.double().numpy()
        self.first = np.array([rng.integers(0, max(n, 1)) if docs else 0 for n in lens])
        self.slopes = 2.0 ** -np.arange(1, Hq + 1) if alibi else np.zeros(Hq)
        self.sink = rng.standard_normal(Hq) if sink else None
        self.scale = d ** -0.5
        ptype = E4M3 if cache == E4M3 else cache
        shape = (dcp, nb, Hkv, bs, d)
        pools = [np.full(shape, np.nan, np.float32) for _ in range(2)]
        sc = np.full((dcp, nb, Hkv, 4), np.nan, np.float32)
        sc[..., :2] = 2.0 ** rng.integers(-9, -3, (dcp, nb, Hkv, 2))
        self.rows = []
        for b, n in enumerate(lens):
            seen = S.seen_mask(n, window, prefix, int(self.first[b]))
            x = np.nonzero(seen)[0]
            kv = []
            for i in range(2):
                vals = torch.from_numpy(rng.standard_normal((len(x), Hkv, d)))
                if cache == E4M3:
                    vals = (vals * 64).to(E4M3)
                else:
                    vals = vals.to(cache)
                vals = vals.double().numpy()
                out = np.empty((Hkv, len(x), d))
                for j, pos in enumerate(x):
                    r, vb, loc = R.place(pos, dcp, bs, I)
                    page = bt[0 if shared else r, b, vb]
                    pools[i][r, page, :, loc] = vals[j]
                    s = sc[r, page, :, i].astype(np.float64) if cache == E4M3 else np.ones(Hkv)
                    out[:, j] = vals[j] * s[:, None]
                kv.append(out)
            self.rows.append((x, *kv))
        to = lambda a: torch.from_numpy(a).to(ptype).cuda()  # noqa: E731
        self.bt = torch.from_numpy(bt).cuda()
        kp, vp = list(to(pools[0])), list(to(pools[1]))
        if cache == E4M3:
            self.kv = lib.PagedKV8(kp, vp, list(torch.from_numpy(sc).cuda()), self.bt, nb)
            self.decode, self.partial = lib.q8_decode_gqa, lib.q8_partial_gqa
        else:
            self.kv = lib.PagedKV(kp, vp, self.bt, nb)
            self.decode, self.partial = lib.scored_decode_gqa, lib.scored_partial_gqa
        self.form = lib.Scores(
            cap=cap, window=window, prefix=prefix,
            slopes=torch.from_numpy(self.slopes).float().cuda() if alibi else None,
            first=torch.from_numpy(self.first).int().cuda() if docs else None)
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dsink = torch.from_numpy(self.sink).float().cuda() if sink else None
        if sink:
            self.sink = self.dsink.double().cpu().numpy()

    def run(self, **kw):
        return self.decode(self.layout, self.q, self.kv, self.dlens, self.scale, self.form,
                           sink=self.dsink, **kw)

    def check(self, out, lse, rank=None, skip=()):
        """Every head of every request; of one rank's tokens, without the sink."""
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, n in enumerate(self.lens):
            if b in skip:
                continue
            x, k, v = self.rows[b]
            if rank is not None:
                on = np.array([R.place(p, self.dcp, self.bs, self.I)[0] == rank for p in x], bool)
                x, k, v = x[on], k[:, on], v[:, on]
            for h in range(self.Hq):
                g = h // self.G
                sink = self.sink[h] if self.sink is not None and rank is None else None
                eo, el, to, tl = S.attend(self.qtype, out.dtype, self.q64[b, h], k[g], v[g], x, n,
                                          self.scale, self.cap, self.slopes[h], sink)
                what = f"request {b} head {h} of {n} tokens"
                assert np.isfinite(o[b, h]).all(), what
                assert (np.abs(o[b, h] - eo) <= to).all(), (what, np.abs(o[b, h] - eo).max(), to)
                if np.isinf(el):
                    assert l[b, h] == el, what
                else:
                    assert abs(l[b, h] - el) <= tl, (what, l[b, h], el, tl)


# cache, q, Hq, Hkv, d, dcp, bs, I, lens, more
CASES = [
    # lengths of zero and one, and around a page and a tile
    (BF16, BF16, 32, 8, 128, 2, 16, 1, [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 100], {}),
    (E4M3, BF16, 32, 8, 128, 2, 16, 1, [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 100], {}),
    (F32, F32, 8, 2, 64, 2, 16, 1, [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 100], {}),
    (E4M3, F32, 8, 2, 64, 2, 16, 1, [0, 1, 17, 65, 200], {}),
    # a long request cut over many CTAs beside short ones, a sink
    (BF16, BF16, 16, 2, 128, 8, 16, 1, [5000, 3, 0, 700], dict(sink=True)),
    (E4M3, BF16, 16, 2, 128, 8, 16, 1, [5000, 3, 0, 700], dict(sink=True)),
    (F32, F32, 4, 1, 128, 3, 16, 4, [2500, 3, 0, 70], dict(sink=True)),
    # caps, large scores under them
    (BF16, BF16, 32, 8, 128, 4, 32, 1, [300, 77], dict(cap=20.0, spread=20.0)),
    (E4M3, BF16, 32, 8, 128, 4, 32, 1, [300, 77], dict(cap=5.0, spread=20.0)),
    (F32, F32, 4, 4, 64, 4, 32, 1, [300, 77], dict(cap=20.0, spread=20.0)),
    # biased by distance
    (BF16, BF16, 8, 8, 128, 3, 16, 2, [900, 5, 1], dict(alibi=True)),
    (E4M3, BF16, 8, 8, 128, 3, 16, 2, [900, 5, 1], dict(alibi=True, cap=30.0)),
    (F32, F32, 8, 4, 96, 3, 16, 2, [900, 5, 1], dict(alibi=True)),
    # windows, with first tokens kept, at every place of a page
    (BF16, BF16, 16, 4, 128, 2, 16, 1, [500, 133, 64, 40, 3], dict(window=37, prefix=5)),
    (E4M3, BF16, 16, 4, 128, 2, 16, 1, [500, 133, 64, 40, 3], dict(window=37, prefix=5)),
    (E4M3, BF16, 16, 4, 128, 8, 16, 16, [2100, 133, 64, 40, 3], dict(window=1, prefix=1)),
    (F32, F32, 4, 4, 32, 2, 8, 4, [500, 133, 64, 40, 3], dict(window=37, prefix=50)),
    # packed documents
    (BF16, BF16, 16, 1, 64, 3, 32, 4, [901, 333, 64, 1], dict(docs=True, alibi=True, cap=20.0)),
    (E4M3, BF16, 16, 1, 64, 3, 32, 4, [901, 333, 64, 1], dict(docs=True, window=100, prefix=3)),
    # 64-wide heads, many ranks, whole pages in turn, one table for all ranks
    (BF16, BF16, 8, 2, 64, 16, 16, 16, [1999, 256], dict(shared=True)),
    (E4M3, BF16, 8, 2, 64, 16, 16, 16, [1999, 256], dict(shared=True)),
    (E4M3, BF16, 12, 4, 128, 1, 64, 64, [1999, 256], dict(sink=True)),
    # nine to sixteen query heads for a key/value head; pages of three tiles, five ranks
    (BF16, BF16, 32, 2, 128, 2, 16, 1, [1100, 37], dict(cap=30.0, sink=True)),
    (E4M3, BF16, 32, 2, 128, 2, 16, 1, [1100, 37], dict(cap=30.0, alibi=True)),
    (E4M3, BF16, 18, 2, 64, 5, 48, 3, [1100, 37], dict(window=300)),
    (BF16, BF16, 11, 1, 128, 5, 48, 3, [1100, 37], dict(alibi=True)),
    (F32, F32, 12, 1, 128, 5, 48, 3, [600, 37], dict(sink=True)),
    # pages and heads that tiles do not fit
    (BF16, BF16, 6, 2, 96, 2, 24, 3, [301, 11], dict(window=90)),
    (E4M3, BF16, 5, 1, 256, 2, 8, 1, [301, 11], dict(cap=30.0)),
    (BF16, BF16, 3, 3, 128, 2, 1, 1, [301, 11], {}),
    (F32, F32, 16, 1, 256, 2, 16, 1, [301, 11], {}),
    (E4M3, F32, 2, 2, 32, 2, 16, 1, [301, 11], dict(alibi=True)),
    # several passes of heads over one cluster's tokens, the last of them not full
    (F32, F32, 16, 1, 64, 2, 16, 1, [300, 0, 37, 1], dict(sink=True)),
    (E4M3, F32, 14, 2, 64, 2, 16, 1, [200, 5], dict(alibi=True, cap=30.0)),
    # one request long enough for clusters of sixteen
    (E4M3, BF16, 8, 2, 128, 2, 16, 1, [3001], dict(cap=30.0, sink=True)),
    (BF16, BF16, 16, 1, 64, 2, 16, 1, [3001], {}),
]


def name(c):
    return (f"{str(c[0])[6:]}-q{str(c[1])[6:]}-{c[2]}.{c[3]}-d{c[4]}-dcp{c[5]}-bs{c[6]}-I{c[7]}-"
            + "-".join(c[9]))


@pytest.mark.parametrize("room", [0, 1 << 20])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_fused_and_partials(lib, case, room):
    cache, qtype, Hq, Hkv, d, dcp, bs, I, lens, more = case
    p = Problem(lib, cache, qtype, Hq, Hkv, d, dcp, bs, I, lens, room=room, **more)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = p.run(err=err)
    assert out.dtype == qtype and err.item() == 0
    p.check(out, lse)
    po, pl = p.partial(p.layout, p.q, p.kv, p.dlens, p.scale, p.form, err=err)
    assert err.item() == 0
    for r in range(dcp):
        p.check(po[r], pl[r], rank=r)
    # the ranks' results merge into the fused one, and a call repeats itself bit for bit
    mo, ml = lib.lse_merge(po, pl, sink=p.dsink)
    p.check(mo, ml)
    again = p.run()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
def test_types_of_the_output(lib, cache):
    q = F32 if cache == F32 else BF16
    p = Problem(lib, cache, q, 8, 2, 128, 2, 16, 1, [700, 20])
    for t in (BF16, F32):
        out, lse = p.run(out_dtype=t)
        assert out.dtype == t
        p.check(out, lse)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
def test_data_errors_are_counted(lib, cache):
    """Negative lengths, lengths beyond the table, and pages that are not there."""
    q = F32 if cache == F32 else BF16
    p = Problem(lib, cache, q, 4, 1, 128, 2, 16, 1, [64, 96, 40, 70])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.dlens[0] = -5
    room = p.bt.shape[-1] * 32
    p.dlens[1] = room + 1000        # what the table has is attended: 96 tokens
    out, lse = p.run(err=err)
    assert err.item() == 2
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all()
    # the others' tiles are cut elsewhere now, so they are near, not the same bit for bit
    p.check(out, lse, skip=(0,))
    for bad in (-1, p.kv.num_blocks):
        err.zero_()
        p.bt[0, 2, 0] = bad
        out, lse = p.run(err=err)
        assert err.item() > 2
        x, k, v = p.rows[2]
        on = np.array([R.place(i, 2, 16, 1)[:2] != (0, 0) for i in x])
        rows, p.rows[2] = p.rows[2], (x[on], k[:, on], v[:, on])
        p.check(out, lse, skip=(0, 1))
        p.rows[2] = rows


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
def test_visible_nan_and_infinities_reach_the_output(lib, cache):
    q = F32 if cache == F32 else BF16
    p = Problem(lib, cache, q, 2, 1, 128, 1, 16, 1, [50, 50, 50])
    page = int(p.bt[0, 0, 0])
    bad = torch.tensor(float("nan")).to(p.kv.v_pools[0].dtype).cuda()
    if cache == E4M3:
        p.kv.v_pools[0].view(torch.uint8)[page, 0, 3, 7] = bad.view(torch.uint8)
    else:
        p.kv.v_pools[0][page, 0, 3, 7] = bad
    out, lse = p.run()
    assert torch.isnan(out[0, :, 7]).all()
    assert torch.isfinite(out[0, :, :7]).all() and torch.isfinite(lse).all()
    assert torch.isfinite(out[1:]).all()
    if cache != E4M3:               # a key of -inf products: a weight of nothing
        p.q[1] = 1.0
        p.kv.k_pools[0][int(p.bt[0, 1, 0]), 0, 5] = -float("inf")
        out, lse = p.run()
        assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()
        p.kv.k_pools[0][:] = -float("inf")
        p.q[:] = 1.0
        out, lse = p.run()
        assert (lse[1] == -float("inf")).all() and (out[1] == 0).all()


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("room", [0, 1 << 20])
@pytest.mark.parametrize("one", [False, True])
def test_values_of_any_size(lib, cache, one, room):
    """Scales and values from the smallest to the largest: what counts is not lost beside them."""
    q = F32 if cache == F32 else BF16
    lens = [9] if one else [400, 31]
    p = Problem(lib, cache, q, 4, 2, 128, 2, 16, 1, lens, seed=3, room=room)
    for b in range(len(lens)):
        x, k, v = p.rows[b]
        for vb in range(p.bt.shape[-1]):
            for r in range(2):
                page = int(p.bt[r, b, vb])
                if page < 0:
                    continue
                f = 2.0 ** ((vb * 7 + r * 3) % 5 * 10 - 20)
                if cache == E4M3:
                    p.kv.scales[r][page, :, 1] *= f
                else:
                    p.kv.v_pools[r][page] *= f
                for j, pos in enumerate(x):
                    if R.place(pos, 2, 16, 1)[:2] == (r, vb):
                        v[:, j] *= f
    out, lse = p.run()
    p.check(out, lse)


def test_pages_that_hold_only_zeros(lib):
    """Their tokens count in the sum, however small the pages' scales."""
    p = Problem(lib, E4M3, BF16, 4, 2, 128, 2, 16, 1, [200, 40])
    for b in range(2):
        x, k, v = p.rows[b]
        for r in range(2):
            page = int(p.bt[r, b, 0])
            p.kv.v_pools[r].view(torch.uint8)[page] = 0
            p.kv.scales[r][page, :, 1] = 2.0 ** -60
            v[:, [j for j, pos in enumerate(x) if R.place(pos, 2, 16, 1)[:2] == (r, 0)]] = 0.0
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("cache", [BF16, E4M3], ids=str)
def test_a_long_flat_tail_beside_one_large_weight(lib, cache):
    """Half of the mass in one token, the other half spread over 3000 small ones with like values."""
    p = Problem(lib, cache, BF16, 4, 1, 128, 1, 16, 1, [3001])
    dt = p.kv.k_pools[0].dtype
    x, k, v = p.rows[0]
    p.q[:] = 1.0
    p.q64[:] = 1.0
    k[:], v[:] = 0.0, 1.5
    k[0, 17] = 1.0 / 16
    p.scale = float(np.log(3000.0)) / (128 / 16)
    for i, (pool, rows) in enumerate(((p.kv.k_pools[0], k), (p.kv.v_pools[0], v))):
        if cache == E4M3:
            p.kv.scales[0][..., i] = 1.0
        vb, loc = np.divmod(x, 16)
        page = p.bt[0, 0].cpu().numpy()[vb]
        full = np.zeros(pool.shape, np.float32)
        full[page, 0, loc] = rows[0]
        pool.copy_(torch.from_numpy(full).to(dt).cuda())
    out, lse = p.run(out_dtype=F32)
    p.check(out, lse)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("room", [0, 1 << 20])
def test_captured_with_changing_lengths(lib, cache, room):
    q = F32 if cache == F32 else BF16
    p = Problem(lib, cache, q, 8, 2, 128, 2, 16, 1, [700, 650, 20], cap=30.0, sink=True, room=room)
    B, Hq, d = p.q.shape
    ws = torch.empty(lib.scored_workspace_size(p.layout, B, Hq, 2, d), dtype=torch.uint8,
                     device="cuda")
    out, lse = torch.empty_like(p.q), torch.empty((B, Hq), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.run(out=out, out_lse=lse, workspace=ws, err=err)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run(out=out, out_lse=lse, workspace=ws, err=err)
    for lens in ([700, 650, 20], [1, 0, 20], [333, 650, 7]):
        p.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        ws.fill_(255)
        g.replay()
        want = p.run()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert err.item() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("room", [0, 1 << 20])
def test_requests_that_see_nothing(lib, cache, room):
    """A document that begins at or behind the end; with and without a sink."""
    q = F32 if cache == F32 else BF16
    for sink in (False, True):
        p = Problem(lib, cache, q, 8, 2, 128, 2, 16, 1, [70, 40, 33], sink=sink, room=room)
        first = torch.tensor([70, 1000, -3], dtype=torch.int32, device="cuda")
        p.form = lib.Scores(first=first, window=20 if room == 0 else 1 << 30)
        out, lse = p.run()
        assert (out[:2] == 0).all()
        want = p.dsink.expand(2, -1) if sink else torch.full_like(lse[:2], -np.inf)
        assert torch.equal(lse[:2], want)
        x, k, v = p.rows[2]
        n = 13 if room == 0 else 0
        p.rows[2] = (x[n:], k[:, n:], v[:, n:])
        p.check(out, lse, skip=(0, 1))


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
def test_more_requests_than_threads(lib, cache):
    """Hundreds of requests, some empty, so that a thread counts several; and their ranks apart."""
    q = F32 if cache == F32 else BF16
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.choice([0, 0, 1, 5, 16, 40, 100], 700)]
    lens[350] = 900
    p = Problem(lib, cache, q, 2, 1, 64, 2, 16, 1, lens, alibi=True)
    out, lse = p.run()
    p.check(out, lse)
    po, pl = p.partial(p.layout, p.q, p.kv, p.dlens, p.scale, p.form)
    for r in range(2):
        p.check(po[r], pl[r], rank=r)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
def test_windows_of_more_units_than_ctas(lib, cache):
    """Windows and kept tokens where units are cut anywhere, and several lie in one CTA."""
    q = F32 if cache == F32 else BF16
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.choice([0, 1, 20, 45, 64, 333, 500], 170)]
    p = Problem(lib, cache, q, 8, 4, 64, 2, 16, 1, lens, window=37, prefix=5, docs=True, cap=20.0,
                sink=True)
    p.check(*p.run())


def test_calls_at_once(lib):
    """Calls on several streams, each with a workspace of its own, beside one another."""
    ps = [Problem(lib, c, BF16, 8, 2, 128, 2, 16, 1, [900, 20], seed=i, cap=30.0)
          for i, c in enumerate((E4M3, BF16, E4M3, BF16))]
    want = [p.run() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for p, s in zip(ps, streams):
            got.append((p, p.run(stream=s)))
    torch.cuda.synchronize()
    for p, (o, l) in got:
        w = want[ps.index(p)]
        assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_outputs_are_tensors_of_their_own(lib):
    p = Problem(lib, E4M3, BF16, 3, 1, 64, 1, 16, 1, [50])
    out, lse = p.run()
    assert out.is_contiguous() and lse.is_contiguous() and out._base is None and lse._base is None
    o, l = out.clone(), lse.clone()
    out.zero_()
    assert torch.equal(lse, l)
    out.copy_(o)
    lse.zero_()
    assert torch.equal(out, o)


def test_another_stream(lib):
    p = Problem(lib, E4M3, BF16, 8, 2, 128, 2, 16, 1, [700, 20])
    want = p.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = p.run(stream=s)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_refusals(lib):
    p = Problem(lib, E4M3, BF16, 8, 2, 128, 2, 16, 1, [70, 20])
    w = Problem(lib, BF16, BF16, 8, 2, 128, 2, 16, 1, [70, 20])
    L = p.layout
    with pytest.raises(lib.DcpError, match="8 bits"):
        lib.scored_decode_gqa(L, p.q, p.kv, p.dlens, 1.0, p.form)
    with pytest.raises(lib.DcpError, match="PagedKV8"):
        lib.q8_decode_gqa(L, p.q, w.kv, p.dlens, 1.0)
    with pytest.raises(lib.DcpError):
        lib.decode_gqa(L, p.q, p.kv, lib.local_seq_lens(L, p.dlens), 1.0)
    with pytest.raises(lib.DcpError, match="Float"):
        lib.scored_decode_gqa(L, w.q.float(), w.kv, w.dlens, 1.0, w.form)
    for kw in (dict(scores=lib.Scores(cap=-1.0)), dict(scores=lib.Scores(window=-1)),
               dict(scores=lib.Scores(prefix=-1)), dict(scores=lib.Scores(cap=float("nan"))),
               dict(scores=lib.Scores(slopes=torch.ones(4, device="cuda"))),
               dict(scores=lib.Scores(first=torch.zeros(2, device="cuda"))),
               dict(sink=torch.zeros(3, device="cuda")), dict(out=p.q),
               dict(out_dtype=torch.float16),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(lib.DcpError):
            lib.q8_decode_gqa(L, p.q, p.kv, p.dlens, 1.0, **kw)
    for bad in (p.dlens[:1], p.dlens.long()):
        with pytest.raises(lib.DcpError):
            lib.q8_decode_gqa(L, p.q, p.kv, bad, 1.0)
    with pytest.raises(lib.DcpError):
        lib.q8_decode_gqa(L, p.q, p.kv, p.dlens, float("inf"))
    with pytest.raises(lib.DcpError):
        lib.q8_decode_gqa(lib.Layout(2, 32, 1), p.q, p.kv, p.dlens, 1.0)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("room", [0, 1 << 20])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e6, -1e9, 1e30])
def test_any_scale(lib, cache, scale, room):
    """Scores of nothing, below 0, and so large that one token has all the weight."""
    q = F32 if cache == F32 else BF16
    p = Problem(lib, cache, q, 4, 2, 64, 2, 16, 1, [150, 33, 1], sink=scale == 0.0, room=room)
    p.scale = scale
    out, lse = p.run()
    if abs(scale) < 1:
        p.check(out, lse)
        return
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(3):
        x, k, v = p.rows[b]
        for h in range(4):
            t = np.sort(k[h // 2] @ p.q64[b, h])
            t = (t if scale > 0 else t[::-1])
            # the two largest are apart by more than the error of a product of 64 terms
            size = (np.abs(k[h // 2]) @ np.abs(p.q64[b, h])).max() * 68 * 2.0 ** -24
            best = (k[h // 2] @ p.q64[b, h] * np.sign(scale)).argmax()
            assert abs(l[b, h] - abs(t[-1] * scale) * np.sign(t[-1] * scale)) <= 2 * size * abs(scale)
            if len(t) > 1 and abs(t[-1] - t[-2]) > 2 * size + 100 / abs(scale):
                assert (np.abs(o[b, h] - v[h // 2][best]) <= np.abs(v[h // 2][best]) * 2.0 ** -7).all()
