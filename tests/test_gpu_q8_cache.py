"""The 8-bit cache: what is written, read back, copied and attended, against 64 bits.

Numbers are held exactly as the definition says, so pools and scales are compared for equality."""
import numpy as np
import pytest
import torch

from tests import scored_ref as S
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Cache:
    """A cache and its 64-bit model; what nobody has written holds garbage."""

    def __init__(self, lib, rng, Hkv, d, dcp, bs, I, room, nb_more=3, shared=False):
        self.lib, self.layout, self.geo = lib, lib.Layout(dcp, bs, I), (dcp, bs, I)
        tables = 1 if shared else dcp
        bt, nb = R.random_tables(rng, room, tables, bs * dcp // tables, spare=nb_more)
        self.bt = bt
        junk = rng.integers(0, 256, (2, dcp, nb, Hkv, bs, d)).astype(np.uint8)
        pools = torch.from_numpy(junk).cuda().view(E4M3)
        sc = torch.from_numpy(np.float32(rng.choice([np.nan, -1.0, 0.0, np.inf, 3.7e5],
                                                    (dcp, nb, Hkv, 4)))).cuda()
        self.kv = lib.PagedKV8(list(pools[0]), list(pools[1]), list(sc),
                               torch.from_numpy(bt).cuda(), nb)
        self.pools = [pools[i].double().cpu().numpy() for i in range(2)]
        self.scales = [sc[..., i].double().cpu().numpy() for i in range(2)]
        self.spare = sc[..., 2:].clone()

    def append(self, k, v, q_start, ctx, **kw):
        self.lib.q8_append_gqa(self.layout, k, v, self.kv,
                               torch.tensor(q_start, dtype=torch.int32, device="cuda"),
                               torch.tensor(ctx, dtype=torch.int32, device="cuda"), **kw)

    def model(self, k, v, q_start, ctx, skip=()):
        for b in range(len(ctx)):
            if b in skip:
                continue
            rows = slice(q_start[b], q_start[b + 1])
            table = [self.bt[r if self.bt.shape[0] > 1 else 0, b] for r in range(self.geo[0])]
            for i, x in enumerate((k, v)):
                S.append(self.pools[i], self.scales[i], x[rows].double().cpu().numpy(), table,
                         ctx[b], *self.geo)

    def check(self):
        for i, got in enumerate((self.kv.k_pools, self.kv.v_pools)):
            got = torch.stack(got).double().cpu().numpy()
            assert np.array_equal(got, self.pools[i], equal_nan=True)
        sc = torch.stack(self.kv.scales)
        for i in range(2):
            assert np.array_equal(sc[..., i].double().cpu().numpy(), self.scales[i], equal_nan=True)
        assert np.array_equal(sc[..., 2:].cpu().numpy(), self.spare.cpu().numpy(), equal_nan=True)


def rows(rng, N, Hkv, d, dtype, fused, sizes=(1.0,)):
    """k, v [N, Hkv, d]; each token of a size of its own."""
    s = rng.choice(sizes, (N, 1, 1))
    x = torch.from_numpy(rng.standard_normal((N, 3 * Hkv, d)) * s).to(dtype).cuda()
    q, k, v = x.split([Hkv, Hkv, Hkv], 1)
    return (k, v) if fused else (k.contiguous(), v.contiguous())


# dtype, Hkv, d, dcp, bs, I, ctx, T, fused
CASES = [
    (BF16, 8, 128, 8, 16, 1, [1000, 0, 5, 16 * 8 * 3, 127], [1, 1, 1, 1, 1], True),
    (BF16, 2, 128, 2, 16, 1, [0], [1], False),
    (BF16, 2, 128, 2, 16, 1, [7, 33], [300, 95], True),
    (BF16, 1, 64, 3, 32, 4, [0, 50, 95, 96, 97], [200, 1, 37, 0, 64], True),
    (F32, 2, 64, 3, 64, 4, [77, 0], [37, 500], False),
    (F32, 1, 256, 1, 16, 16, [5, 30], [50, 7], True),
    (BF16, 1, 256, 2, 128, 2, [100], [600], False),
    (BF16, 3, 96, 2, 24, 3, [11, 47], [90, 2], True),
    (BF16, 1, 32, 16, 8, 8, [3], [400], False),
    (BF16, 1, 128, 4, 1, 1, [3, 0], [20, 9], False),
    (F32, 1, 96, 2, 3, 3, [3, 0], [20, 9], True),
    (F32, 2, 160, 5, 48, 3, [13, 0, 500], [31, 9, 200], True),
    (BF16, 2, 224, 2, 16, 4, [13, 0], [31, 90], False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}-H{c[1]}-d{c[2]}-dcp{c[3]}-bs{c[4]}-I{c[5]}-{sum(c[7])}of{max(c[6])}")
def test_append(lib, case):
    dtype, H, d, dcp, bs, I, ctx, T, fused = case
    rng = np.random.default_rng(d + sum(T))
    # three runs one behind the other, with tokens of unlike sizes
    c = Cache(lib, rng, H, d, dcp, bs, I, [x + 3 * t for x, t in zip(ctx, T)])
    if max(ctx):
        first = np.r_[0, np.cumsum(ctx)]
        k, v = rows(rng, first[-1], H, d, dtype, fused)
        c.append(k, v, first, [0] * len(ctx))
        c.model(k, v, first, [0] * len(ctx))
        c.check()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(3):
        start = np.r_[0, np.cumsum(T)]
        k, v = rows(rng, start[-1], H, d, dtype, fused, (0.0, 1e-3, 1.0, 30.0, 1e4))
        at = [x + i * t for x, t in zip(ctx, T)]
        c.append(k, v, start, at, err=err)
        c.model(k, v, start, at)
        c.check()
    assert err.item() == 0


def test_rows_of_no_request_and_bad_requests(lib):
    """Rows in front of, between and behind the sequences are not read; requests that cannot be
    are counted and left alone."""
    rng = np.random.default_rng(5)
    c = Cache(lib, rng, 2, 64, 2, 16, 1, [200] * 6)
    k, v = rows(rng, 60, 2, 64, BF16, True)
    k[50:] = float("nan")
    k[:3] = float("nan")
    start = np.array([3, 10, 10, 30, 40, 45, 50])
    ctx = [9, 0, -1, 224 - 9, 224 - 2, 17]     # the table has room for 224
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(k, v, start, ctx, err=err)
    c.model(k, v, start, ctx, skip=(2, 3, 4))
    c.check()
    assert err.item() == 3
    # starts that go down or leave the rows: no request is read beyond them
    for start, skip in ([3, 10, 5, 30, 40, 45, 50], (1,)), ([-4, 10, 10, 30, 40, 45, 70], (0, 5)):
        err.zero_()
        before = [torch.stack(x).view(torch.uint8).clone() for x in (c.kv.k_pools, c.kv.v_pools)]
        c.append(k, v, start, [224] * 6 if len(skip) == 1 else [9, 0, 0, 0, 0, 0], err=err)
        assert err.item() >= len(skip)
        if len(skip) == 1:      # all of them refused
            for x, y in zip(before, (c.kv.k_pools, c.kv.v_pools)):
                assert torch.equal(torch.stack(y).view(torch.uint8), x)


def test_pages_that_are_not_there(lib):
    rng = np.random.default_rng(6)
    c = Cache(lib, rng, 2, 64, 2, 16, 1, [100])
    for bad in (-1, c.kv.num_blocks, 2 ** 31 - 1):
        c.bt[1, 0, 1] = bad
        c.kv.block_table.copy_(torch.from_numpy(c.bt))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = rows(rng, 90, 2, 64, BF16, False)
        c.append(k, v, [0, 90], [5], err=err)
        c.model(k, v, [0, 90], [5])
        c.check()
        assert err.item() == 1


@pytest.mark.parametrize("B", [31, 32, 33, 150])
def test_many_requests(lib, B):
    """Short runs of many requests, long stretches of which have none."""
    rng = np.random.default_rng(B)
    T = rng.choice([0, 1, 1, 2, 40], B)
    T[3:3 + B // 2] = 0
    ctx = rng.integers(0, 60, B)
    c = Cache(lib, rng, 1, 32, 2, 16, 1, [int(x + 2 * t) for x, t in zip(ctx, T)])
    for i in range(2):
        start = np.r_[0, np.cumsum(T)]
        k, v = rows(rng, int(start[-1]), 1, 32, BF16, True, (1.0, 20.0))
        at = [int(x + i * t) for x, t in zip(ctx, T)]
        c.append(k, v, start, at)
        c.model(k, v, start, at)
        c.check()


def test_odd_numbers(lib):
    """Zeros, infinities, NaN, the smallest and the largest numbers."""
    rng = np.random.default_rng(7)
    c = Cache(lib, rng, 1, 64, 1, 16, 1, [96])
    odd = [0.0, -0.0, float("inf"), -float("inf"), float("nan"), 3.3e38, -1e-38, 1e-45, 2.0 ** -70,
           448.0, 449.0, 464.0, 465.0, 1.0, 2.0 ** -9, 2.0 ** -10]
    for dtype in (F32, BF16):
        for j, few in enumerate((odd, [0.0, float("nan")], [float("inf"), 1.0], odd[9:], [1e-30], [0.0])):
            x = torch.tensor(few, dtype=torch.float64)
            k = x[torch.from_numpy(rng.integers(0, len(few), (16, 1, 64)))].to(dtype).cuda()
            v = x[torch.from_numpy(rng.integers(0, len(few), (16, 1, 64)))].to(dtype).cuda()
            for t0 in (0, 5):                     # the second run is written over the first's end
                c.append(k[t0:], v[t0:], [0, 16 - t0], [16 * j + t0])
                c.model(k[t0:], v[t0:], [0, 16 - t0], [16 * j + t0])
                c.check()


def test_scales_of_others(lib):
    """A page whose scale is no power of two: the larger of it and what the tokens need stays."""
    rng = np.random.default_rng(8)
    c = Cache(lib, rng, 2, 64, 1, 16, 1, [32])
    for s, size in ((0.037, 1.0), (0.003, 1.0), (1e-30, 1.0)):
        for r, held in enumerate(c.kv.scales):
            held[..., :2] = s
            for i in range(2):
                c.scales[i][r] = np.float32(s)
        k, v = rows(rng, 6, 2, 64, BF16, False, (size,))
        c.append(k, v, [0, 6], [7])
        got = torch.stack(c.kv.k_pools).double().cpu().numpy()
        sc = torch.stack(c.kv.scales)[..., 0].double().cpu().numpy()
        page = c.bt[0, 0, 0]
        for h in range(2):
            new = max(np.float64(np.float32(s)), S.need(k[:, h].abs().max().item()))
            assert sc[0, page, h] == new
            want = S.nearest8(k[:, h].double().cpu().numpy() / new)
            # the quotient is rounded to 32 bits first: next to a border the neighbour
            far = np.abs(got[0, page, h, 7:13] - want)
            assert (far <= 2.0 ** -3 * np.maximum(np.abs(want), 2.0 ** -6)).all()
            assert (far == 0).mean() > 0.99


def test_a_token_at_a_time_or_all_at_once(lib):
    """Prefix by prefix: what is read back of a request that came in runs of any length is near
    what came in, and a run's pages do not depend on its neighbours."""
    rng = np.random.default_rng(9)
    k, v = rows(rng, 150, 2, 64, BF16, False, (1.0, 3.0))
    for runs in ([150], [1] * 150, [7, 64, 1, 78]):
        c = Cache(lib, rng, 2, 64, 2, 16, 1, [150, 150])
        at = 0
        for n in runs:
            c.append(k[at:at + n], v[at:at + n], [0, 0, n], [3, at])
            c.model(k[at:at + n], v[at:at + n], [0, 0, n], [3, at])
            at += n
        c.check()
        pos = torch.arange(150, device="cuda")
        gk, gv = lib.q8_gather_gqa(c.layout, c.kv, torch.ones(150, dtype=torch.int32, device="cuda"),
                                   pos, dtype=F32)
        for got, x in ((gk, k), (gv, v)):
            # half a step of e4m3 for the first rounding and as much for each requantising, of
            # which a page whose size grows from the smallest to the largest here has few, and
            # they only touch what the larger scale cannot hold: half of its smallest step
            step = 2.0 ** -10 * 2.0 ** -4          # pages' scales are at most 2^-4 (max < 28)
            far = (got.double() - x.double()).abs()
            assert (far <= x.double().abs() * 2.0 ** -4 + 3 * step).all()


# dtype, Hkv, d, dcp, bs, I, T
GATHER = [(BF16, 8, 128, 8, 16, 1, 500), (F32, 8, 128, 2, 16, 1, 77), (BF16, 1, 64, 3, 64, 4, 1),
          (F32, 3, 96, 2, 24, 3, 131), (BF16, 2, 256, 1, 1, 1, 40), (BF16, 5, 32, 16, 8, 8, 9000)]


@pytest.mark.parametrize("case", GATHER, ids=lambda c: f"{str(c[0])[6:]}-H{c[1]}-d{c[2]}-dcp{c[3]}-bs{c[4]}-T{c[6]}")
def test_gather(lib, case):
    dtype, H, d, dcp, bs, I, T = case
    rng = np.random.default_rng(T)
    lens = [min(T, 700), 33, 1]
    c = Cache(lib, rng, H, d, dcp, bs, I, lens, shared=T == 131)
    for i, s in enumerate(c.kv.scales):
        s[..., :2] = torch.from_numpy(2.0 ** rng.integers(-12, 12, s[..., :2].shape)).float().cuda()
    req = rng.integers(0, 3, T)
    pos = np.array([rng.integers(0, lens[b]) for b in req])
    bad = {3: (5, 0), 7: (-1, 0), 9: (0, -4), 11: (0, 1 << 40), 13: (2, 100000)} if T > 20 else {}
    for t, (b, x) in bad.items():
        req[t], pos[t] = b, x
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = lib.q8_gather_gqa(c.layout, c.kv, torch.from_numpy(req).int().cuda(),
                             torch.from_numpy(pos).cuda(), dtype=dtype, err=err)
    assert err.item() == len(bad) and k.dtype == dtype and k.shape == (T, H, d)
    sc = torch.stack(c.kv.scales).double().cpu().numpy()
    for i, got in enumerate((k, v)):
        want = np.zeros((T, H, d))
        for t in range(T):
            if t in bad:
                continue
            r, vb, loc = R.place(pos[t], dcp, bs, I)
            page = c.bt[r if c.bt.shape[0] > 1 else 0, req[t], vb]
            want[t] = c.pools[i][r, page, :, loc] * sc[r, page, :, i, None]
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


def test_a_table_of_more_than_its_pages(lib):
    """Offsets behind 2^31 bytes of one rank's pool."""
    bs, H, d = 64, 8, 128
    nb = (1 << 31) // (bs * H * d) + 40
    L = lib.Layout(1, bs, 1)
    bt = torch.tensor([[nb - 1, 0, nb - 2]], dtype=torch.int32, device="cuda")
    kv = lib.PagedKV8.new(L, nb, H, d, bt)
    rng = np.random.default_rng(1)
    k, v = rows(rng, 150, H, d, BF16, False)
    st = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    lib.q8_append_gqa(L, k, v, kv, st, torch.zeros(1, dtype=torch.int32, device="cuda"))
    pos = torch.arange(150, device="cuda")
    gk, gv = lib.q8_gather_gqa(L, kv, torch.zeros(150, dtype=torch.int32, device="cuda"), pos,
                               dtype=F32)
    for got, x in ((gk, k), (gv, v)):
        assert ((got - x.float()).abs() <= x.float().abs() * 2.0 ** -4 + 2.0 ** -10 * 2.0 ** -6).all()
    q = torch.from_numpy(rng.standard_normal((1, 32, d))).to(BF16).cuda()
    out, lse = lib.q8_decode_gqa(L, q, kv, torch.tensor([150], dtype=torch.int32, device="cuda"),
                                 d ** -0.5)
    for h in range(32):
        o, l, to, tl = S.attend(BF16, BF16, q[0, h].double().cpu().numpy(),
                                gk[:, h // 4].double().cpu().numpy(),
                                gv[:, h // 4].double().cpu().numpy(), np.arange(150), 150,
                                d ** -0.5)
        assert (np.abs(out[0, h].double().cpu().numpy() - o) <= to).all()
        assert abs(lse[0, h].item() - l) <= tl


def test_captured_with_changing_lengths(lib):
    rng = np.random.default_rng(12)
    c = Cache(lib, rng, 2, 64, 2, 16, 1, [200, 200])
    k, v = rows(rng, 64, 2, 64, BF16, False)
    start = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    run = lambda: lib.q8_append_gqa(c.layout, k, v, c.kv, start, ctx)  # noqa: E731
    run()
    c.model(k, v, [0, 10, 20], [0, 5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for s, x in (([0, 64, 64], [10, 15]), ([0, 0, 30], [74, 3]), ([5, 6, 7], [74, 33])):
        start.copy_(torch.tensor(s, dtype=torch.int32))
        ctx.copy_(torch.tensor(x, dtype=torch.int32))
        g.replay()
        c.model(k, v, s, x)
        c.check()


def test_serving_steps(lib):
    """Prompt, steps, a fork with its copies, and a trim that is written over: rotated keys go into
    the 8-bit cache and the window's tokens are attended, over the pages' own state."""
    rng = np.random.default_rng(20)
    dcp, bs, I, H, Hq, d, nb = 2, 16, 1, 2, 8, 64, 64
    L = lib.Layout(dcp, bs, I)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = lib.Pages.new(L, 3, 8, nb)
    caches = [lib.PagedKV8.new(L, nb, H, d, pages.block_table) for _ in range(2)]
    pools = lib.Q8Pools(caches)
    form = lib.Scores(cap=30.0, window=40, prefix=2)
    inv = torch.from_numpy((1e4 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)).cuda()
    none = [torch.zeros((1, H, bs, d), dtype=BF16, device="cuda") for _ in range(dcp)]
    seen = [[], [], []]      # what each request's tokens were, rotated: (k, v) per layer

    def step(reqs, T):
        """T new tokens of each of these requests, in every layer; checks the last one's attention."""
        lens = pages.seq_lens.tolist()
        new = [lens[b] + T for b in reqs]
        src, dst = lib.pages_resize(L, pages, i32(reqs), i32(new))
        lib.q8_pages_copy(L, pools, src, dst)
        N, start, ctx = len(reqs) * T, [0], lens[:]
        for b in range(3):
            start.append(start[-1] + (T if b in reqs else 0))
        pos = torch.tensor([lens[b] + t for b in sorted(reqs) for t in range(T)], device="cuda")
        rows_ = []
        for c in caches:
            x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * H, d))).to(BF16).cuda()
            q, k, v = x.split([Hq, H, H], 1)
            kr = torch.empty((N, H, d), dtype=BF16, device="cuda")
            skip = torch.full((dcp, N), -1, dtype=torch.int64, device="cuda")
            q = lib.rope_write_gqa(L, q, k, v, pos, inv, skip, none, none, 1, k_out=kr)
            lib.q8_append_gqa(L, kr, v, c, i32(start), i32(ctx))
            rows_.append((q, kr, v))
        for n, b in enumerate(sorted(reqs)):
            for t in range(T):
                seen[b].append([(k[n * T + t].double().cpu().numpy(), v[n * T + t].double().cpu().numpy())
                                for _, k, v in rows_])
        full = pages.seq_lens.tolist()
        last = torch.stack([rows_[1][0][n * T + T - 1] for n in range(len(reqs))])
        qs = torch.zeros((3, Hq, d), dtype=BF16, device="cuda")
        qs[sorted(reqs)] = last
        # no request here has more than a few sizes of scale, so a number is off by 2^-4 of
        # itself for its own rounding, and by half a smallest step of the page's scale, three
        # times over at most; the attention over what is held is checked to its own bounds
        out, lse = lib.q8_decode_gqa(L, qs, caches[1], pages.seq_lens, d ** -0.5, scores=form)
        for b in range(3):
            if full[b] == 0:
                continue
            p = torch.arange(full[b], device="cuda")
            gk, gv = lib.q8_gather_gqa(L, caches[1], torch.full((full[b],), b, dtype=torch.int32,
                                                                 device="cuda"), p, dtype=F32)
            for got, i in ((gk, 0), (gv, 1)):
                want = np.stack([s[1][i] for s in seen[b]])
                far = np.abs(got.double().cpu().numpy() - want)
                assert (far <= np.abs(want) * 2.0 ** -4 + 3 * 2.0 ** -10 * 2.0 ** -5).all()
            if b not in reqs:
                continue
            x = np.nonzero(S.seen_mask(full[b], 40, 2, 0))[0]
            for h in range(Hq):
                o, l, to, tl = S.attend(BF16, BF16, qs[b, h].double().cpu().numpy(),
                                        gk[x, h // 4].double().cpu().numpy(),
                                        gv[x, h // 4].double().cpu().numpy(), x, full[b], d ** -0.5,
                                        cap=30.0)
                assert (np.abs(out[b, h].double().cpu().numpy() - o) <= to).all()
                assert abs(lse[b, h].item() - l) <= tl

    step([0], 37)
    for _ in range(3):
        step([0], 1)
    step([0, 1], 20)
    # request 2 becomes a copy of request 0: the open page is copied with its scales
    src, dst = lib.pages_fork(L, pages, i32([0]), i32([2]))
    lib.q8_pages_copy(L, pools, src, dst)
    seen[2] = list(seen[0])
    step([0, 2], 1)
    step([2], 5)
    # five tokens are taken back and others written there
    n = pages.seq_lens.tolist()[2] - 5
    src, dst = lib.pages_resize(L, pages, i32([2]), i32([n]))
    lib.q8_pages_copy(L, pools, src, dst)
    del seen[2][n:]
    step([0, 1, 2], 3)


def test_refusals(lib):
    rng = np.random.default_rng(2)
    c = Cache(lib, rng, 2, 64, 2, 16, 1, [50])
    k, v = rows(rng, 10, 2, 64, BF16, False)
    st = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    x = torch.zeros(1, dtype=torch.int32, device="cuda")
    app = lambda **kw: lib.q8_append_gqa(**{**dict(  # noqa: E731
        layout=c.layout, k=k, v=v, kv=c.kv, q_start=st, ctx_lens=x), **kw})
    for kw in (dict(k=k.half(), v=v.half()), dict(v=v.float()), dict(v=v[:5]), dict(k=k[..., :32]),
               dict(q_start=st.long()), dict(q_start=st[:1]), dict(ctx_lens=x.long()),
               dict(layout=lib.Layout(2, 32, 1)), dict(layout=lib.Layout(3, 16, 1)),
               dict(k=k.cpu()), dict(k=k.transpose(0, 1)),
               dict(k=torch.empty(1, 10, 2, 64, dtype=BF16, device="cuda")),
               dict(k=torch.empty(10 * 128 + 1, dtype=BF16, device="cuda")[1:].view(10, 2, 64))):
        with pytest.raises(lib.DcpError):
            app(**kw)
    with pytest.raises(lib.DcpError, match="PagedKV8"):
        app(kv=lib.PagedKV([p.to(BF16) for p in c.kv.k_pools], [p.to(BF16) for p in c.kv.v_pools],
                           c.kv.block_table, c.kv.num_blocks))
    # keys that lie in the cache itself
    inside = c.kv.k_pools[0].view(torch.uint8).view(-1)[:10 * 256].view(BF16).view(10, 2, 64)
    with pytest.raises(lib.DcpError):
        app(k=inside)
    pos = torch.arange(10, device="cuda")
    req = torch.zeros(10, dtype=torch.int32, device="cuda")
    gat = lambda **kw: lib.q8_gather_gqa(**{**dict(  # noqa: E731
        layout=c.layout, kv=c.kv, req_idx=req, positions=pos), **kw})
    for kw in (dict(dtype=torch.float16), dict(positions=pos.int()), dict(positions=pos[:5]),
               dict(req_idx=req.long()), dict(k_out=torch.empty((9, 2, 64), dtype=BF16, device="cuda")),
               dict(k_out=k, v_out=k), dict(k_out=inside)):
        with pytest.raises(lib.DcpError):
            gat(**kw)
    for bad in (dict(k_pools=[p.view(torch.uint8) for p in c.kv.k_pools]),
                dict(scales=[s[..., :2].contiguous() for s in c.kv.scales]),
                dict(scales=[s.double() for s in c.kv.scales])):
        with pytest.raises(lib.DcpError):
            lib.PagedKV8(**{**dict(k_pools=c.kv.k_pools, v_pools=c.kv.v_pools, scales=c.kv.scales,
                                   block_table=c.kv.block_table, num_blocks=c.kv.num_blocks), **bad})
    with pytest.raises(lib.DcpError):
        c.kv.struct()


@pytest.mark.parametrize("qtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("graph", [False, True])
def test_steps_in_a_row(lib, qtype, graph):
    """Steps that follow one another without a wait (each call's kernels may start before those
    in front of them have ended) give what they give one by one: lengths are raised on the
    device, tokens that make scales grow are appended, and the cache is attended and read."""
    dcp, bs, I, H, Hq, d, steps = 2, 16, 1, 2, 4, 64, 60
    L = lib.Layout(dcp, bs, I)
    rng = np.random.default_rng(33)
    bt, nb = R.random_tables(rng, [200, 150, 90], dcp, bs)
    tab = torch.from_numpy(bt).cuda()
    k, v = (torch.from_numpy(rng.standard_normal((steps, 3, H, d))
                             * rng.choice([0.1, 1.0, 40.0], (steps, 3, 1, 1))).to(BF16).cuda()
            for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((steps, 3, Hq, d))).to(qtype).cuda()
    start = torch.arange(4, dtype=torch.int32, device="cuda")
    req = torch.arange(3, dtype=torch.int32, device="cuda").repeat_interleave(40)
    form = lib.Scores(cap=20.0, window=50, prefix=3)

    def run(wait):
        kv = lib.PagedKV8.new(L, nb, H, d, tab)
        for p in kv.k_pools + kv.v_pools:
            p.view(torch.uint8).fill_(0x7f)
        ctx = torch.tensor([0, 17, 30], dtype=torch.int32, device="cuda")
        first = torch.zeros((47, H, d), dtype=BF16, device="cuda") + 0.5
        fs = torch.tensor([0, 0, 17, 47], dtype=torch.int32, device="cuda")
        lib.q8_append_gqa(L, first, first, kv, fs, torch.zeros_like(ctx))
        lens, pos = torch.empty_like(ctx), torch.empty(120, dtype=torch.int64, device="cuda")
        back = torch.arange(40, device="cuda").repeat(3)
        out = torch.zeros((steps, 3, Hq, d), dtype=qtype, device="cuda")
        lse = torch.zeros((steps, 3, Hq), device="cuda")
        rows_ = torch.zeros((steps, 120, H, d), device="cuda")

        def steps_():
            for t in range(steps):
                lib.q8_append_gqa(L, k[t], v[t], kv, start, ctx)
                wait()
                torch.add(ctx, 1, out=lens)
                lib.q8_decode_gqa(L, q[t], kv, lens, d ** -0.5, scores=form, out=out[t],
                                  out_lse=lse[t])
                wait()
                torch.sub(lens[:, None].long(), 1 + back.view(3, 40), out=pos.view(3, 40)).clamp_(min=0)
                lib.q8_gather_gqa(L, kv, req, pos, k_out=rows_[t],
                                  v_out=torch.empty_like(rows_[t]))
                wait()
                ctx.copy_(lens)

        if graph and wait is nothing:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                steps_()
            g.replay()
        else:
            steps_()
        torch.cuda.synchronize()
        return out, lse, rows_, torch.stack(kv.scales)[..., :2], torch.stack(kv.k_pools).view(torch.uint8)

    def nothing():
        pass

    want = run(torch.cuda.synchronize)
    got = run(nothing)
    for a, b in zip(got, want):
        assert torch.equal(torch.nan_to_num(a) if a.is_floating_point() else a,
                           torch.nan_to_num(b) if b.is_floating_point() else b)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
