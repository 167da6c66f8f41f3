"""Attention of drafted token trees against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def random_masks(rng, T):
    """Each node sees itself and what its parent, an earlier node, sees."""
    out = []
    for j in range(T):
        out.append((out[rng.integers(max(0, j - 4), j)] if j else 0) | 1 << j)
    return out


class Case:
    """Inputs of one call; cache rows that no token was stored in hold NaN."""

    def __init__(self, lib, dtype, Hq, Hkv, d, dcp, bs, I, ctx, T, seed=0, scale=None,
                 max_vb=None):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.dims = rng, dtype, (Hq, Hkv, d, dcp, bs, I)
        self.ctx, self.T = list(ctx), list(T)
        self.layout = lib.Layout(dcp, bs, I)
        lens = [c + t for c, t in zip(ctx, T)]
        self.bt, self.nb = R.random_tables(rng, lens, dcp, bs, max_vb=max_vb)
        shape = (dcp, self.nb, Hkv, bs, d)
        self.k = np.full(shape, np.nan, dtype=np.float32)
        self.v = np.full(shape, np.nan, dtype=np.float32)
        for b, L in enumerate(lens):
            for x in range(L):
                r, vb, loc = R.place(x, dcp, bs, I)
                self.k[r, self.bt[r, b, vb], :, loc] = rng.standard_normal((Hkv, d))
                self.v[r, self.bt[r, b, vb], :, loc] = rng.standard_normal((Hkv, d))
        self.N = sum(T)
        self.start = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
        self.mask = [m for t in T for m in random_masks(rng, t)]
        self.q = rng.standard_normal((self.N, Hq, d)).astype(np.float32)
        self.scale = scale or d ** -0.5
        self.round()

    def round(self):
        for n in ("q", "k", "v"):
            a = torch.from_numpy(getattr(self, n)).to(self.dtype)
            setattr(self, n + "_t", a.cuda())
            setattr(self, n, a.float().numpy())

    def args(self, lib):
        m = np.array(self.mask, dtype=np.uint64).view(np.int64)
        kv = lib.PagedKV(list(self.k_t), list(self.v_t), torch.from_numpy(self.bt).cuda(), self.nb)
        return (self.layout, self.q_t, kv, torch.from_numpy(self.start).cuda(),
                torch.tensor(self.ctx, dtype=torch.int32).cuda(), torch.from_numpy(m).cuda(),
                self.scale, max(max(self.T), 1))

    def expected(self, b, rank=None, sink=None):
        """o, lse and their bounds' parts [T, Hq, ...] of request b (of one rank's tokens)."""
        Hq, Hkv, d, dcp, bs, I = self.dims
        n, T = self.ctx[b], self.T[b]
        pos = [x for x in range(n + T) if rank is None or R.place(x, dcp, bs, I)[0] == rank]
        k = R.gather(self.k, self.bt, b, pos, dcp, bs, I)
        v = R.gather(self.v, self.bt, b, pos, dcp, bs, I)
        s0 = self.start[b]
        seen = np.array([[x < n or (self.mask[s0 + t] >> (x - n)) & 1 == 1 for x in pos]
                         for t in range(T)], dtype=bool).reshape(T, len(pos))
        out = []
        for h in range(Hq):
            g = h // (Hq // Hkv)
            q = self.q[s0:s0 + T, h].astype(np.float64)
            out.append(R.attend(q, k[g], v[g], seen, self.scale,
                                None if sink is None else float(sink[h])))
        return [np.stack([o[i] for o in out], 1) for i in range(4)], len(pos)

    def check(self, out, lse, out_dtype, rank=None, sink=None, requests=None):
        d = self.dims[2]
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in requests if requests is not None else range(len(self.T)):
            if self.T[b] == 0:
                continue
            (o, el, wabs, size), L = self.expected(b, rank, sink)
            rows = slice(self.start[b], self.start[b + 1])
            tol = R.attend_tol(self.dtype, out_dtype, o.reshape(-1, d), wabs.reshape(-1, d),
                               size.reshape(-1), d, L).reshape(o.shape)
            bad = ~(np.abs(out[rows] - o) <= tol)
            assert not bad.any(), (b, rank, np.argwhere(bad)[:3], out[rows][bad][:3], o[bad][:3],
                                   tol[bad][:3])
            empty = np.isneginf(el)
            assert np.array_equal(np.isneginf(lse[rows]), empty), (b, rank)
            off = np.abs(lse[rows] - el)[~empty]
            assert (off <= R.lse_tol(el, size, d, L)[~empty]).all(), (b, rank, off.max())


# dtype, Hq, Hkv, d, dcp, bs, I, ctx, T
CASES = [
    (F32, 8, 2, 64, 2, 16, 1, [100, 37], [5, 11]),
    (F32, 4, 4, 32, 1, 16, 16, [0, 1, 33], [1, 1, 3]),
    (F32, 6, 2, 96, 3, 8, 4, [65, 0, 7], [2, 9, 0]),
    (F32, 16, 1, 256, 4, 16, 4, [130], [6]),
    (F32, 8, 1, 128, 2, 32, 8, [1500], [64]),
    (BF16, 32, 8, 128, 2, 16, 1, [300], [8]),
    (BF16, 32, 8, 128, 8, 16, 1, [1, 2100, 17, 0], [1, 16, 3, 7]),
    (BF16, 8, 2, 128, 4, 64, 64, [700, 0, 255, 256, 257], [64, 64, 63, 1, 33]),
    (BF16, 16, 1, 64, 3, 32, 4, [901, 12], [5, 64]),
    (BF16, 16, 2, 64, 8, 16, 16, [3000], [17]),
    (BF16, 8, 8, 128, 16, 16, 2, [513, 5], [2, 64]),
    (BF16, 3, 1, 96, 2, 48, 3, [100, 200], [4, 30]),
    (BF16, 4, 2, 128, 2, 8, 2, [70], [9]),
    (BF16, 4, 2, 256, 2, 16, 1, [90], [12]),
    (BF16, 16, 1, 128, 1, 128, 128, [0, 127, 128, 129], [64, 40, 1, 2]),
    (BF16, 12, 4, 64, 5, 16, 1, [40] * 20, [1 + i % 5 for i in range(20)]),
    (BF16, 32, 8, 128, 1, 256, 4, [4000, 1], [32, 32]),
]


def cid(c):
    return f"{str(c[0])[6:]}-{c[1]}.{c[2]}-d{c[3]}-dcp{c[4]}-bs{c[5]}-I{c[6]}-{sum(c[8])}of{max(c[7])}"


@pytest.mark.parametrize("case", CASES, ids=cid)
def test_fused_and_partials(lib, case):
    c = Case(lib, *case, seed=sum(case[7]) + case[3])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = c.args(lib)
    odt = torch.float32 if case[0] == F32 else torch.bfloat16
    out, lse = lib.tree_decode_gqa(*a, err=err)
    assert out.dtype == odt
    c.check(out, lse, odt)
    sink = torch.linspace(-2, 3, case[1]).cuda()
    out, lse = lib.tree_decode_gqa(*a, sink=sink, out_dtype=F32, err=err)
    c.check(out, lse, F32, sink=sink.cpu().numpy())
    po, pl = lib.tree_partial_gqa(*a, err=err)
    for r in range(case[4]):
        c.check(po[r], pl[r], F32, rank=r)
    # the ranks' parts joined are the fused call
    mo, ml = lib.lse_merge(po, pl, sink)
    c.check(mo, ml, F32, sink=sink.cpu().numpy())
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nodes_that_see_nothing(lib, dtype):
    c = Case(lib, dtype, 8, 2, 64, 2, 16, 1, [0, 40, 0], [4, 3, 64])
    c.mask[0] = c.mask[2] = 0                 # no context and no node
    c.mask[4] = 0                             # the context alone
    c.mask[10] = 1 << 63                      # the last of 64 nodes
    c.mask[1] |= 0xFF << 20                   # nodes that the request does not have
    out, lse = lib.tree_decode_gqa(*c.args(lib))
    c.mask[1] &= 0xF
    c.check(out, lse, dtype)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    sink = torch.linspace(-1, 1, 8).cuda()
    c.mask[1] |= 0xFF << 20
    out, lse = lib.tree_decode_gqa(*c.args(lib), sink=sink)
    assert (out[0] == 0).all()
    assert torch.allclose(lse[0], sink, rtol=0, atol=2.0 ** -20)


@pytest.mark.parametrize("dtype,G,dcp,T", [(F32, 2, 2, 9), (BF16, 2, 2, 9), (BF16, 4, 1, 64),
                                           (BF16, 4, 4, 40)])
def test_unseen_nodes_may_hold_anything(lib, dtype, G, dcp, T):
    """Infinities and NaN in a node's key and value reach only those that see it."""
    Hkv, d = 2, 128
    c = Case(lib, dtype, Hkv * G, Hkv, d, dcp, 16, 1, [50, 129], [T, 5])
    bad = T // 2
    for j in range(T):                        # nobody but `bad` itself sees it
        if j != bad:
            c.mask[j] &= ~(1 << bad)
    for x, kind in ((50 + bad, np.nan),):
        r, vb, loc = R.place(x, dcp, 16, 1)
        c.k[r, c.bt[r, 0, vb], :, loc, ::3] = kind
        c.v[r, c.bt[r, 0, vb], :, loc, ::5] = kind
        c.v[r, c.bt[r, 0, vb], 1, loc, 1::5] = -np.inf
    c.round()
    out, lse = lib.tree_decode_gqa(*c.args(lib), out_dtype=F32)
    rows = [j for j in range(T) if j != bad]
    # rows of request 0 but the bad one
    d0 = c.expected(0)
    (o, el, wabs, size), L = d0
    got = out[:T].double().cpu().numpy()
    tol = R.attend_tol(dtype, F32, o.reshape(-1, d), wabs.reshape(-1, d), size.reshape(-1), d,
                       L).reshape(o.shape)
    assert (np.abs(got - o) <= tol)[rows].all()
    assert np.isfinite(lse[:T].cpu().numpy()[rows]).all()
    assert torch.isnan(lse[bad]).all() and torch.isnan(out[bad]).all()
    c.check(out, lse, F32, requests=[1])
    # a finite key and infinite values: the node that sees it gets them in those columns alone
    c = Case(lib, dtype, Hkv * G, Hkv, d, dcp, 16, 1, [50, 129], [T, 5], seed=4)
    for j in range(T):
        if j != bad:
            c.mask[j] &= ~(1 << bad)
    r, vb, loc = R.place(50 + bad, dcp, 16, 1)
    c.v[r, c.bt[r, 0, vb], :, loc, 7] = np.inf
    c.v[r, c.bt[r, 0, vb], :, loc, 9] = np.nan
    c.round()
    out, lse = lib.tree_decode_gqa(*c.args(lib), out_dtype=F32)
    (o, el, wabs, size), L = c.expected(0)
    tol = R.attend_tol(dtype, F32, o.reshape(-1, d), wabs.reshape(-1, d), size.reshape(-1), d,
                       L).reshape(o.shape)
    got = out[:T].double().cpu().numpy()
    assert (got[bad][:, 7] == np.inf).all() and np.isnan(got[bad][:, 9]).all()
    ok = np.abs(got - o) <= tol
    ok[bad][:, [7, 9]] = True
    assert ok[rows].all() and ok[bad][:, [i for i in range(d) if i not in (7, 9)]].all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_node_is_the_decode_step(lib, dtype):
    c = Case(lib, dtype, 8, 2, 128, 4, 16, 1, [99, 0, 1000], [1, 1, 1])
    a = c.args(lib)
    out, lse = lib.tree_decode_gqa(*a, out_dtype=F32)
    c.check(out, lse, F32)
    seq = torch.tensor([100, 1, 1001], dtype=torch.int32).cuda()
    o2, l2 = lib.decode_gqa(c.layout, a[1], a[2], lib.local_seq_lens(c.layout, seq), c.scale,
                            out_dtype=F32)
    c.check(o2, l2, F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores_and_scale(lib, dtype):
    """Scores of hundreds: one token takes all the weight, maxima grow along the row."""
    c = Case(lib, dtype, 8, 2, 128, 2, 16, 1, [600], [20], scale=3.0)
    out, lse = lib.tree_decode_gqa(*c.args(lib))
    c.check(out, lse, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_refused_requests_and_rows_behind_the_last(lib, dtype):
    c = Case(lib, dtype, 8, 2, 128, 2, 16, 1, [30, 40, 50, 60], [3, 4, 5, 6])
    layout, q, kv, start, ctx, mask, scale, _ = c.args(lib)
    N = c.N
    q2 = torch.cat([q, torch.full_like(q[:5], float("nan"))])
    mask2 = torch.cat([mask, torch.zeros_like(mask[:5])])
    for b, change in ((1, "ctx"), (2, "long"), (3, "table"), (0, "rows")):
        ctx2, start2, most = ctx.clone(), start.clone(), 6
        if change == "ctx":
            ctx2[b] = -1
        if change == "long":
            most = 5                          # request 3 has 6 nodes
            b = 3
        if change == "table":
            ctx2[b] = kv.max_vb * 32 - 5      # the sixth node lies behind the table
        if change == "rows":
            start2[0] = -1
        out = torch.full((N + 5, 8, 128), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((N + 5, 8), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.tree_decode_gqa(layout, q2, kv, start2, ctx2, mask2, scale, most, out=out,
                            out_lse=lse, err=err)
        assert err.item() == 1, change
        rows = slice(c.start[b], c.start[b + 1])
        assert (out[rows] == 7).all() and (lse[rows] == 7).all(), change
        assert (out[N:] == 7).all() and (lse[N:] == 7).all(), change
        c.check(out[:N], lse[:N], dtype, requests=[x for x in range(4) if x != b])


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 128), (BF16, 64)])
def test_bad_pages_are_skipped_and_counted(lib, dtype, d):
    c = Case(lib, dtype, 8, 2, d, 2, 16, 1, [300, 90], [6, 6])
    layout, q, kv, start, ctx, mask, scale, most = c.args(lib)
    bt = kv.block_table.clone()
    bt[1, 0, 2] = c.nb + 5
    bt[0, 1, 0] = -3
    bt[0, 0, 9] = 2 ** 31 - 1                  # the page of the nodes
    kv2 = lib.PagedKV(kv.k_pools, kv.v_pools, bt, c.nb)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.tree_decode_gqa(layout, q, kv2, start, ctx, mask, scale, most, err=err)
    torch.cuda.synchronize()
    assert err.item() >= 3
    Hq, Hkv, _, dcp, bs, I = c.dims
    gone = {(1, 0, 2), (0, 1, 0), (0, 0, 9)}
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(2):
        n, T = c.ctx[b], c.T[b]
        pos = [x for x in range(n + T)
               if (R.place(x, dcp, bs, I)[0], b, R.place(x, dcp, bs, I)[1]) not in gone]
        k, v = (R.gather(p, c.bt, b, pos, dcp, bs, I) for p in (c.k, c.v))
        s0 = c.start[b]
        seen = np.array([[x < n or (c.mask[s0 + t] >> (x - n)) & 1 == 1 for x in pos]
                         for t in range(T)], dtype=bool)
        for h in range(Hq):
            o, el, wabs, size = R.attend(c.q[s0:s0 + T, h].astype(np.float64), k[h // 4], v[h // 4],
                                         seen, scale)
            tol = R.attend_tol(dtype, dtype, o, wabs, size, d, len(pos))
            assert (np.abs(got[s0:s0 + T, h] - o) <= tol).all()
            assert (np.abs(gl[s0:s0 + T, h] - el) <= R.lse_tol(el, size, d, len(pos))).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed_with_other_lengths(lib, dtype):
    c = Case(lib, dtype, 8, 2, 128, 2, 16, 1, [500, 300, 20], [9, 1, 12])
    layout, q, kv, start, ctx, mask, scale, _ = c.args(lib)
    need = lib.tree_workspace_size(layout, 3, 16, 8, 2, 128, dtype)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((c.N, 8), device="cuda")
    call = lambda w: lib.tree_decode_gqa(layout, q, kv, start, ctx, mask, scale, 16, out=out,  # noqa: E731
                                         out_lse=lse, workspace=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ws)
    for lens in ([500, 300, 20], [0, 1, 2], [499, 7, 0]):
        c.ctx = lens
        # the nodes' cache rows move with the length: expectations read the same pools
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        c.check(*got, dtype)
        call(ws2)
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


def test_two_calls_at_once_on_two_streams(lib):
    cs = [Case(lib, BF16, 8, 2, 128, 2, 16, 1, [700, 30], [9, 20], seed=s) for s in (1, 2)]
    args = [c.args(lib) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lib.tree_decode_gqa(*args[i]))
    torch.cuda.synchronize()
    for c, rows in zip(cs, got):
        c.check(*rows[0], BF16)
        for o, l in rows[1:]:
            assert torch.equal(o, rows[0][0]) and torch.equal(l, rows[0][1])


def test_nothing_to_do(lib):
    c = Case(lib, BF16, 8, 2, 128, 2, 16, 1, [3], [1])
    layout, q, kv, start, ctx, mask, scale, _ = c.args(lib)
    out, lse = lib.tree_decode_gqa(layout, q[:0], kv, start[:1] * 0, ctx[:0], mask[:0], scale, 1)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


def test_refusals(lib):
    c = Case(lib, BF16, 8, 2, 128, 2, 16, 1, [30], [3])
    layout, q, kv, start, ctx, mask, scale, most = c.args(lib)

    def call(layout=layout, q=q, kv=kv, start=start, ctx=ctx, mask=mask, scale=scale, most=most,
             **kw):
        with pytest.raises(lib.DcpError):
            lib.tree_decode_gqa(layout, q, kv, start, ctx, mask, scale, most, **kw)

    call(q=q.half())
    call(q=q.float())
    call(q=q.transpose(0, 1))
    call(q=q[:, :7])
    call(q=q.cpu())
    call(q=q[..., :96].contiguous())
    call(start=start.long())
    call(start=start[:1])
    call(ctx=ctx.long())
    call(mask=mask.int())
    call(mask=mask[:2])
    call(most=0)
    call(most=65)
    call(scale=0.0)
    call(scale=-1.0)
    call(scale=float("nan"))
    call(layout=lib.Layout(3, 16, 1))
    call(layout=lib.Layout(2, 32, 1))
    call(sink=torch.zeros(7, device="cuda"))
    call(sink=torch.zeros(8, device="cuda", dtype=torch.float64))
    call(out=torch.empty((2, 8, 128), dtype=BF16, device="cuda"))
    call(out_dtype=torch.float16)
    call(out_lse=torch.empty((3, 8), dtype=BF16, device="cuda"))
    call(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
    call(err=torch.zeros(1, device="cuda"))
