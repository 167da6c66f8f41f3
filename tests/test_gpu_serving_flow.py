"""A run of the calls around the decode step together, as a serving loop makes
them: admit, write prompts, draft, attend, accept, trim, fork, decode on, free.
What each request has stored is kept on the host, and every attention result is
compared with plain 64-bit attention over it."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.asarray(x, dtype=dtype)).cuda()


class Loop:
    """Two layers of keys and values, their pages, and the tokens of each request."""

    def __init__(self, lib, dtype, Hq, Hkv, d, dcp, bs, I, reqs, VB, nb, shared, seed):
        self.lib, self.dtype, self.Hq, self.Hkv, self.d = lib, dtype, Hq, Hkv, d
        self.geo = dcp, bs, I
        self.L = lib.Layout(dcp, bs, I)
        self.nb = nb
        self.pages = lib.Pages.new(self.L, reqs, VB, nb, shared=shared)
        shape = (nb, Hkv, bs, d)
        mk = lambda: [torch.full(shape, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
                      for _ in range(dcp)]
        self.k, self.v = [mk() for _ in range(2)], [mk() for _ in range(2)]
        self.set = lib.PoolSet([*self.k, *self.v])
        self.table = self.pages.block_table[0] if shared else self.pages.block_table
        self.kv = [lib.PagedKV(k, v, self.table, nb) for k, v in zip(self.k, self.v)]
        self.inv = dev(10000.0 ** (-np.arange(d // 2) / (d // 2)), np.float32)
        self.stored = {}                   # request -> [layer][k or v] list of rows [Hkv, d]
        self.gen = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.err = torch.zeros(1, dtype=I32, device="cuda")

    def resize(self, reqs, lens):
        src, dst = self.lib.pages_resize(self.L, self.pages, dev(reqs), dev(lens), err=self.err)
        self.lib.pages_copy(self.L, self.set, src, dst, err=self.err)

    def write(self, req, at, positions):
        """Tokens at cache places `at` with rotary `positions`; returns the rotated queries."""
        T = len(req)
        _, slot = self.lib.slot_mapping(self.L, dev(req), dev(at, np.int64), self.table, self.nb,
                                        err=self.err)
        out = []
        for layer in range(2):
            x = torch.randn((T, self.Hq + 2 * self.Hkv, self.d), generator=self.gen)
            q, k, v = x.to(self.dtype).cuda().split([self.Hq, self.Hkv, self.Hkv], 1)
            k_out = torch.empty((T, self.Hkv, self.d), dtype=self.dtype, device="cuda")
            out.append(self.lib.rope_write_gqa(self.L, q, k, v, dev(positions, np.int64), self.inv,
                                               slot, self.k[layer], self.v[layer], self.nb,
                                               k_out=k_out, err=self.err))
            kr, vr = k_out.float().cpu().numpy(), v.float().cpu().numpy()
            for t, (b, a) in enumerate(zip(req, at)):
                rows = self.stored.setdefault(b, [[{}, {}], [{}, {}]])[layer]
                rows[0][a], rows[1][a] = kr[t], vr[t]
        return out

    def expect(self, layer, req, q, seen, out, lse):
        """out [T, Hq, d] of queries q [T, Hq, d] that see `seen` [T, tokens] of a request."""
        rows = self.stored[req][layer]
        n = seen.shape[1]
        k, v = (np.stack([rows[i][x] for x in range(n)], 1).astype(np.float64) for i in (0, 1))
        q = q.double().cpu().numpy()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for h in range(self.Hq):
            g = h // (self.Hq // self.Hkv)
            o, el, wabs, size = R.attend(q[:, h], k[g], v[g], seen, self.d ** -0.5)
            tol = R.attend_tol(self.dtype, self.dtype, o, wabs, size, self.d, n)
            assert (np.abs(out[:, h] - o) <= tol).all(), (layer, req, h)
            assert (np.abs(lse[:, h] - el) <= R.lse_tol(el, size, self.d, n)).all()


@pytest.mark.parametrize("dtype,Hq,Hkv,d,dcp,bs,I,shared", [
    (BF16, 8, 2, 128, 2, 16, 1, False),
    (BF16, 8, 2, 64, 3, 32, 8, True),
    (F32, 4, 2, 64, 4, 16, 16, False),
])
def test_a_serving_loop(lib, dtype, Hq, Hkv, d, dcp, bs, I, shared):
    s = Loop(lib, dtype, Hq, Hkv, d, dcp, bs, I, 8, 12, 200, shared, seed=d + dcp)
    lens = {0: 37, 1: 1, 2: bs * dcp * 2 + 3}
    s.resize(list(lens), list(lens.values()))
    req = [b for b, n in lens.items() for _ in range(n)]
    at = [x for n in lens.values() for x in range(n)]
    s.write(req, at, at)

    for step in range(3):
        # draft: a random tree for each request, stored behind its tokens
        T = {b: int(s.rng.integers(1, 9)) for b in lens}
        parent = {b: [-1] + [int(s.rng.integers(max(0, j - 3), j)) for j in range(1, T[b])]
                  for b in lens}
        s.resize(list(lens), [lens[b] + T[b] for b in lens])
        req, at, pos, mask = [], [], [], []
        for b in lens:
            bits, depth = [], []
            for j, p in enumerate(parent[b]):
                bits.append((bits[p] if p >= 0 else 0) | 1 << j)
                depth.append(depth[p] + 1 if p >= 0 else 0)
            req += [b] * T[b]
            at += [lens[b] + j for j in range(T[b])]
            pos += [lens[b] + x for x in depth]
            mask += bits
        qs = s.write(req, at, pos)
        # the calls take rows of the block table in order: all requests, some without nodes
        count = [T.get(b, 0) for b in range(8)]
        start = np.concatenate([[0], np.cumsum(count)])
        ctx = [lens.get(b, 0) for b in range(8)]
        for layer in range(2):
            out, lse = lib.tree_decode_gqa(s.L, qs[layer], s.kv[layer], dev(start), dev(ctx),
                                           dev(mask, np.int64), d ** -0.5, 8, err=s.err)
            for b in lens:
                rows = slice(int(start[b]), int(start[b + 1]))
                seen = np.array([[x < lens[b] or (m >> (x - lens[b])) & 1 == 1
                                  for x in range(lens[b] + T[b])] for m in mask[rows]], dtype=bool)
                s.expect(layer, b, qs[layer][rows], seen, out[rows], lse[rows])
        # accept a path from the root, and drop the rest
        path = np.full((8, 8), -1, dtype=np.int32)
        kept = [0] * 8
        for b in lens:
            node, got = 0, [0]
            while True:
                nxt = [j for j in range(T[b]) if parent[b][j] == node]
                if not nxt or s.rng.random() < 0.2:
                    break
                node = nxt[int(s.rng.integers(len(nxt)))]
                got.append(node)
            path[b, :len(got)], kept[b] = got, len(got)
            for layer in s.stored[b]:
                for rows in layer:
                    new = {i: rows[lens[b] + j] for i, j in enumerate(got)}
                    for i, r in new.items():
                        rows[lens[b] + i] = r
        new = lib.cache_compact(s.L, s.set, s.table, s.nb, dev(ctx), dev(path), dev(kept),
                                err=s.err)
        for b in lens:
            lens[b] += kept[b]
        assert new.tolist() == [lens.get(b, 0) for b in range(8)]
        s.resize(list(lens), list(lens.values()))

    # two samples of request 2 and one of request 0, then every request goes on by itself
    src, dst = lib.pages_fork(s.L, s.pages, dev([2, 2, 0]), dev([5, 6, 7]), err=s.err)
    lib.pages_copy(s.L, s.set, src, dst, err=s.err)
    import copy
    for child, p in ((5, 2), (6, 2), (7, 0)):
        lens[child] = lens[p]
        s.stored[child] = copy.deepcopy(s.stored[p])
    for _ in range(2):
        order = sorted(lens)
        s.resize(order, [lens[b] + 1 for b in order])
        qs = s.write(order, [lens[b] for b in order], [lens[b] for b in order])
        for b in order:
            lens[b] += 1
        full = torch.zeros((8, Hq, d), dtype=dtype, device="cuda")
        seq = dev([lens.get(b, 0) for b in range(8)])
        for layer in range(2):
            full[order] = qs[layer]
            out, lse = lib.decode_gqa(s.L, full, s.kv[layer], lib.local_seq_lens(s.L, seq),
                                      d ** -0.5, err=s.err)
            one, l1 = lib.tree_decode_gqa(
                s.L, full, s.kv[layer], dev(np.arange(9)), seq - 1 * (seq > 0).int(),
                torch.ones(8, dtype=torch.int64, device="cuda"), d ** -0.5, 1, err=s.err)
            for i, b in enumerate(order):
                seen = np.ones((1, lens[b]), dtype=bool)
                s.expect(layer, b, qs[layer][i:i + 1], seen, out[b:b + 1], lse[b:b + 1])
                s.expect(layer, b, qs[layer][i:i + 1], seen, one[b:b + 1], l1[b:b + 1])
    # a request that has no pages (rows 3 and 4) looked for its own node's page above
    missing = s.err.item()
    s.resize(list(range(8)), [0] * 8)
    assert s.err.item() == missing
    assert (s.pages.ref_count == 0).all() and (s.pages.seq_lens == 0).all()
    assert (s.pages.block_table == -1).all()


def test_a_step_in_a_graph(lib):
    """Rotary write, attention and compaction of a step, captured and replayed on new inputs."""
    Hq, Hkv, d, dcp, bs, B, T, ctx0 = 8, 2, 128, 2, 16, 3, 4, 40
    L = lib.Layout(dcp, bs, 1)
    rng = np.random.default_rng(3)
    bt, nb = R.random_tables(rng, [200] * B, dcp, bs)
    base = torch.randn((2, dcp, nb, Hkv, bs, d), generator=torch.Generator().manual_seed(1)).to(BF16)
    pools = base.cuda()
    table = dev(bt)
    kv = lib.PagedKV(list(pools[0]), list(pools[1]), table, nb)
    pset = lib.PoolSet([list(pools[0]), list(pools[1])])
    x = torch.empty((B * T, Hq + 2 * Hkv, d), dtype=BF16, device="cuda")
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    inv = dev(10000.0 ** (-np.arange(64) / 64), np.float32)
    ctx = torch.empty(B, dtype=I32, device="cuda")
    req = dev(np.repeat(np.arange(B), T))
    node = dev(np.tile(np.arange(T), B), np.int64)
    start, path, n = dev(np.arange(B + 1) * T), dev([[0, 2], [1, 3], [3, 0]]), dev([2, 2, 1])
    mask = dev(np.tile([1, 3, 5, 13], B), np.int64)

    def step():
        at = ctx.long().repeat_interleave(T) + node
        _, slot = lib.slot_mapping(L, req, at, table, nb)
        qr = lib.rope_write_gqa(L, q, k, v, at, inv, slot, list(pools[0]), list(pools[1]), nb)
        out, lse = lib.tree_decode_gqa(L, qr, kv, start, ctx, mask, d ** -0.5, T)
        return out, lse, lib.cache_compact(L, pset, table, nb, ctx, path, n)

    ctx.fill_(ctx0)
    x.copy_(torch.randn(x.shape))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for lens in ([40, 0, 7], [150, 33, 64], [1, 2, 3]):
        ctx.copy_(torch.tensor(lens, dtype=I32))
        x.copy_(torch.randn(x.shape))
        pools.copy_(base)
        g.replay()
        after = pools.clone(), [t.clone() for t in got]
        pools.copy_(base)
        want = step()
        for a, b in zip(after[1], want):
            assert torch.equal(a, b)
        assert torch.equal(after[0], pools)


def test_what_a_call_allocates_belongs_to_its_stream(lib):
    """Memory that another stream's queued work still writes is not handed out."""
    L = lib.Layout(2, 16, 1)
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=gen).to(BF16).cuda()
               for s in ((64, 8, 128), (2, 6, 2, 16, 128), (2, 6, 2, 16, 128)))
    bt = dev([[[0, 1, 2]], [[3, 4, 5]]])
    kv = lib.PagedKV(list(k), list(v), bt, 6)
    mask = torch.full((64,), -1, dtype=torch.int64, device="cuda")
    args = L, q, kv, dev([0, 64]), dev([20]), mask, 0.1, 64
    want, lse = lib.tree_decode_gqa(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(want) for _ in range(4)] + \
        [torch.empty(n, dtype=torch.uint8, device="cuda")
         for n in (lib.tree_workspace_size(L, 1, 64, 8, 2, 128, BF16), lse.nbytes)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)         # some 50 ms, then the memory is written
    for x in freed:
        x.zero_()
    del freed, x
    got, got_lse = lib.tree_decode_gqa(*args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_lse, lse)


def test_streams_named_one_by_one(lib):
    """The default and the current stream given by name are the call without one."""
    L = lib.Layout(2, 16, 1)
    pages = [lib.Pages.new(L, 4, 4, 20, stream=s) for s in (None, torch.cuda.default_stream())]
    for p, s in zip(pages, (torch.cuda.current_stream(), None)):
        lib.pages_resize(L, p, dev([0, 3]), dev([70, 9]), stream=s)
        src, dst = lib.pages_fork(L, p, dev([0]), dev([2]), stream=torch.cuda.default_stream())
        assert (src >= 0).all() and (dst >= 0).all()
    for a in ("block_table", "seq_lens", "ref_count", "free_bits"):
        assert torch.equal(getattr(pages[0], a), getattr(pages[1], a))


def test_the_state_of_new_pages_belongs_to_its_stream(lib):
    """As above, for the tensors that Pages.new makes on a stream of the caller's."""
    L = lib.Layout(2, 16, 1)
    B, VB, nb = 512, 256, 1 << 18
    side = torch.cuda.Stream()
    want = lib.Pages.new(L, B, VB, nb)
    names = ("block_table", "seq_lens", "ref_count", "free_bits")
    want = [getattr(want, a).clone() for a in names]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty_like(x) for x in want for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)         # some 50 ms, then the memory is written
    for x in freed:
        x.fill_(77)
    del freed, x
    p = lib.Pages.new(L, B, VB, nb, stream=side)
    torch.cuda.synchronize()
    for a, w in zip(names, want):
        assert torch.equal(getattr(p, a), w), a


@pytest.mark.parametrize("dcp", [1, 3])
def test_a_shared_table_as_the_state_has_it(lib, dcp):
    """[1, B, max_vb] is one table for all ranks in every call that takes a table."""
    L, nb, Hkv, d, B = lib.Layout(dcp, 16, 1), 30, 2, 64, 3
    pages = lib.Pages.new(L, B, 4, nb, shared=True)
    lens = [40, 1, 33]
    lib.pages_resize(L, pages, dev(range(B)), dev(lens))
    gen = torch.Generator().manual_seed(dcp)
    k, v = (torch.randn((dcp, nb, Hkv, 16, d), generator=gen).to(BF16).cuda() for _ in range(2))
    q = torch.randn((B, 8, d), generator=gen).to(BF16).cuda()
    whole, flat = pages.block_table, pages.block_table[0]
    assert whole.shape == (1, B, 4)
    kvs = [lib.PagedKV(list(k), list(v), t, nb) for t in (whole, flat)]
    req, pos = dev([0, 1, 2, 2]), dev([39, 0, 20, 32], np.int64)
    topk, seq = dev([[0, 17, 39], [0, 0, 0], [5, 32, 31]]), dev(lens)
    calls = (lambda t, kv: lib.slot_mapping(L, req, pos, t, nb),
             lambda t, kv: lib.sfa_remap(L, topk, seq, t, nb),
             lambda t, kv: lib.decode_gqa(L, q, kv, lib.local_seq_lens(L, seq), d ** -0.5),
             lambda t, kv: lib.tree_decode_gqa(L, q, kv, dev([0, 1, 2, 3]), seq - 1,
                                               torch.ones(3, dtype=torch.int64, device="cuda"),
                                               d ** -0.5, 1),
             lambda t, kv: lib.tree_partial_gqa(L, q, kv, dev([0, 1, 2, 3]), seq - 1,
                                                torch.ones(3, dtype=torch.int64, device="cuda"),
                                                d ** -0.5, 1))
    for call in calls:
        for a, b in zip(call(whole, kvs[0]), call(flat, kvs[1])):
            assert torch.equal(a, b)
    # two tables are not enough for three ranks
    two, L3 = torch.cat([whole, whole]), lib.Layout(3, 16, 1)
    kv2 = lib.PagedKV(list(k[:1]), list(v[:1]), two, nb)
    for bad in (lambda: lib.slot_mapping(L3, req, pos, two, nb),
                lambda: lib.sfa_remap(L3, topk, seq, two, nb),
                lambda: lib.decode_gqa(L3, q, lib.PagedKV([k[0]] * 3, [v[0]] * 3, two, nb),
                                       lib.local_seq_lens(L3, seq), d ** -0.5),
                lambda: lib.tree_decode_gqa(L3, q, kv2, dev([0, 1, 2, 3]), seq - 1,
                                            torch.ones(3, dtype=torch.int64, device="cuda"),
                                            d ** -0.5, 1)):
        with pytest.raises(lib.DcpError):
            bad()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pages_beyond_thirty_two_bits(lib, dtype):
    """A step on the last pages of pools of more than 2^31 elements gives what it gives on the
    first pages of small ones."""
    Hq, Hkv, d, bs, B, T = 8, 2, 128, 16, 3, 5
    far = 2 ** 31 // (Hkv * bs * d)              # pages
    L = lib.Layout(1, bs, 1)
    inv = dev(10000.0 ** (-np.arange(64) / 64), np.float32)
    ctx, mask = dev([40, 0, 100]), dev([1, 3, 5, 13, 17] * B, np.int64)
    got = []
    for first, nb in ((0, 40), (far - 3, far + 40)):      # the border lies among them
        gen = torch.Generator().manual_seed(1)
        k, v = (torch.empty((nb, Hkv, bs, d), dtype=dtype, device="cuda") for _ in range(2))
        for p in (k, v):
            p[first:first + 40] = torch.randn((40, Hkv, bs, d), generator=gen).to(dtype).cuda()
        bt = (np.random.default_rng(2).permutation(24) + first).astype(np.int32).reshape(1, B, 8)
        table, pset = dev(bt), lib.PoolSet([[k], [v]])
        x = torch.randn((B * T, Hq + 2 * Hkv, d), generator=gen).to(dtype).cuda()
        q, kn, vn = x.split([Hq, Hkv, Hkv], 1)
        at = ctx.long().repeat_interleave(T) + torch.arange(T, device="cuda").repeat(B)
        err = torch.zeros(1, dtype=I32, device="cuda")
        _, slot = lib.slot_mapping(L, dev(np.repeat(np.arange(B), T)), at, table, nb, err=err)
        qr = lib.rope_write_gqa(L, q, kn, vn, at, inv, slot, [k], [v], nb, err=err)
        kv = lib.PagedKV([k], [v], table, nb)
        out, lse = lib.tree_decode_gqa(L, qr, kv, dev(np.arange(B + 1) * T), ctx, mask, 0.1, T,
                                       err=err)
        new = lib.cache_compact(L, pset, table, nb, ctx, dev([[0, 2, 3], [1, 4, 0], [3, 0, 0]]),
                                dev([3, 2, 1]), err=err)
        lib.pages_copy(L, pset, dev([[first, first + 39]]), dev([[first + 30, first + 31]]), err=err)
        assert err.item() == 0
        got.append((qr, out, lse, new, k[first:first + 40].clone(), v[first:first + 40].clone()))
        del k, v, kv, pset
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_pages_in_a_graph(lib):
    """Free, fork, copy and grow, captured and replayed on other lists, against the model."""
    dcp, bs, I, B, VB, nb = 3, 16, 4, 12, 6, 60
    L = lib.Layout(dcp, bs, I)
    pages, m = lib.Pages.new(L, B, VB, nb), R.PageModel(dcp, bs, I, B, VB, nb, False)
    pool = torch.randn((dcp, nb, 2, bs, 32), generator=torch.Generator().manual_seed(0)).cuda()
    start, pset = pool.clone(), lib.PoolSet([list(pool)])
    rng = np.random.default_rng(4)
    lens = rng.integers(1, VB * bs * dcp // 2, 4)
    lib.pages_resize(L, pages, dev(range(4)), dev(lens))
    m.resize(np.arange(4), lens)
    state = [getattr(pages, a) for a in ("block_table", "seq_lens", "ref_count", "free_bits")]
    before = [x.clone() for x in state]
    zero, child, parent = torch.zeros(6, dtype=I32, device="cuda"), dev([0] * 6), dev([0] * 6)
    grown = dev([0] * 6)

    def step():
        lib.pages_resize(L, pages, child, zero)
        src, dst = lib.pages_fork(L, pages, parent, child)
        lib.pages_copy(L, pset, src, dst)
        s2, d2 = lib.pages_resize(L, pages, child, grown)
        lib.pages_copy(L, pset, s2, d2)
        return src, dst, s2, d2

    def lists():
        c, p = 4 + rng.permutation(8)[:6], rng.integers(0, 4, 6)
        g = np.minimum(m.seq[p] + rng.integers(-20, 9, 6), VB * bs * dcp).clip(0)
        for to, x in ((child, c), (parent, p), (grown, g)):
            to.copy_(dev(x))
        return c, p, g

    lists()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for x, y in zip(state, before):          # as it was before the warm-up
        x.copy_(y)
    pool.copy_(start)
    want = start.cpu().clone()
    for _ in range(6):
        c, p, grow = lists()
        m.resize(c, np.zeros(6, dtype=int))
        es = list(m.fork(p, c))
        es += m.resize(c, grow)
        g.replay()
        assert m.err == 0
        for x, y in zip(got, es):
            assert np.array_equal(x.cpu().numpy(), y)
        for a, b in ((es[0], es[1]), (es[2], es[3])):
            for r in range(dcp):
                for x, y in zip(a[r], b[r]):
                    if x >= 0:
                        want[r, y] = want[r, x].clone()
        assert torch.equal(pool.cpu(), want)
        for x, y in zip(state, (m.bt, m.seq, m.ref, m.bits())):
            assert np.array_equal(x.cpu().numpy(), y)
