"""The pages' life against a page-by-page model, copies and compaction byte for byte."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

I32 = torch.int32


def dev(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def same(pages, m):
    assert np.array_equal(pages.seq_lens.cpu().numpy(), m.seq)
    assert np.array_equal(pages.ref_count.cpu().numpy(), m.ref)
    assert np.array_equal(pages.block_table.cpu().numpy(), m.bt)
    assert np.array_equal(pages.free_bits.cpu().numpy(), m.bits())


# dcp, bs, I, requests, max_vb, pages, shared
SHAPES = [
    (2, 16, 1, 9, 6, 60, False),
    (8, 16, 4, 12, 4, 37, False),
    (3, 8, 8, 40, 9, 400, False),
    (1, 16, 16, 5, 8, 33, False),
    (4, 16, 1, 7, 5, 64, True),
    (16, 16, 16, 6, 3, 31, False),
    (2, 16, 2, 300, 3, 1000, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_random_lives(lib, shape):
    dcp, bs, I, B, VB, nb, shared = shape
    L = lib.Layout(dcp, bs, I)
    pages = lib.Pages.new(L, B, VB, nb, shared=shared)
    m = R.PageModel(dcp, bs, I, B, VB, nb, shared)
    same(pages, m)
    rng = np.random.default_rng(nb)
    err = torch.zeros(1, dtype=I32, device="cuda")
    most = VB * bs * dcp
    for step in range(25):
        # what fits: the model's own count decides how far the requests grow
        n = int(rng.integers(1, B + 1))
        if step % 3 != 2:
            req = rng.permutation(B)[:n]
            new = np.where(rng.random(n) < 0.3, 0, rng.integers(0, most + 1, n))
            room = (m.ref == 0).sum(1).min() // 2
            keep, used = [], 0
            for i, (r, x) in enumerate(zip(req, new)):
                used += max(0, m.blocks(x) - m.blocks(m.seq[r])) + 1
                if used <= room or x <= m.seq[r]:
                    keep.append(i)
                else:
                    used -= max(0, m.blocks(x) - m.blocks(m.seq[r])) + 1
            req, new = req[keep], new[keep]
            if not len(req):
                continue
            src, dst = lib.pages_resize(L, pages, dev(req), dev(new), err=err)
            es, ed = m.resize(req, new)
        else:
            order = rng.permutation(B)
            k = max(1, min(n, B // 2, int((m.ref == 0).sum(1).min())))
            child, parent = order[:k], rng.choice(order[k:], k)
            src, dst = lib.pages_fork(L, pages, dev(parent), dev(child), err=err)
            es, ed = m.fork(parent, child)
        same(pages, m)
        assert np.array_equal(src.cpu().numpy(), es) and np.array_equal(dst.cpu().numpy(), ed)
    assert err.item() == 0 and m.err == 0
    # everything goes: no page is lost
    lib.pages_resize(L, pages, dev(np.arange(B)), dev(np.zeros(B)), err=err)
    assert (pages.ref_count == 0).all() and (pages.block_table == -1).all() and err.item() == 0


def test_entries_that_cannot_be(lib):
    """Rows out of range, named twice, too long; parents that are children; no page left."""
    L = lib.Layout(2, 16, 1)
    pages, m = lib.Pages.new(L, 8, 4, 12), R.PageModel(2, 16, 1, 8, 4, 12, False)
    err = torch.zeros(1, dtype=I32, device="cuda")
    for req, new in (([0, 0, 9, -1, 1, 2, 3], [40, 90, 5, 5, -2, 129, 33]),
                     ([4, 4, 5], [128, 0, 100])):
        s, d = lib.pages_resize(L, pages, dev(req), dev(new), err=err)
        es, ed = m.resize(req, new)
        same(pages, m)
        assert np.array_equal(s.cpu().numpy(), es) and np.array_equal(d.cpu().numpy(), ed)
    for parent, child in (([0, 3, 0, 5, 8, 0], [6, 0, 6, 7, 2, -1]), ([4, 4], [4, 1])):
        s, d = lib.pages_fork(L, pages, dev(parent), dev(child), err=err)
        es, ed = m.fork(parent, child)
        same(pages, m)
        assert np.array_equal(s.cpu().numpy(), es) and np.array_equal(d.cpu().numpy(), ed)
    assert err.item() == m.err > 0
    before = m.err
    # twelve pages a table: the third request does not fit
    pages, m = lib.Pages.new(L, 8, 8, 12), R.PageModel(2, 16, 1, 8, 8, 12, False)
    req, new = [1, 2, 3, 0], [160, 150, 200, 10]
    lib.pages_resize(L, pages, dev(req), dev(new), err=err)
    m.resize(req, new)
    same(pages, m)
    assert err.item() == before + m.err and m.err > 0


def test_a_cut_page_that_others_hold_is_replaced(lib):
    L = lib.Layout(2, 16, 1)
    pages, m = lib.Pages.new(L, 6, 4, 40), R.PageModel(2, 16, 1, 6, 4, 40, False)

    def both(name, a, b):
        s, d = getattr(lib, "pages_" + name)(L, pages, dev(a), dev(b))
        es, ed = getattr(m, name)(a, b)
        same(pages, m)
        assert np.array_equal(s.cpu().numpy(), es) and np.array_equal(d.cpu().numpy(), ed)
        return es, ed

    both("resize", [0], [100])
    both("fork", [0, 0], [1, 2])
    s, d = both("resize", [1, 2, 0], [70, 70, 35])     # cut inside pages that all three hold
    assert (s[:, :2] >= 0).all() and (d >= 0).all()
    s, d = both("resize", [1], [71])                   # its own page: no copy
    assert (s == -1).all()
    both("resize", [0, 1, 2], [0, 0, 0])
    assert (m.ref == 0).all()


@pytest.mark.parametrize("tables", [1, 3])
@pytest.mark.parametrize("latent", [False, True])
def test_copies(lib, tables, latent):
    dcp, nb, bs, H, d = 3, 20, 16, 3, 64
    L = lib.Layout(dcp, bs, 1)
    shape = (nb, bs, d) if latent else (nb, H, bs, d)
    pools = [[torch.randn(shape, device="cuda").to(torch.bfloat16) for _ in range(dcp)]
             for _ in range(5)]
    want = [[p.clone() for p in ps] for ps in pools]
    src = np.array([[0, -1, 7, 3, 5]] * tables) + np.arange(tables)[:, None] * 2
    dst = np.array([[10, -1, 12, 15, 5]] * tables) + np.arange(tables)[:, None]
    src[:, 1] = dst[:, 1] = -1
    for ps in want:
        for r, p in enumerate(ps):
            t = 0 if tables == 1 else r
            old = p.clone()
            for a, b in zip(src[t], dst[t]):
                if a >= 0:
                    p[b] = old[a]
    err = torch.zeros(1, dtype=I32, device="cuda")
    lib.pages_copy(L, lib.PoolSet(pools), dev(src), dev(dst), err=err)
    for a, b in zip(pools, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert err.item() == 0
    src[0, 0], dst[-1, 2] = nb, -1
    lib.pages_copy(L, lib.PoolSet(pools), dev(src), dev(dst), err=err)
    assert err.item() > 0


# dcp, bs, I, H, d, dtype, ctx, paths
COMPACT = [
    (2, 16, 1, 2, 64, torch.bfloat16, [30, 0, 100], [[0, 2, 3, 7], [1], []]),
    (8, 16, 4, 8, 128, torch.bfloat16, [127, 1], [list(range(1, 40)), [0, 1, 2]]),
    (3, 32, 32, 1, 576, torch.bfloat16, [95, 96, 97], [[3, 4, 63], [0, 63], list(range(0, 64, 2))]),
    (1, 16, 16, 4, 96, torch.float32, [5], [list(range(3, 300))]),
    (4, 8, 2, 1, 32, torch.float32, [0, 9], [list(range(0, 400, 3)), [0, 5, 6, 7, 8, 9, 10, 11, 30]]),
]


@pytest.mark.parametrize("case", COMPACT, ids=lambda c: f"dcp{c[0]}-bs{c[1]}-I{c[2]}-H{c[3]}-d{c[4]}")
def test_compaction(lib, case):
    dcp, bs, I, H, d, dtype, ctx, paths = case
    rng = np.random.default_rng(bs)
    lens = [c + (max(p) + 1 if p else 0) for c, p in zip(ctx, paths)]
    bt, nb = R.random_tables(rng, lens, dcp, bs)
    shape = (nb, bs, d) if H == 1 else (nb, H, bs, d)
    pools = [[torch.randn(shape, device="cuda").to(dtype) for _ in range(dcp)] for _ in range(3)]
    want = [[p.cpu().clone() for p in ps] for ps in pools]
    for ps in want:
        for b, path in enumerate(paths):
            rows = []
            for j in path:
                r, vb, loc = R.place(ctx[b] + j, dcp, bs, I)
                p = ps[r][int(bt[r, b, vb])]
                rows.append((p[loc] if H == 1 else p[:, loc]).clone())
            for i, row in enumerate(rows):
                r, vb, loc = R.place(ctx[b] + i, dcp, bs, I)
                p = ps[r][int(bt[r, b, vb])]
                if H == 1:
                    p[loc] = row
                else:
                    p[:, loc] = row
    most = max(1, max(map(len, paths)))
    path = np.full((len(paths), most), -9, dtype=np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    err = torch.zeros(1, dtype=I32, device="cuda")
    L = lib.Layout(dcp, bs, I)
    new = lib.cache_compact(L, lib.PoolSet(pools), dev(bt), nb, dev(ctx), dev(path),
                            dev([len(p) for p in paths]), err=err)
    assert new.tolist() == [c + len(p) for c, p in zip(ctx, paths)]
    for a, b in zip(pools, want):
        for x, y in zip(a, b):
            assert torch.equal(x.cpu(), y)
    assert err.item() == 0


def test_compaction_stops_at_bad_entries(lib):
    dcp, bs, H, d = 2, 16, 2, 64
    L = lib.Layout(dcp, bs, 1)
    rng = np.random.default_rng(1)
    ctx = [10] * 8
    bt, nb = R.random_tables(rng, [40] * 8, dcp, bs)
    bt[:, 6, 1] = nb                                   # the nodes behind token 31 are nowhere
    pools = [[torch.randn((nb, H, bs, d), device="cuda") for _ in range(dcp)]]
    before = [p.clone() for p in pools[0]]
    path = [[0, 3, 3, 5], [2, 1, 0, 0], [-1, 0, 0, 0], [0, 1, 2, 3], [0, 4, 9, 2000], [5, 6, 7, 8],
            [1, 2, 24, 25], [0, 0, 0, 0]]
    n = [4, 2, 1, 5, 4, -1, 4, 0]
    kept = [2, 1, 0, 0, 3, 0, 2, 0]
    err = torch.zeros(1, dtype=I32, device="cuda")
    new = lib.cache_compact(L, lib.PoolSet(pools), dev(bt), nb, dev(ctx), dev(path), dev(n), err=err)
    assert new.tolist() == [10 + k for k in kept]
    assert err.item() == 7
    for b in range(8):
        for x in range(40):
            r, vb, loc = R.place(x, dcp, bs, 1)
            if bt[r, b, vb] >= nb:
                continue
            y = x
            if 10 <= x < 10 + kept[b]:
                y = 10 + path[b][x - 10]
            r2, vb2, loc2 = R.place(y, dcp, bs, 1)
            assert torch.equal(pools[0][r][int(bt[r, b, vb]), :, loc],
                               before[r2][int(bt[r2, b, vb2]), :, loc2]), (b, x)


def test_refusals(lib):
    L = lib.Layout(2, 16, 1)
    pages = lib.Pages.new(L, 4, 4, 20)
    a = dev([0, 1])
    for bad in (lambda: lib.pages_resize(L, pages, a.long(), a),
                lambda: lib.pages_resize(L, pages, a, a[:1]),
                lambda: lib.pages_resize(L, pages, a, a, copy_src=dev([[0, 0]])),
                lambda: lib.pages_resize(L, pages, a, a, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
                lambda: lib.pages_resize(lib.Layout(3, 16, 1), pages, a, a),
                lambda: lib.pages_fork(L, pages, a.cpu(), a),
                lambda: lib.Pages(pages.block_table, pages.seq_lens.long(), pages.ref_count, pages.free_bits, 20),
                lambda: lib.Pages(pages.block_table, pages.seq_lens, pages.ref_count, pages.free_bits, 21),
                lambda: lib.PoolSet([]),
                lambda: lib.PoolSet([[torch.zeros((4, 16, 64), device="cuda")] * 2, [torch.zeros((4, 16, 32), device="cuda")] * 2]),
                lambda: lib.pages_copy(L, lib.PoolSet([[torch.zeros((4, 16, 64), device="cuda")]]), dev([[0]]), dev([[1]])),
                lambda: lib.pages_copy(L, lib.PoolSet([[torch.zeros((4, 16, 64), device="cuda")] * 2]), dev([[0]]), dev([[1, 2]])),
                lambda: lib.pages_copy(L, lib.PoolSet([[torch.zeros((4, 16, 3), device="cuda")] * 2]), dev([[0]]), dev([[1]])),
                lambda: lib.cache_compact(L, lib.PoolSet([[torch.zeros((4, 16, 64), device="cuda")] * 2]),
                                          pages.block_table, 5, a, a.view(2, 1), a),
                lambda: lib.cache_compact(L, lib.PoolSet([[torch.zeros((4, 16, 64), device="cuda")] * 2]),
                                          pages.block_table, 4, a, a, a)):
        with pytest.raises(lib.DcpError):
            bad()
    with pytest.raises(lib.DcpError):                    # pages of 2^31 tokens a request
        lib.Pages.new(lib.Layout(16, 1 << 20, 1), 1, 1 << 8, 4)


@pytest.mark.parametrize("shape", [(5, 16, 1, 30, 6, 120, False), (2, 16, 2, 2048, 2, 3000, False),
                                   (8, 16, 16, 170, 30, 1500, False)], ids=str)
def test_whole_lists(lib, shape):
    """Every request in one call: the longest list, more CTAs than tables need, a cluster each."""
    dcp, bs, I, B, VB, nb, shared = shape
    L = lib.Layout(dcp, bs, I)
    pages, m = lib.Pages.new(L, B, VB, nb, shared=shared), R.PageModel(dcp, bs, I, B, VB, nb, shared)
    rng = np.random.default_rng(B)
    err = torch.zeros(1, dtype=I32, device="cuda")
    half = B // 2
    for lens in (rng.integers(0, bs * dcp + 1, B), rng.integers(0, 9, B)):
        new = np.where(np.arange(B) < half, lens, 0)
        order = rng.permutation(B)
        src, dst = lib.pages_resize(L, pages, dev(order), dev(new[order]), err=err)
        es, ed = m.resize(order, new[order])
        same(pages, m)
        assert np.array_equal(src.cpu().numpy(), es) and np.array_equal(dst.cpu().numpy(), ed)
        parent, child = rng.permutation(half), half + rng.permutation(half)
        src, dst = lib.pages_fork(L, pages, dev(parent), dev(child), err=err)
        es, ed = m.fork(parent, child)
        same(pages, m)
        assert np.array_equal(src.cpu().numpy(), es) and np.array_equal(dst.cpu().numpy(), ed)
    assert err.item() == 0 and m.err == 0


def test_lengths_from_the_state_itself(lib):
    """The list of lengths may be the state's own: nothing changes."""
    L = lib.Layout(2, 16, 1)
    pages = lib.Pages.new(L, 4, 4, 20)
    lib.pages_resize(L, pages, dev([0, 2]), dev([40, 7]))
    before = [x.clone() for x in (pages.block_table, pages.ref_count, pages.seq_lens)]
    src, dst = lib.pages_resize(L, pages, dev([0, 1, 2, 3]), pages.seq_lens)
    assert (src == -1).all() and (dst == -1).all()
    for a, b in zip(before, (pages.block_table, pages.ref_count, pages.seq_lens)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("order", ["chain", "shift", "exchange", "twice", "mixed", "long"])
@pytest.mark.parametrize("d", [64, 576])
def test_copies_of_the_same_pages_keep_the_order_of_the_list(lib, order, d):
    dcp, nb, bs, pools = 2, 700, 16, 3
    rng = np.random.default_rng(d)
    n = np.arange(40)
    pairs = {
        "chain": list(zip(n, n + 1)),                       # page 0 goes everywhere
        "shift": list(zip(n[::-1], n[::-1] + 1)),           # every page moves one up
        "exchange": [(1, 2), (2, 1), (3, 4), (4, 5), (5, 3)],
        "twice": [(1, 9), (2, 9), (3, 9), (9, 10), (4, 9)],
        "mixed": [(100, 200), (5, 6), (101, 201), (-1, -1), (6, 7), (102, 202), (7, 7), (8, 6),
                  (103, 200)] + [(300 + i, 400 + i) for i in range(50)],
        "long": list(zip(rng.integers(0, nb, 600), rng.integers(0, nb, 600))),
    }[order]
    src, dst = (np.array([[p[i] for p in pairs], [p[i] for p in pairs[::-1]]]) for i in (0, 1))
    ps = torch.randn((pools, dcp, nb, bs, d), generator=torch.Generator().manual_seed(d)).to(
        torch.bfloat16).cuda()
    want = ps.clone()
    for r in range(dcp):
        for a, b in zip(src[r], dst[r]):
            if a >= 0:
                want[:, r, b] = want[:, r, a].clone()
    L, err = lib.Layout(dcp, bs, 1), torch.zeros(1, dtype=I32, device="cuda")
    lib.pages_copy(L, lib.PoolSet([list(p) for p in ps]), dev(src), dev(dst), err=err)
    assert torch.equal(ps, want) and err.item() == 0
    # what cannot be copied touches nothing
    if order == "mixed":
        src[:, 1], dst[:, 4] = nb, -1
        before = ps.clone()
        lib.pages_copy(L, lib.PoolSet([list(p) for p in ps]), dev(src), dev(dst), err=err)
        for r in range(dcp):
            for a, b in zip(src[r], dst[r]):
                if 0 <= a < nb and 0 <= b < nb:
                    before[:, r, b] = before[:, r, a].clone()
        assert torch.equal(ps, before) and err.item() == 4 * pools


def test_a_pool_named_twice_is_moved_once(lib):
    """Layers that share a cache name it more than once."""
    dcp, bs, H, d, B = 1, 16, 8, 512, 1300
    L = lib.Layout(dcp, bs, 1)
    bt = np.arange(B, dtype=np.int32)[None, :, None]
    gen = torch.Generator().manual_seed(2)
    k, v = (torch.randn((B, H, bs, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    want = [x.clone() for x in (k, v)]
    path = [1, 2, 5, 9]
    for w, x in zip(want, (k, v)):
        for i, j in enumerate(path):
            w[:, :, 3 + i] = x[:, :, 3 + j]
    new = lib.cache_compact(L, lib.PoolSet([[k], [v], [k], [v], [k]]), dev(bt), B, dev([3] * B),
                            dev([path] * B), dev([4] * B))
    assert (new == 7).all()
    for x, w in zip((k, v), want):
        assert torch.equal(x, w)
    for pools in ([[k, v], [v, k]], [[k, v], [k, v.clone()]]):     # alike on a rank and no more
        with pytest.raises(lib.DcpError):
            lib.PoolSet(pools)


def test_compaction_of_more_pools_than_shared_memory_has_addresses_for(lib):
    """70 pools on 16 ranks: 1120 addresses, of which the kernel keeps 1024 at most."""
    dcp, bs, H, d, n = 16, 16, 1, 32, 70
    L = lib.Layout(dcp, bs, 1)
    ctx, paths = [5, 250, 0], [[1, 4, 9], [0, 2, 3, 5, 8, 13, 21, 34, 55, 60], [7]]
    rng = np.random.default_rng(n)
    lens = [c + max(p) + 1 for c, p in zip(ctx, paths)]
    bt, nb = R.random_tables(rng, lens, dcp, bs)
    before = torch.randn((n, dcp, nb, bs, d), generator=torch.Generator().manual_seed(n)).cuda()
    after, want = before.clone(), before.clone()
    for b, path in enumerate(paths):
        for i, j in enumerate(path):
            r, vb, loc = R.place(ctx[b] + i, dcp, bs, 1)
            r2, vb2, loc2 = R.place(ctx[b] + j, dcp, bs, 1)
            want[:, r, int(bt[r, b, vb]), loc] = before[:, r2, int(bt[r2, b, vb2]), loc2]
    path = np.full((3, 10), -9, dtype=np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    err = torch.zeros(1, dtype=I32, device="cuda")
    new = lib.cache_compact(L, lib.PoolSet([list(p) for p in after]), dev(bt), nb, dev(ctx),
                            dev(path), dev([len(p) for p in paths]), err=err)
    assert new.tolist() == [c + len(p) for c, p in zip(ctx, paths)] and err.item() == 0
    assert torch.equal(after, want)


@pytest.mark.parametrize("n", [300, 2048, 2500])
@pytest.mark.parametrize("d", [8, 512])
def test_a_few_copies_of_the_same_pages_in_a_long_list(lib, n, d):
    """Lists that CTAs share out, that sets of pages look through first (small pages), and that
    are too long for shared memory; page numbers that fall on the same bits of the sets."""
    dcp, bs, pools = 2, 16, 2
    nb = 40000 if d == 8 else 5600
    rng = np.random.default_rng(n + d)
    src, dst = (np.empty((dcp, n), dtype=np.int64) for _ in range(2))
    for r in range(dcp):
        pages = rng.permutation(nb)[:2 * n]
        src[r], dst[r] = pages[:n], pages[n:]
        for i, j in ((5, 200), (n - 1, 17), (77, n // 2)):
            src[r, i] = dst[r, j]                       # reads what another copy writes
        dst[r, 90] = dst[r, n - 7]                      # a page is written twice
        src[r, 33] = dst[r, 33] = -1
    ps = torch.randn((pools, dcp, nb, bs, d), generator=torch.Generator().manual_seed(n)).to(
        torch.bfloat16).cuda()
    want = ps.clone()
    for r in range(dcp):
        for a, b in zip(src[r], dst[r]):
            if a >= 0:
                want[:, r, b] = want[:, r, a].clone()
    L, err = lib.Layout(dcp, bs, 1), torch.zeros(1, dtype=I32, device="cuda")
    lib.pages_copy(L, lib.PoolSet([list(p) for p in ps]), dev(src), dev(dst), err=err)
    assert torch.equal(ps, want) and err.item() == 0
