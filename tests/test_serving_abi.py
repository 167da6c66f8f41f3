"""Host-side refusals of the calls around the decode step (CPU only: each
returns before anything is launched; the pointers are never followed), and the
page model that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest

from tests import serving_ref as R

EINVAL, EWORKSPACE, EUNSUPPORTED = -1, -2, -4
P = C.c_void_p(1 << 20)          # an aligned address that nothing reads


@pytest.fixture(scope="module")
def dcp():
    from context_paged_decode_gb300 import build
    build.build_all()
    import context_paged_decode_gb300 as d
    d.load()
    return d


def ranks(dcp, n, base=1 << 20):
    rp = dcp.RankPtrs()
    for i in range(n):
        rp.ptr[i] = base
    return rp


def kv(dcp, n=2, base=1 << 20, max_vb=4, nb=8):
    s = dcp.PagedKVStruct()
    s.k = s.v = ranks(dcp, n, base)
    s.num_blocks, s.block_table, s.max_vblocks, s.bt_rank_stride = nb, 1 << 20, max_vb, 16
    return s


def test_tree(dcp):
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)

    def call(layout=L, q=P, start=P, N=5, B=2, most=4, Hq=8, Hkv=2, d=128, scale=1.0, dt=1,
             cache=None, ctx=P, mask=P, out=P, odt=1, ws=P, n=1 << 40):
        return lib.dcp_tree_decode_gqa(layout, q, start, N, B, most, Hq, Hkv, d, scale, dt,
                                       cache or kv(dcp), ctx, mask, None, out, odt, None, ws, n,
                                       None, None)

    assert call(N=0) == 0 and call(B=0) == 0
    for bad in (dict(layout=dcp.Layout(0, 16, 1)), dict(layout=dcp.Layout(2, 16, 3)), dict(N=-1),
                dict(B=-1), dict(most=0), dict(most=65), dict(Hq=6, Hkv=4), dict(Hq=34, Hkv=2),
                dict(Hkv=0), dict(d=0), dict(d=48), dict(d=288), dict(dt=2), dict(odt=2),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(q=None),
                dict(start=None), dict(ctx=None), dict(mask=None), dict(out=None),
                dict(cache=kv(dcp, 1)), dict(cache=kv(dcp, nb=-1)), dict(cache=kv(dcp, max_vb=-1))):
        assert call(**bad) == EINVAL, bad
    assert call(ws=None) == EWORKSPACE and call(n=100) == EWORKSPACE
    assert call(q=C.c_void_p((1 << 20) + 2)) == EUNSUPPORTED
    assert call(cache=kv(dcp, base=(1 << 20) + 8)) == EUNSUPPORTED
    assert call(cache=kv(dcp, max_vb=1 << 27)) == EUNSUPPORTED
    assert call(B=1 << 27) == EUNSUPPORTED
    n = C.c_size_t(0)
    assert lib.dcp_tree_workspace_size(L, 2, 4, 8, 2, 128, 1, C.byref(n)) == 0 and n.value > 0
    assert lib.dcp_tree_workspace_size(L, 2, 65, 8, 2, 128, 1, C.byref(n)) == EINVAL
    assert lib.dcp_tree_partial_gqa(L, P, P, 5, 2, 4, 8, 2, 128, 1.0, 1, kv(dcp), P, P, P, None, P,
                                    1 << 40, None, None) == EINVAL


def test_rope(dcp):
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)

    def call(layout=L, q=P, qs=1024, k=P, ks=256, v=P, vs=256, T=3, Hq=8, Hkv=2, d=128, dt=1, pos=P,
             axes=1, inv=P, rot=128, slot=P, nb=8, kc=None, vc=None, q_out=P, k_out=None):
        return lib.dcp_rope_write_gqa(layout, q, qs, k, ks, v, vs, T, Hq, Hkv, d, dt, pos, axes,
                                      inv, None, rot, 0, 1.0, slot, nb, kc or ranks(dcp, 2),
                                      vc or ranks(dcp, 2), q_out, k_out, None, None)

    assert call(T=0) == 0
    for bad in (dict(layout=dcp.Layout(2, 16, 5)), dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(d=0),
                dict(dt=7), dict(rot=0), dict(rot=144), dict(axes=0), dict(nb=-1), dict(q=None),
                dict(q_out=None), dict(k=None), dict(v=None), dict(pos=None), dict(inv=None),
                dict(slot=None), dict(kc=ranks(dcp, 1)), dict(vc=ranks(dcp, 1)), dict(qs=1000),
                dict(ks=255), dict(vs=0)):
        assert call(**bad) == EINVAL, bad
    odd = C.c_void_p((1 << 20) + 8)
    for bad in (dict(rot=24), dict(d=132, qs=1 << 20, ks=1 << 20, vs=1 << 20), dict(T=1 << 31),
                dict(d=16384, qs=1 << 20, ks=1 << 20, vs=1 << 20), dict(q=odd), dict(k=odd),
                dict(v=odd), dict(q_out=odd), dict(k_out=odd), dict(qs=1028), dict(ks=257),
                dict(kc=ranks(dcp, 2, (1 << 20) + 4)), dict(Hq=1 << 30, qs=1 << 40)):
        assert call(**bad) == EUNSUPPORTED, bad
    mla = lambda **k: lib.dcp_rope_write_mla(  # noqa: E731
        L, P, k.get("qs", 4608), P, k.get("ks", 576), 3, 8, 576, 1, P, 1, P, None, k.get("rot", 64),
        1, 1.0, P, 8, ranks(dcp, k.get("n", 2)), P, None, None)
    assert mla(rot=592) == EINVAL and mla(qs=4000) == EINVAL and mla(n=1) == EINVAL
    assert mla(rot=56) == EUNSUPPORTED and mla(ks=577) == EUNSUPPORTED


def test_pages(dcp):
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)

    def pages(**k):
        s = dict(block_table=1 << 20, seq_lens=1 << 20, ref_count=1 << 20, free_bits=1 << 20,
                 num_reqs=4, max_vblocks=8, bt_rank_stride=32, num_blocks=100)
        s.update(k)
        return dcp.PagesStruct(*s.values())

    def call(p=None, layout=L, a=P, b=P, n=3, src=P, dst=P, ws=P, nb=1 << 40, name="resize"):
        return getattr(lib, "dcp_pages_" + name)(layout, p or pages(), a, b, n, src, dst, ws, nb,
                                                 None, None)

    for name in ("resize", "fork"):
        assert call(n=0, name=name) == 0
        for bad in (dict(layout=dcp.Layout(2, 0, 1)), dict(n=-1), dict(a=None), dict(b=None),
                    dict(src=None), dict(dst=None), dict(p=pages(num_reqs=-1)),
                    dict(p=pages(max_vblocks=-1)), dict(p=pages(num_blocks=-1)),
                    dict(p=pages(bt_rank_stride=-1)), dict(p=pages(bt_rank_stride=31)),
                    dict(p=pages(block_table=None)), dict(p=pages(seq_lens=None)),
                    dict(p=pages(ref_count=None)), dict(p=pages(free_bits=None))):
            assert call(name=name, **bad) == EINVAL, bad
        assert call(ws=None, name=name) == EWORKSPACE and call(nb=64, name=name) == EWORKSPACE
        assert call(p=pages(num_blocks=1 << 31), name=name) == EUNSUPPORTED
        assert call(n=2049, name=name) == EUNSUPPORTED
        assert call(p=pages(max_vblocks=1 << 26, bt_rank_stride=1 << 40), name=name) == EUNSUPPORTED
    n = C.c_size_t(0)
    assert lib.dcp_pages_workspace_size(L, pages(), 3, C.byref(n)) == 0 and n.value > 0
    assert lib.dcp_pages_workspace_size(L, pages(), -1, C.byref(n)) == EINVAL
    assert lib.dcp_pages_init(L, pages(seq_lens=None), None) == EINVAL


def test_moves(dcp):
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)

    def pools(**k):
        s = dict(ptr=1 << 20, num_pools=2, num_heads=2, row_bytes=256, num_blocks=8)
        s.update(k)
        return dcp.PoolSetStruct(*s.values())

    copy = lambda p=None, L=L, src=P, dst=P, t=2, n=3: lib.dcp_pages_copy(  # noqa: E731
        L, p or pools(), src, dst, t, n, None, None)
    assert copy(n=0) == 0 and copy(p=pools(num_pools=0)) == 0
    for bad in (dict(L=dcp.Layout(2, 16, 7)), dict(p=pools(num_pools=-1)), dict(p=pools(num_heads=0)),
                dict(p=pools(row_bytes=0)), dict(p=pools(num_blocks=-1)), dict(p=pools(ptr=None)),
                dict(src=None), dict(dst=None), dict(t=3), dict(n=-1)):
        assert copy(**bad) == EINVAL, bad
    assert copy(p=pools(row_bytes=24)) == EUNSUPPORTED

    def move(p=None, L=L, bt=P, B=2, vb=4, stride=8, ctx=P, path=P, n=P, most=4):
        return lib.dcp_cache_compact(L, p or pools(), bt, B, vb, stride, ctx, path, n, most, None,
                                     None, None)

    assert move(B=0) == 0
    for bad in (dict(L=dcp.Layout(17, 16, 1)), dict(p=pools(ptr=None)), dict(bt=None), dict(B=-1),
                dict(vb=-1), dict(stride=-1), dict(ctx=None), dict(path=None), dict(n=None),
                dict(most=-1)):
        assert move(**bad) == EINVAL, bad
    assert move(p=pools(row_bytes=8)) == EUNSUPPORTED


def test_page_model_keeps_its_invariants():
    """Counts are the holders, every page is held or free, open pages have one holder."""
    rng = np.random.default_rng(0)
    for dcp, bs, I, shared in ((2, 4, 2, False), (3, 4, 4, False), (2, 4, 1, True)):
        m = R.PageModel(dcp, bs, I, 6, 5, 80, shared)
        for step in range(60):
            if step % 3 < 2:
                k = rng.permutation(6)[:3]
                m.resize(k, rng.integers(0, 5 * bs * dcp + 1, 3))
            else:
                p = rng.permutation(6)
                m.fork(p[3:], p[:3])
            for t in range(m.tables):
                held = np.bincount(m.bt[t][m.bt[t] >= 0], minlength=80)
                assert np.array_equal(held, m.ref[t])
                for b in range(6):
                    assert ((m.bt[t, b] >= 0).sum()) == m.blocks(m.seq[b])
                    at = m.open(int(m.seq[b]), t)
                    assert at is None or m.ref[t, m.bt[t, b, at[0]]] == 1
        assert m.err == 0


def test_outputs_over_inputs_and_odd_workspaces(dcp):
    """What the kernels could not keep apart is refused before anything is launched."""
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)
    Q, odd = C.c_void_p(1 << 21), lambda n: C.c_void_p((1 << 20) + n)  # noqa: E731

    def tree(out=Q, ws=P, layout=L, cache=None):
        return lib.dcp_tree_decode_gqa(layout, P, P, 5, 2, 4, 8, 2, 128, 1.0, 1, cache or kv(dcp), P,
                                       P, None, out, 1, None, ws, 1 << 40, None, None)

    assert tree(out=P) == EINVAL and tree(out=odd(8)) == EUNSUPPORTED
    assert tree(ws=odd(8)) == EWORKSPACE
    assert tree(layout=dcp.Layout(4, 1 << 29, 1), cache=kv(dcp, 4, max_vb=0)) == EUNSUPPORTED
    pages = lambda vb=8: dcp.PagesStruct(1 << 20, 1 << 20, 1 << 20, 1 << 20, 4, vb, 32, 100)  # noqa: E731
    for name in ("resize", "fork"):
        f = getattr(lib, "dcp_pages_" + name)
        assert f(L, pages(), P, P, 3, P, P, P, 1 << 40, None, None) == EINVAL
        assert f(L, pages(), P, P, 3, P, Q, odd(2), 1 << 40, None, None) == EWORKSPACE
        assert f(dcp.Layout(4, 1 << 29, 1), pages(0), P, P, 3, P, Q, P, 1 << 40, None,
                 None) == EUNSUPPORTED
    pools = dcp.PoolSetStruct(1 << 20, 2, 2, 256, 8)
    assert lib.dcp_pages_copy(L, pools, P, P, 2, 3, None, None) == EINVAL
    move = lambda new, L=L: lib.dcp_cache_compact(  # noqa: E731
        L, pools, P, 2, 4, 8, P, Q, P, 4, new, None, None)
    assert move(P) == EINVAL and move(odd(4)) == EINVAL and move(odd(-4)) == EINVAL
    assert move(None, dcp.Layout(4, 1 << 29, 1)) == EUNSUPPORTED


def test_rotated_rows_over_their_inputs(dcp):
    """CTAs read some tokens while others are written: an output may be its own input, packed,
    and nothing else."""
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)
    at = lambda n: C.c_void_p((1 << 24) + n)  # noqa: E731
    far = [C.c_void_p(x << 20) for x in (1, 2, 3, 4)]
    row, kr = 8 * 128 * 2, 2 * 128 * 2          # bytes of a token's queries and keys

    def gqa(q_out, k_out=None, q=at(0), qs=1024, k=far[0], ks=256, v=far[1], vs=256, T=3, inv=far[2]):
        return lib.dcp_rope_write_gqa(L, q, qs, k, ks, v, vs, T, 8, 2, 128, 1, far[2], 1, inv, None,
                                      128, 0, 1.0, far[3], 8, ranks(dcp, 2), ranks(dcp, 2), q_out,
                                      k_out, None, None)

    wide = 8 * 128 + 4 * 128                    # elements of a token in a fused projection
    assert gqa(at(0), qs=wide) == EINVAL                            # the slice itself
    assert gqa(at(16)) == EINVAL and gqa(at(-16)) == EINVAL         # a packed q, off by a little
    assert gqa(at(3 * row - 16)) == EINVAL and gqa(at(16 - 3 * row)) == EINVAL
    for kw in (dict(k=at(row), v=at(row + kr)), dict(k=at(row), v=far[1]), dict(k=far[0], v=at(row))):
        assert gqa(at(0), q=far[1], ks=wide, vs=wide, **kw) == EINVAL   # over keys or values
    assert gqa(far[1], at(0), qs=wide) == EINVAL and gqa(at(1 << 23), far[1]) == EINVAL
    assert gqa(at(1 << 23), far[0], ks=512) == EINVAL               # keys that are not packed
    assert gqa(at(1 << 23), at((1 << 23) + 16)) == EINVAL           # outputs over one another
    for x in (far[2], far[3], C.c_void_p((2 << 20) + 16)):
        assert gqa(x) == EINVAL
    mla = lambda q_out, qs=8 * 576, ks=576, kv=far[0], T=3: lib.dcp_rope_write_mla(  # noqa: E731
        L, at(0), qs, kv, ks, T, 8, 576, 1, far[2], 1, far[2], None, 64, 1, 1.0, far[3], 8,
        ranks(dcp, 2), q_out, None, None)
    assert mla(at(0), qs=9 * 576) == EINVAL and mla(at(0), kv=at(8 * 576 * 2), ks=9 * 576) == EINVAL
    assert mla(at(32)) == EINVAL and mla(far[0]) == EINVAL and mla(far[3]) == EINVAL


def test_lists_of_pages_lie_apart(dcp):
    """A list that the call itself writes over would name requests that were never checked."""
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)
    at = lambda mib, off=0: C.c_void_p((mib << 20) + off)  # noqa: E731
    # 4 requests of 8 pages, 2 tables of 100 pages
    state = dict(block_table=1, seq_lens=2, ref_count=3, free_bits=4)
    pages = dcp.PagesStruct(*(x << 20 for x in state.values()), 4, 8, 32, 100)
    size = dict(block_table=256, seq_lens=16, ref_count=800, free_bits=32)

    def call(name, a=at(5), b=at(6), src=at(7), dst=at(8), ws=at(9)):
        return getattr(lib, "dcp_pages_" + name)(L, pages, a, b, 3, src, dst, ws, 1 << 20, None, None)

    for name in ("resize", "fork"):
        row = "a" if name == "resize" else "b"       # the requests that change
        for a, b in (("src", "dst"), ("src", "a"), ("src", "b"), ("dst", "a"), ("dst", "b"),
                     ("ws", "a"), ("ws", "b"), ("src", "ws"), ("dst", "ws")):
            assert call(name, **{a: at(20), b: at(20, 8)}) == EINVAL, (a, b)
            assert call(name, **{b: at(20), a: at(20, 8)}) == EINVAL, (a, b)
        for what, mib in state.items():
            end = at(mib, size[what] - 4)
            for arg in ("src", "dst", "ws", row) + (() if what == "seq_lens" else ("a", "b")):
                assert call(name, **{arg: at(mib)}) == EINVAL, (what, arg)
                assert call(name, **{arg: end}) == EINVAL, (what, arg)


def test_new_lengths_lie_apart_from_what_a_compaction_reads(dcp):
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)
    at = lambda mib, off=0: C.c_void_p((mib << 20) + off)  # noqa: E731
    pools = dcp.PoolSetStruct(1 << 20, 2, 2, 256, 8)
    # 3 requests, paths of 5 entries, tables of 3 x 4 pages 16 apart, 4 pool addresses
    move = lambda new: lib.dcp_cache_compact(  # noqa: E731
        L, pools, at(2), 3, 4, 16, at(3), at(4), at(5), 5, new, None, None)
    for mib, size in ((1, 4 * 8), (2, (16 + 12) * 4), (3, 12), (4, 60), (5, 12)):
        for off in (0, size - 4, -8):
            assert move(at(mib, off)) == EINVAL, (mib, off)


def test_tree_outputs_lie_apart(dcp):
    """From the queries, the lists, the masks and the table, which CTAs read to the end."""
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)
    at = lambda mib, off=0: C.c_void_p((mib << 20) + off)  # noqa: E731
    N, B, Hq, d = 5, 2, 8, 128
    cache = kv(dcp, base=30 << 20)
    cache.block_table = 1 << 20                  # 2 tables of 2 x 4 entries, 16 apart
    read = {1: (16 + 8) * 4, 2: N * Hq * d * 2, 3: (B + 1) * 4, 4: B * 4, 5: N * 8, 6: Hq * 4}

    def call(out=at(7), lse=at(8), ws=at(9), partial=False):
        if partial:
            return lib.dcp_tree_partial_gqa(L, at(2), at(3), N, B, 4, Hq, 2, d, 1.0, 1, cache, at(4),
                                            at(5), out, lse, ws, 1 << 40, None, None)
        return lib.dcp_tree_decode_gqa(L, at(2), at(3), N, B, 4, Hq, 2, d, 1.0, 1, cache, at(4), at(5),
                                       at(6), out, 1, lse, ws, 1 << 40, None, None)

    for partial in (False, True):
        for mib, size in read.items():
            if partial and mib == 6:
                continue
            for arg in ("out", "lse", "ws"):
                for off in (0, (size - 1) // 16 * 16, -16):
                    assert call(partial=partial, **{arg: at(mib, off)}) == EINVAL, (arg, mib, off)
        for a, b in (("out", "lse"), ("out", "ws"), ("lse", "ws")):
            assert call(partial=partial, **{a: at(20), b: at(20, 32)}) == EINVAL
            assert call(partial=partial, **{b: at(20), a: at(20, 32)}) == EINVAL
