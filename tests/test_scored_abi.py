"""Host-side refusals of the 8-bit cache and of scored decode attention (CPU only:
each returns before anything is launched; the pointers are never followed), and
the models that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests import scored_ref as S
from tests import serving_ref as R
from tests.test_serving_abi import dcp, kv, ranks  # noqa: F401

EINVAL, EWORKSPACE, EUNSUPPORTED = -1, -2, -4
P = C.c_void_p(1 << 20)          # an aligned address that nothing reads
OUT, WS = C.c_void_p(1 << 50), C.c_void_p(1 << 51)


def kv8(dcp, n=2, base=1 << 40, max_vb=4, nb=8):  # noqa: F811
    s = dcp.PagedKV8Struct()
    s.k = s.v = s.scale = ranks(dcp, n, base)
    s.num_blocks, s.block_table, s.max_vblocks, s.bt_rank_stride = nb, 1 << 20, max_vb, 16
    return s


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("partial", [False, True])
def test_attention(dcp, eight, partial):  # noqa: F811
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)
    make = kv8 if eight else (lambda d, **k: kv(d, **{**dict(base=1 << 40), **k}))
    fn = getattr(lib, f"dcp_{'q8' if eight else 'scored'}_{'partial' if partial else 'decode'}_gqa")

    def call(layout=L, q=P, B=2, Hq=8, Hkv=2, d=128, scale=1.0, dt=1, cache=None, lens=P,
             cap=0.0, window=0, prefix=0, slopes=None, first=None, sink=None, out=OUT, odt=1,
             lse=C.c_void_p(1 << 49), ws=WS, n=1 << 40):
        f = dcp.ScoresStruct(cap, window, prefix, slopes, first)
        head = [layout, q, B, Hq, Hkv, d, scale, dt, cache or make(dcp), lens, f]
        tail = [out, lse] if partial else [sink, out, odt, lse]
        return fn(*head, *tail, ws, n, None, None)

    assert call(B=0) == 0
    bad = [dict(layout=dcp.Layout(0, 16, 1)), dict(layout=dcp.Layout(2, 16, 3)),
           dict(layout=dcp.Layout(16, 1 << 28, 1)), dict(B=-1), dict(Hq=6, Hkv=4),
           dict(Hq=34, Hkv=2), dict(Hkv=0), dict(d=0), dict(d=48), dict(d=288), dict(dt=2),
           dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(lens=None),
           dict(out=None), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")),
           dict(cap=1e-39),   # 1 / cap is beyond 32 bits
           dict(window=-1), dict(prefix=-1), dict(cache=make(dcp, nb=-1)),
           dict(cache=make(dcp, max_vb=-1)), dict(cache=make(dcp, n=1)),
           # outputs, workspace and what is read lie apart
           dict(out=P), dict(ws=OUT), dict(lse=OUT), dict(out=C.c_void_p(1 << 40)),
           dict(ws=C.c_void_p((1 << 40) + 16)), dict(lse=P)]
    if partial:
        bad.append(dict(lse=None))
    else:
        bad += [dict(odt=2), dict(sink=OUT)]
    for b in bad:
        assert call(**b) == EINVAL, b
    assert call(ws=None) == EWORKSPACE and call(n=100) == EWORKSPACE
    for b in (dict(q=C.c_void_p((1 << 20) + 2)), dict(out=C.c_void_p((1 << 50) + 8)),
              dict(ws=C.c_void_p((1 << 51) + 8)), dict(cache=make(dcp, base=(1 << 40) + 8)),
              dict(B=1 << 29),
              # room for more tokens of a request than 31 bits count, products beyond 63 bits
              dict(B=1, Hkv=1, cache=make(dcp, max_vb=1 << 26)),
              dict(layout=dcp.Layout(2, 1 << 28, 1), B=4096, Hq=8192, Hkv=8192,
                   cache=make(dcp, nb=0, max_vb=(1 << 31) - 1))):
        assert call(**b) == EUNSUPPORTED, b


def test_workspace(dcp):  # noqa: F811
    lib, L = dcp.load(), dcp.Layout(8, 16, 1)
    n, m = C.c_size_t(0), C.c_size_t(0)
    assert lib.dcp_scored_workspace_size(L, 4, 32, 8, 128, 0, C.byref(n)) == 0
    assert lib.dcp_scored_workspace_size(L, 4, 32, 8, 128, 1, C.byref(m)) == 0
    assert 0 < n.value < m.value
    assert lib.dcp_scored_workspace_size(L, 4, 32, 8, 100, 0, C.byref(n)) == EINVAL
    assert lib.dcp_scored_workspace_size(L, -1, 32, 8, 128, 0, C.byref(n)) == EINVAL
    assert lib.dcp_scored_workspace_size(L, 4, 32, 8, 128, 0, None) == EINVAL


def test_append(dcp):  # noqa: F811
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)

    def call(layout=L, k=P, ks=256, v=P, vs=256, N=5, start=P, ctx=P, B=2, Hkv=2, d=128, dt=1,
             cache=None):
        return lib.dcp_q8_append_gqa(layout, k, ks, v, vs, N, start, ctx, B, Hkv, d, dt,
                                     cache or kv8(dcp), None, None)

    assert call(N=0) == 0 and call(B=0) == 0
    for bad in (dict(layout=dcp.Layout(2, 16, 5)), dict(N=-1), dict(B=-1), dict(Hkv=0), dict(d=0),
                dict(d=40), dict(d=288), dict(dt=2), dict(ks=255), dict(vs=0), dict(k=None),
                dict(v=None), dict(start=None), dict(ctx=None), dict(cache=kv8(dcp, n=1)),
                dict(cache=kv8(dcp, nb=-1)), dict(cache=kv8(dcp, max_vb=-1)),
                dict(k=C.c_void_p(1 << 40)), dict(v=C.c_void_p((1 << 40) - 16)),
                dict(ctx=C.c_void_p(1 << 40))):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(k=C.c_void_p((1 << 20) + 8)), dict(v=C.c_void_p((1 << 20) + 2)),
                dict(ks=257), dict(vs=260), dict(cache=kv8(dcp, base=(1 << 40) + 4))):
        assert call(**bad) == EUNSUPPORTED, bad


def test_gather(dcp):  # noqa: F811
    lib, L = dcp.load(), dcp.Layout(2, 16, 1)

    def call(layout=L, B=2, Hkv=2, d=128, req=P, pos=P, N=5, k=OUT, v=WS, dt=1, cache=None):
        return lib.dcp_q8_gather_gqa(layout, cache or kv8(dcp), B, Hkv, d, req, pos, N, k, v, dt,
                                     None, None)

    assert call(N=0) == 0
    for bad in (dict(layout=dcp.Layout(2, 16, 5)), dict(N=-1), dict(B=-1), dict(Hkv=0), dict(d=33),
                dict(dt=3), dict(req=None), dict(pos=None), dict(k=None), dict(v=None),
                dict(cache=kv8(dcp, n=1)), dict(v=OUT), dict(k=P), dict(v=C.c_void_p(1 << 40))):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(k=C.c_void_p((1 << 50) + 8)), dict(cache=kv8(dcp, base=(1 << 40) + 4)),
                dict(N=1 << 31)):
        assert call(**bad) == EUNSUPPORTED, bad


def test_model_of_e4m3():
    """Every fp16 number, against torch's conversion."""
    x = np.arange(1 << 16, dtype=np.uint16).view(np.float16).astype(np.float64)
    got = S.nearest8(x)
    want = torch.from_numpy(x).float().clamp(-448, 448).to(S.E4M3).double().numpy()
    assert np.array_equal(got, want, equal_nan=True)


def test_model_of_scales():
    for top, s in ((0.0, 2.0 ** -60), (448.0, 1.0), (448.1, 2.0), (1.75, 2.0 ** -8),
                   (1.76, 2.0 ** -7), (3.3e38, 2.0 ** 120), (1e-30, 2.0 ** -60)):
        assert S.need(top) == s and top / s <= 448


def test_model_of_append_by_tokens():
    """Token by token, a page's numbers are what came in to e4m3's rounding."""
    rng = np.random.default_rng(0)
    dcp_, bs, I, H, d = 2, 8, 2, 1, 32
    bt, nb = R.random_tables(rng, [50], dcp_, bs)
    pool = np.full((dcp_, nb, H, bs, d), np.nan)
    sc = np.full((dcp_, nb, H), np.nan)
    x = rng.standard_normal((50, H, d)) * rng.choice([0.01, 1.0, 100.0], (50, 1, 1))
    for t in range(50):
        S.append(pool, sc, x[t:t + 1], bt[:, 0], t, dcp_, bs, I)
    for t in range(50):
        r, vb, loc = R.place(t, dcp_, bs, I)
        assert S.position(vb, r, loc, dcp_, bs, I) == t
        page = bt[r, 0, vb]
        y = pool[r, page, 0, loc] * sc[r, page, 0]
        # one rounding of the number, and one below the smallest step at each growth (two at most)
        assert (np.abs(y - x[t, 0]) <= np.abs(x[t, 0]) * 2.0 ** -4 + 3 * 2.0 ** -10 * sc[r, page, 0]).all()


def test_model_of_attention():
    """The cap, the bias and the window against a sum written out."""
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal(8), rng.standard_normal((30, 8)), rng.standard_normal((30, 8))
    seen = S.seen_mask(30, 7, 3, 4)
    assert list(np.nonzero(seen)[0]) == [4, 5, 6] + list(range(23, 30))
    x = np.nonzero(seen)[0]
    o, lse, to, tl = S.attend(torch.bfloat16, torch.float32, q, k[x], v[x], x, 30, 0.3, 2.0, 0.1, 0.5)
    num, den = np.zeros(8), np.exp(0.5)
    for j in x:
        w = np.exp(2.0 * np.tanh(0.3 * (q @ k[j]) / 2.0) - 0.1 * (29 - j))
        num, den = num + w * v[j], den + w
    assert np.allclose(o, num / den, rtol=1e-13) and np.isclose(lse, np.log(den), rtol=1e-13)
    assert (to < 0.02).all() and tl < 1e-4
