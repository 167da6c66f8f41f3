"""Scored decode attention at its edges, against 64 bits: scales and queries of any size, the
cap's accuracy, weights' roundings, and windows where units are cut anywhere."""
import numpy as np
import pytest
import torch

from tests import scored_ref as S
from tests import serving_ref as R
from tests.test_gpu_scored import Problem

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("q", [BF16, F32], ids=str)
@pytest.mark.parametrize("room", [0, 1 << 20])
@pytest.mark.parametrize("lens", [[37], [3000, 5]], ids=str)
def test_values_scales_of_any_size(lib, q, room, lens):
    """Every positive finite scale is read, subnormal ones too, and one of 0 gives zeros: in units
    of the scale the result is what a scale of 1 gives."""
    p = Problem(lib, E4M3, q, 4, 1, 128, 2, 16, 1, lens, room=room, seed=5)
    held = [s.clone() for s in p.kv.scales]
    for b in range(len(lens)):       # the values themselves
        x, k, v = p.rows[b]
        for j, pos in enumerate(x):
            r, vb, _ = R.place(pos, 2, 16, 1)
            v[:, j] /= held[r][int(p.bt[r, b, vb]), :, 1].double().cpu().numpy()[:, None]
    for s in (1.0, 0.037, 2.0 ** 118, 2.0 ** -60, 1.7 * 2.0 ** -100, 2.0 ** -110, 2.0 ** -120,
              2.0 ** -126, 1.375 * 2.0 ** -128, 2.0 ** -130):
        s = float(np.float32(s))
        for t in p.kv.scales:
            t[..., 1] = s
        out, lse = p.run(out_dtype=F32)
        o, l = out.double().cpu().numpy() / s, lse.double().cpu().numpy()
        for b, n in enumerate(lens):
            x, k, v = p.rows[b]
            for h in range(4):
                eo, el, to, tl = S.attend(q, F32, p.q64[b, h], k[0], v[0], x, n, p.scale)
                # of numbers below 2^-126 half of 2^-149 is lost: in a token's weight times the
                # scale and in the factor (of at most 2^-4) of a warp's sum, each beside values of
                # at most 448, and in the result
                lost = 2.0 ** -150 / s * (2 ** 5 * 448 + 1)
                assert (np.abs(o[b, h] - eo) <= to + lost).all(), (s, b, h)
                assert abs(l[b, h] - el) <= tl, (s, b, h)
    for t in p.kv.scales:
        t[..., 1] = 0.0
    out, lse = p.run(out_dtype=F32)
    assert (out == 0).all() and torch.isfinite(lse).all()


def one_hot(p, dims):
    """Every token's key is 1 at its number modulo `dims`, else 0, with scales of 1."""
    for r, pool in enumerate(p.kv.k_pools):
        pool.copy_(torch.zeros(pool.shape, device="cuda").to(E4M3))
        p.kv.scales[r][..., 0] = 1.0
    one = torch.ones(1, device="cuda").to(E4M3).view(torch.uint8)
    for b in range(len(p.lens)):
        for pos in range(p.lens[b]):
            r, vb, loc = R.place(pos, p.dcp, p.bs, p.I)
            p.kv.k_pools[r].view(torch.uint8)[int(p.bt[r, b, vb]), :, loc, pos % dims] = one


@pytest.mark.parametrize("q", [BF16, F32], ids=str)
def test_small_entries_of_a_query(lib, q):
    """A token whose key picks out one entry of the query, down to 2^-45 of the largest: exact to
    2^-31 of it, and off by at most half of 2^-38 of it below (bf16 queries)."""
    p = Problem(lib, E4M3, q, 1, 1, 64, 1, 16, 1, [1] * 48)
    one_hot(p, 1)
    p.q.zero_()
    p.q[:, 0, 1] = 3.0                     # the largest; no key has that dimension
    vals = torch.tensor([1.2890625 * 2.0 ** (1 - e) for e in range(48)])
    p.q[:, 0, 0] = vals.to(q).cuda()
    x = p.q[:, 0, 0].double().cpu().numpy()
    for scale in (1.0, 2.0 ** 40):         # the smallest of them are scores of weight with this
        out, lse = p.decode(p.layout, p.q, p.kv, p.dlens, scale, None)
        got = lse[:, 0].double().cpu().numpy() / scale
        off = 0.0 if q == F32 else np.where(x >= 3.0 * 2.0 ** -31, 0.0, 2.0 * 2.0 ** -39)
        # log2(e), ln(2) and the products with them: 6 roundings at most
        assert (np.abs(got - x) <= np.abs(x) * 6 * 2.0 ** -24 + off).all(), (scale, got, x)


@pytest.mark.parametrize("q", [BF16, F32], ids=str)
def test_infinities_of_a_query(lib, q):
    """Beside an infinite entry the others stay finite: a score of -infinity has no weight."""
    p = Problem(lib, E4M3, q, 2, 1, 64, 1, 16, 1, [20])
    one_hot(p, 1)
    for pool in p.kv.k_pools:              # a second dimension that all keys have
        pool.view(torch.uint8)[..., 1] = torch.ones(1, device="cuda").to(E4M3).view(torch.uint8)
    p.q.zero_()
    p.q[0, 0, 0] = -float("inf")
    p.q[0, 0, 1] = 2.0 ** 100              # no infinity of its own
    p.q[0, 1, 1] = float("nan")
    sink = torch.tensor([0.5, 0.5], device="cuda")
    out, lse = p.decode(p.layout, p.q, p.kv, p.dlens, 1.0, None, sink=sink)
    assert (out[0, 0] == 0).all() and lse[0, 0].item() == 0.5
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("cap", [1.0, 50.0])
def test_a_capped_score(lib, cache, cap):
    """Requests of one token: the LSE is the score, cap * tanh(y / cap), over the range of y."""
    n = 1500
    y = np.exp(np.linspace(np.log(1e-3), np.log(12.0), n)) * cap
    y[::2] *= -1
    p = Problem(lib, cache, F32 if cache == F32 else BF16, 1, 1, 64, 1, 16, 1, [1] * n)
    p.q.zero_()
    pages = p.bt[0, :, 0].long()
    for pool in p.kv.k_pools:
        pool.copy_(torch.zeros(pool.shape, device="cuda").to(cache))
    if cache == E4M3:         # y is a page's scale
        p.q[:, 0, 0] = torch.from_numpy(np.sign(y)).to(p.q.dtype).cuda()
        p.kv.scales[0][pages, 0, 0] = torch.from_numpy(np.abs(y)).float().cuda()
        p.kv.k_pools[0].view(torch.uint8)[pages, 0, 0, 0] = torch.ones(1).to(E4M3).view(torch.uint8).cuda()
        y = (p.q[:, 0, 0].double() * p.kv.scales[0][pages, 0, 0].double()).cpu().numpy()
    else:                     # of bf16 a product of two numbers, exactly; in 32 bits y itself
        q = torch.from_numpy(y).to(p.q.dtype)
        k = (torch.from_numpy(y) / q.double()).to(BF16).to(cache)
        p.q[:, 0, 0] = q.cuda()
        p.kv.k_pools[0][pages, 0, 0, 0] = k.cuda()
        y = (q.double() * k.double()).numpy()
    out, lse = p.decode(p.layout, p.q, p.kv, p.dlens, 1.0, lib.Scores(cap=cap))
    t = cap * np.tanh(y / cap)
    off = np.abs(lse[:, 0].double().cpu().numpy() / t - 1) * 2.0 ** 24
    # in units of 2^-24: tanh 8; y 1 / cap, the constant 1 / cap and the product with the cap 1 each
    # (nothing for a cap of 1); the changes to base 2 and back 1 each, and their constants 1
    assert off.max() <= (11 if cap == 1.0 else 14), (off.max(), y[off.argmax()])


def check_tight(p, out, lse, rounding, floor):
    """The bounds of a kernel in 32 bits whose weights are off by `rounding` relatively, and by
    `floor` of the largest weight times its page's scale of the values."""
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(p.lens):
        x, k, v = p.rows[b]
        for h in range(p.Hq):
            g = h // p.G
            sink = p.sink[h] if p.sink is not None else None
            eo, el, to, tl = S.attend(F32, out.dtype, p.q64[b, h], k[g], v[g], x, n, p.scale, p.cap,
                                      p.slopes[h], sink)
            t = k[g] @ p.q64[b, h] * p.scale
            t = p.cap * np.tanh(t / p.cap) if p.cap else t
            w = np.exp(t - p.slopes[h] * (n - 1 - x) - el)
            to = to + 1.05 * rounding * (w @ np.abs(v[g])) + floor * w.max(initial=0.0) * np.abs(v[g]).sum(0)
            what = f"request {b} head {h} of {n} tokens"
            assert (np.abs(o[b, h] - eo) <= to).all(), (what, (np.abs(o[b, h] - eo) / to).max())
            assert abs(l[b, h] - el) <= tl, what


# cache, q, d, rounding of the weights, floor.  On the tensor cores bf16 caches take weights in two
# bf16 terms, the upper bits and the rest, which is at most 2^-7 of the weight and off by 2^-8 of it,
# together 2^-15 (and 2^-24); 8-bit ones in fp16, held times 2^11 (at least,
# for the largest), so that what falls below fp16's smallest step loses 2^-25 of one at most: 2^-36
# of the largest, and 2^-30 where scales differ by 2^6.  On the CUDA cores nothing is rounded.
WEIGHTS = [(BF16, BF16, 128, 1.01 * 2.0 ** -15, 0.0), (BF16, BF16, 64, 1.01 * 2.0 ** -15, 0.0),
           (E4M3, BF16, 128, 2.0 ** -11, 2.0 ** -30), (E4M3, BF16, 64, 2.0 ** -11, 2.0 ** -30),
           (E4M3, F32, 128, 0.0, 0.0), (BF16, BF16, 96, 0.0, 0.0), (F32, F32, 128, 0.0, 0.0)]


@pytest.mark.parametrize("room", [0, 1 << 20])
@pytest.mark.parametrize("more", [{}, dict(cap=20.0, alibi=True, sink=True)], ids=["", "formed"])
@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: f"{str(c[0])[6:]}-q{str(c[1])[6:]}-d{c[2]}")
def test_roundings_of_the_weights(lib, case, room, more):
    cache, q, d, rounding, floor = case
    for Hq, Hkv in ((8, 2), (16, 1)):
        p = Problem(lib, cache, q, Hq, Hkv, d, 2, 16, 1, [1500, 37, 1], room=room, seed=6, **more)
        check_tight(p, *p.run(out_dtype=F32), rounding, floor)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("window, prefix", [(700, 5), (100000, 0), (2500, 300)])
def test_windows_cut_anywhere(lib, cache, window, prefix):
    """Heads of 128 with a window and kept tokens: units too long for a cluster and more units than
    CTAs, whole and by ranks."""
    q = F32 if cache == F32 else BF16
    rng = np.random.default_rng(window)
    lens = [3000, 2999] if window > 1000 else [int(n) for n in rng.choice([0, 1, 20, 333, 900], 150)]
    p = Problem(lib, cache, q, 8, 4, 128, 2, 16, 1, lens, window=window, prefix=prefix, cap=20.0,
                sink=True, room=1 << 20)
    p.check(*p.run())
    po, pl = p.partial(p.layout, p.q, p.kv, p.dlens, p.scale, p.form)
    for r in range(2):
        p.check(po[r], pl[r], rank=r)


@pytest.mark.parametrize("cache, d", [(BF16, 128), (BF16, 64), (BF16, 96), (F32, 128)], ids=str)
@pytest.mark.parametrize("room", [0, 1 << 20])
def test_infinite_values(lib, cache, d, room):
    """A value of infinity gives one, whatever the weight's bits (a weight of 1 among them)."""
    p = Problem(lib, cache, F32 if cache == F32 else BF16, 8, 2, d, 2, 16, 1, [300, 40, 1], room=room)
    for b, pos, c, x in ((0, 200, 3, float("inf")), (0, 7, 9, -float("inf")), (2, 0, 5, float("inf"))):
        r, vb, loc = R.place(pos, 2, 16, 1)
        p.kv.v_pools[r][int(p.bt[r, b, vb]), :, loc, c] = x
    out, lse = p.run()
    assert (out[0, :, 3] == float("inf")).all() and (out[0, :, 9] == -float("inf")).all()
    assert (out[2, :, 5] == float("inf")).all()
    rest = torch.ones(d, dtype=torch.bool, device="cuda")
    rest[[3, 9, 5]] = False
    assert torch.isfinite(out[..., rest]).all() and torch.isfinite(out[1]).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("cache", [BF16, E4M3, F32], ids=str)
@pytest.mark.parametrize("tokens", [300, 1500, 5000, 12000])
def test_documents_from_0_are_requests(lib, cache, tokens):
    """A call whose documents all start at 0 is cut as one without starts, and gives the same bits."""
    q = F32 if cache == F32 else BF16
    L, B, H, d, bs = lib.Layout(3, 32, 4), 16, 1, 64, 32
    blocks = -(-tokens // 96)
    bt = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(1, B, blocks).expand(3, -1, -1).contiguous()
    mk = lambda: [torch.randn((B * blocks, H, bs, d), device="cuda").to(cache) for _ in range(3)]  # noqa: E731
    if cache == E4M3:
        kv = lib.PagedKV8(mk(), mk(), [torch.ones((B * blocks, H, 4), device="cuda") for _ in range(3)],
                          bt, B * blocks)
        decode = lib.q8_decode_gqa
    else:
        kv, decode = lib.PagedKV(mk(), mk(), bt, B * blocks), lib.scored_decode_gqa
    x = torch.randn((B, 16, d), device="cuda").to(q)
    lens = torch.linspace(tokens // 16, tokens, B, device="cuda").int()
    zeros = torch.zeros(B, dtype=torch.int32, device="cuda")
    for kw in ({}, dict(window=tokens // 2, prefix=4)):
        a = decode(L, x, kv, lens, d ** -0.5, lib.Scores(first=zeros, **kw))
        b = decode(L, x, kv, lens, d ** -0.5, lib.Scores(**kw))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q", [BF16, F32], ids=str)
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scales_that_are_none_show(lib, q, which, bad):
    """A seen page whose scale is NaN or infinite does not give numbers that look like results."""
    p = Problem(lib, E4M3, q, 4, 1, 64, 2, 16, 1, [100, 40])
    p.kv.scales[1][int(p.bt[1, 0, 1]), 0, which] = bad
    out, lse = p.run()
    assert not torch.isfinite(out[0]).any() and torch.isfinite(out[1]).all()
    assert torch.isfinite(lse[1]).all() and (which == 1 or not torch.isfinite(lse[0]).any())


FIRST = """
import torch, sys
sys.path.insert(0, {root!r})
import context_paged_decode_gb300 as dcp
L = dcp.Layout(2, 16, 1)
bt = torch.zeros((2, 1, 1), dtype=torch.int32, device="cuda")
lens = torch.tensor([20], dtype=torch.int32, device="cuda")
calls = []
for dt in (torch.bfloat16, torch.float32):
    for d in (64, 256):
        q = torch.ones((1, 4, d), dtype=dt, device="cuda")
        pool = [torch.ones((1, 2, 16, d), dtype=dt, device="cuda")] * 2
        kv8 = dcp.PagedKV8([p.to(torch.float8_e4m3fn) for p in pool], [p.to(torch.float8_e4m3fn) for p in pool],
                           [torch.ones((1, 2, 4), device="cuda")] * 2, bt, 1)
        calls.append((dcp.scored_decode_gqa, q, dcp.PagedKV(pool, pool, bt, 1)))
        calls.append((dcp.q8_decode_gqa, q, kv8))
torch.cuda.synchronize()
for call, q, kv in calls:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call(L, q, kv, lens, 1.0, dcp.Scores())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, torch.ones_like(q)), call
print("ok")
"""


def test_first_calls_captured():
    """In a process of their own, calls that are captured before any other has run."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
