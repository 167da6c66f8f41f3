"""Rotary positions fused with the cache write, against 64-bit rotation."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def slots(rng, T, dcp, nb, bs):
    """Slots of T tokens [dcp, T]: one rank each, no two alike; every seventh is padding."""
    out = np.full((dcp, T), -1, dtype=np.int64)
    at = rng.permutation(nb * bs)[:T]
    for t in range(T):
        if t % 7 != 6:
            out[t % dcp, t] = at[t]
    return out


def inv_freqs(half, base=10000.0):
    return (base ** (-np.arange(half) / half)).astype(np.float32)


def pools(dcp, shape, dtype):
    return [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(dcp)]


def stored(pool, slot, bs, latent):
    """Rows of a rank's pool at slots [n] -> [n, ...]."""
    s = torch.from_numpy(slot).cuda()
    return pool[s // bs, s % bs] if latent else pool[s // bs, :, s % bs]


# dtype, T, Hq, Hkv, d, rot, axes, interleaved, far, dcp, bs, scaling
GQA = [
    (F32, 1, 8, 2, 64, 64, 1, False, 100, 2, 16, 1.0),
    (F32, 33, 3, 1, 128, 64, 3, True, 1 << 20, 1, 16, 1.25),
    (F32, 9, 1, 1, 48, 16, 2, False, 1 << 31, 3, 8, 1.0),
    (BF16, 70, 32, 8, 128, 128, 1, False, 1 << 17, 8, 16, 1.0),
    (BF16, 29, 8, 8, 128, 128, 3, False, 1 << 17, 4, 32, 1.0),
    (BF16, 29, 16, 2, 64, 32, 4, True, 1 << 32, 2, 64, 0.8),
    (BF16, 5, 6, 3, 96, 96, 1, True, 1000, 16, 16, 1.0),
    (BF16, 1, 64, 8, 256, 128, 1, False, 1000, 2, 16, 1.0),
    (BF16, 3, 5, 1, 72, 16, 1, False, 1000, 2, 16, 1.0),
]


@pytest.mark.parametrize("case", GQA, ids=lambda c: f"{str(c[0])[6:]}-T{c[1]}-{c[2]}.{c[3]}-d{c[4]}-rot{c[5]}-ax{c[6]}")
@pytest.mark.parametrize("fused", [False, True])
def test_gqa(lib, case, fused):
    dtype, T, Hq, Hkv, d, rot, axes, inter, far, dcp, bs, scaling = case
    rng = np.random.default_rng(T * d + axes)
    nb = T // bs + 3
    inv = inv_freqs(rot // 2)
    pos = rng.integers(0, far, (axes, T))
    axis = np.sort(rng.integers(0, axes, rot // 2)).astype(np.int32)
    slot = slots(rng, T, dcp, nb, bs)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=torch.Generator().manual_seed(T)).to(dtype).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kp, vp = pools(dcp, (nb, Hkv, bs, d), dtype), pools(dcp, (nb, Hkv, bs, d), dtype)
    k_out = torch.empty((T, Hkv, d), dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lib.Layout(dcp, bs, 1)
    args = [torch.from_numpy(a).cuda() for a in (pos, inv, slot)]
    q_out = lib.rope_write_gqa(L, q, k, v, *args, kp, vp, nb, axis=torch.from_numpy(axis).cuda(),
                               interleaved=inter, scaling=scaling, k_out=k_out, err=err)
    assert err.item() == 0
    for got, src in ((q_out, q), (k_out, k)):
        y, mag = R.rotated(src.double().cpu().numpy(), pos, inv, axis, 0, inter, scaling)
        tol = R.rope_tol(dtype, y, mag)
        assert (np.abs(got.double().cpu().numpy() - y) <= tol).all()
        assert torch.equal(got[..., rot:], src[..., rot:])
    for r in range(dcp):
        mine = slot[r] >= 0
        rows = torch.from_numpy(np.nonzero(mine)[0]).cuda()
        assert torch.equal(stored(kp[r], slot[r][mine], bs, False), k_out[rows])
        assert torch.equal(stored(vp[r], slot[r][mine], bs, False), v[rows])
        # nothing else was written
        n = int(mine.sum()) * Hkv * d
        for p in (kp[r], vp[r]):
            assert int((p != 7.0).sum()) <= n and int((p == 7.0).sum()) >= p.numel() - n


# dtype, T, Hq, dim, rot, interleaved, dcp, bs
MLA = [
    (BF16, 33, 128, 576, 64, True, 8, 64),
    (BF16, 4, 16, 576, 64, False, 3, 16),
    (F32, 7, 3, 96, 32, True, 2, 16),
    (BF16, 1, 1, 64, 64, True, 1, 16),
]


@pytest.mark.parametrize("case", MLA, ids=str)
@pytest.mark.parametrize("place", ["out", "in", "strided"])
def test_mla(lib, case, place):
    dtype, T, Hq, dim, rot, inter, dcp, bs = case
    rng = np.random.default_rng(T + dim)
    nb = T // bs + 2
    inv, pos = inv_freqs(rot // 2), rng.integers(0, 1 << 18, (1, T))
    slot = slots(rng, T, dcp, nb, bs)
    gen = torch.Generator().manual_seed(T)
    q = torch.randn((T, Hq, dim), generator=gen).to(dtype).cuda()
    kv = torch.randn((T, dim), generator=gen).to(dtype).cuda()
    q0 = q.clone()
    if place == "strided":
        wide = torch.zeros((T, Hq + 1, dim), dtype=dtype, device="cuda")
        wide[:, :Hq] = q
        q = wide[:, :Hq]
        kv = torch.cat([kv, kv], 1)[:, :dim]
    p = pools(dcp, (nb, bs, dim), dtype)
    L = lib.Layout(dcp, bs, 1)
    args = [torch.from_numpy(a).cuda() for a in (pos[0], inv, slot)]
    got = lib.rope_write_mla(L, q, kv, *args, p, nb, interleaved=inter,
                             q_out=q if place == "in" else None)
    if place == "in":
        assert got.data_ptr() == q.data_ptr()
    at = dim - rot
    y, mag = R.rotated(q0.double().cpu().numpy(), pos, inv, None, at, inter)
    assert (np.abs(got.double().cpu().numpy() - y) <= R.rope_tol(dtype, y, mag)).all()
    assert torch.equal(got[..., :at], q0[..., :at])
    y, mag = R.rotated(kv.double().cpu().numpy(), pos, inv, None, at, inter)
    tol = R.rope_tol(dtype, y, mag)
    for r in range(dcp):
        mine = slot[r] >= 0
        rows = stored(p[r], slot[r][mine], bs, True).double().cpu().numpy()
        assert (np.abs(rows - y[mine]) <= tol[mine]).all()


def test_in_place_and_keys_only(lib):
    T, d = 10, 128
    L = lib.Layout(2, 16, 1)
    rng = np.random.default_rng(0)
    slot = torch.from_numpy(slots(rng, T, 2, 3, 16)).cuda()
    inv = torch.from_numpy(inv_freqs(32)).cuda()
    pos = torch.arange(T).cuda() * 1000
    q, k, v = (torch.randn((T, h, d), device="cuda").to(BF16) for h in (4, 2, 2))
    kp, vp = pools(2, (3, 2, 16, d), BF16), pools(2, (3, 2, 16, d), BF16)
    out = lib.rope_write_gqa(L, q, k, v, pos, inv, slot, kp, vp, 3)
    kp2, vp2 = pools(2, (3, 2, 16, d), BF16), pools(2, (3, 2, 16, d), BF16)
    assert lib.rope_write_gqa(L, None, k, v, pos, inv, slot, kp2, vp2, 3) is None
    for a, b in zip(kp + vp, kp2 + vp2):
        assert torch.equal(a, b)
    q2 = q.clone()
    assert lib.rope_write_gqa(L, q2, k, v, pos, inv, slot, kp2, vp2, 3, q_out=q2) is q2
    assert torch.equal(q2, out)


def test_bad_slots_and_axes_are_counted(lib):
    T, d, nb = 4, 64, 2
    L = lib.Layout(2, 16, 1)
    slot = torch.tensor([[0, -1, 32, -1], [-1, 5, -1, -2]]).cuda()
    inv = torch.from_numpy(inv_freqs(32)).cuda()
    k, v = (torch.randn((T, 1, d), device="cuda") for _ in range(2))
    kp, vp = pools(2, (nb, 1, 16, d), F32), pools(2, (nb, 1, 16, d), F32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.rope_write_gqa(L, None, k, v, torch.zeros(T, dtype=torch.int64).cuda(), inv, slot, kp, vp,
                       nb, err=err)
    assert err.item() == 2
    assert torch.equal(kp[0][0, 0, 0], k[0, 0]) and torch.equal(vp[1][0, 0, 5], v[1, 0])
    assert int((kp[0] != 7).sum()) <= d and int((kp[1] != 7).sum()) <= d
    err.zero_()
    axis = torch.zeros(32, dtype=torch.int32).cuda()
    axis[3], axis[9] = 2, -1
    lib.rope_write_gqa(L, None, k, v, torch.zeros((2, T), dtype=torch.int64).cuda(), inv, slot * 0 - 1,
                       kp, vp, nb, axis=axis, err=err)
    assert err.item() == 2


def test_refusals(lib):
    T, d, nb = 4, 64, 2
    L = lib.Layout(2, 16, 1)
    slot = torch.full((2, T), -1, dtype=torch.int64).cuda()
    inv = torch.from_numpy(inv_freqs(32)).cuda()
    pos = torch.zeros(T, dtype=torch.int64).cuda()
    q, k, v = (torch.randn((T, h, d), device="cuda").to(BF16) for h in (4, 2, 2))
    kp, vp = pools(2, (nb, 2, 16, d), BF16), pools(2, (nb, 2, 16, d), BF16)

    def call(q=q, k=k, v=v, pos=pos, inv=inv, slot=slot, kp=kp, vp=vp, nb=nb, **kw):
        with pytest.raises(lib.DcpError):
            lib.rope_write_gqa(L, q, k, v, pos, inv, slot, kp, vp, nb, **kw)

    call(q=q.float())
    call(q=q[:3])
    call(q=q[..., :32])
    call(k=k.half(), q=None, v=v.half())
    call(v=v[:, :1])
    call(v=v.float())
    call(pos=pos.int())
    call(pos=pos[:2])
    call(pos=torch.zeros((3, T), dtype=torch.int64).cuda())    # axes without `axis`
    call(inv=inv.double())
    call(inv=inv[:4])                                           # 8 rotated entries
    call(inv=torch.cat([inv, inv]))                             # more than a head has
    call(slot=slot[:1])
    call(slot=slot.int())
    call(kp=kp[:1])
    call(kp=[p.float() for p in kp])
    call(vp=[p[:, :1].contiguous() for p in vp])
    call(nb=3)
    call(k_out=torch.empty((T, 2, d), device="cuda"))
    call(q_out=torch.empty((T, 3, d), dtype=BF16, device="cuda"))
    call(axis=torch.zeros(31, dtype=torch.int32).cuda())
    call(q=torch.randn((T, 4, d + 4), device="cuda").to(BF16)[..., 4:])   # heads apart
    odd = torch.randn((T * 4 * d + 1), device="cuda").to(BF16)[1:].view(T, 4, d)
    call(q=odd)                                                 # not 16-byte aligned


@pytest.mark.parametrize("T,rot", [(1, 64), (1, 128), (40, 64), (40, 128), (3000, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_packed_inputs_rotated_in_place(lib, dtype, T, rot):
    """q_out and k_out that are q and k themselves, rotated in whole or in part; of a single
    token also when they are slices of one projection."""
    Hq, Hkv, d, dcp, bs = 4, 2, 128, 2, 16
    L, nb = lib.Layout(dcp, bs, 1), T // bs + 2
    rng = np.random.default_rng(T)
    slot = torch.from_numpy(slots(rng, T, dcp, nb, bs)).cuda()
    inv = torch.from_numpy(inv_freqs(rot // 2)).cuda()
    pos = torch.from_numpy(rng.integers(0, 1 << 20, T)).cuda()
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=torch.Generator().manual_seed(T)).to(dtype).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    if T > 1:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    want_k, p, p2 = torch.empty_like(k), *[pools(dcp, (nb, Hkv, bs, d), dtype) for _ in range(2)]
    vp, vp2 = (pools(dcp, (nb, Hkv, bs, d), dtype) for _ in range(2))
    want = lib.rope_write_gqa(L, q, k, v, pos, inv, slot, p, vp, nb, k_out=want_k)
    lib.rope_write_gqa(L, q, k, v, pos, inv, slot, p2, vp2, nb, q_out=q, k_out=k)
    assert torch.equal(q, want) and torch.equal(k, want_k)
    for a, b in zip(p + vp, p2 + vp2):
        assert torch.equal(a, b)


def test_outputs_over_inputs_are_refused(lib):
    T, d, nb = 4, 64, 2
    L = lib.Layout(1, 16, 1)
    slot = torch.full((1, T), -1, dtype=torch.int64).cuda()
    inv, pos = torch.from_numpy(inv_freqs(32)).cuda(), torch.zeros(T, dtype=torch.int64).cuda()
    x = torch.randn((T, 6, d), device="cuda")
    q, k, v = x.split([2, 2, 2], 1)
    p = pools(1, (nb, 2, 16, d), F32)
    over = x.view(-1)[:T * 2 * d].view(T, 2, d)           # packed, over the projection
    other = torch.empty((T, 2, d), device="cuda")
    for q_out, k_out in ((over, None), (None, over), (other, other)):
        with pytest.raises(lib.DcpError):
            lib.rope_write_gqa(L, q, k, v, pos, inv, slot, p, p, nb, q_out=q_out, k_out=k_out)


def test_the_angle_of_far_positions(lib):
    """Cosines and sines as they are (pairs (1, 0) in 32 bits), for positions up to 2^32: the angle
    is exact to 2^-31 of a turn, which is 2 pi 2^-31 of their value at most; sincospi and the two
    roundings around it stay within 3 ulp, 3 * 2^-23 of the value."""
    T, rot = 4096, 128
    rng = np.random.default_rng(11)
    pos = np.concatenate([rng.integers(0, 1 << 32, T - 96), rng.integers(-(1 << 32), 0, 32),
                          np.arange(32), (1 << 32) - 1 - np.arange(32)])
    inv = inv_freqs(rot // 2)
    inv[1:4] = np.float32(np.pi), np.float32(np.pi / 4), np.float32(2 * np.pi)
    k = torch.zeros((T, 1, rot), device="cuda")
    k[..., :rot // 2] = 1.0
    wide = torch.zeros((T, 1, rot + 16), device="cuda")     # rotated in part: in place by itself
    wide[..., :rot // 2] = 1.0
    slot = torch.full((1, T), -1, dtype=torch.int64, device="cuda")
    L, out = lib.Layout(1, 16, 1), torch.empty_like(k)
    args = [torch.from_numpy(a).cuda() for a in (pos, inv)]
    p, pw = pools(1, (1, 1, 16, rot), F32), pools(1, (1, 1, 16, rot + 16), F32)
    lib.rope_write_gqa(L, None, k, k, *args, slot, p, p, 1, k_out=out)
    lib.rope_write_gqa(L, wide, wide.clone(), wide.clone(), *args, slot, pw, pw, 1, q_out=wide)
    x = np.zeros((T, 1, rot))
    x[..., :rot // 2] = 1.0
    y, _ = R.rotated(x, pos[None], inv, None, 0, False)
    tol = 2 * np.pi * 2.0 ** -31 + 3 * 2.0 ** -23 * np.abs(y)
    for got in (out, wide[..., :rot]):
        off = np.abs(got.double().cpu().numpy() - y)
        assert (off <= tol).all(), (off / tol).max()
    assert (wide[..., rot:] == 0).all()


# dtype, T, Hq, Hkv, d, rot, interleaved, dcp, bs
MANY = [
    (BF16, 6001, 3, 1, 64, 64, False, 8, 16),
    (BF16, 5000, 2, 2, 128, 32, True, 2, 64),
    (F32, 701, 64, 8, 128, 128, False, 3, 16),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{str(c[0])[6:]}-T{c[1]}-{c[2]}.{c[3]}-d{c[4]}")
def test_many_tokens(lib, case):
    """More items than the card holds CTAs, so that each goes through several: stages and tables
    are used again, and what comes next is loaded ahead."""
    dtype, T, Hq, Hkv, d, rot, inter, dcp, bs = case
    row = d * (4 if dtype == F32 else 2)
    parts = -(-(Hq + 2 * Hkv) // min(Hq + 2 * Hkv, 16384 // row))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T * parts > 2 * 8 * sms or (parts > 1 and T * parts > 2 * 6 * sms)
    rng = np.random.default_rng(T)
    nb, axes = T // bs + 3, 3
    inv, pos = inv_freqs(rot // 2), rng.integers(0, 1 << 20, (axes, T))
    axis = np.sort(rng.integers(0, axes, rot // 2)).astype(np.int32)
    slot = slots(rng, T, dcp, nb, bs)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=torch.Generator().manual_seed(T)).to(dtype).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    kp, vp = pools(dcp, (nb, Hkv, bs, d), dtype), pools(dcp, (nb, Hkv, bs, d), dtype)
    k_out = torch.empty((T, Hkv, d), dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [torch.from_numpy(a).cuda() for a in (pos, inv, slot)]
    q_out = lib.rope_write_gqa(lib.Layout(dcp, bs, 1), q, k, v, *args, kp, vp, nb,
                               axis=torch.from_numpy(axis).cuda(), interleaved=inter, k_out=k_out,
                               err=err)
    assert err.item() == 0
    for got, src in ((q_out, q), (k_out, k)):
        y, mag = R.rotated(src.double().cpu().numpy(), pos, inv, axis, 0, inter)
        assert (np.abs(got.double().cpu().numpy() - y) <= R.rope_tol(dtype, y, mag)).all()
        assert torch.equal(got[..., rot:], src[..., rot:])
    for r in range(dcp):
        mine = slot[r] >= 0
        rows = torch.from_numpy(np.nonzero(mine)[0]).cuda()
        assert torch.equal(stored(kp[r], slot[r][mine], bs, False), k_out[rows])
        assert torch.equal(stored(vp[r], slot[r][mine], bs, False), v[rows])
        n = int(mine.sum()) * Hkv * d
        for p in (kp[r], vp[r]):
            assert int((p == 7.0).sum()) >= p.numel() - n


def test_many_latent_rows(lib):
    T, Hq, dim, rot, dcp, bs = 1501, 20, 576, 64, 4, 64     # two items a token
    rng = np.random.default_rng(T)
    nb = T // bs + 2
    inv, pos = inv_freqs(rot // 2), rng.integers(0, 1 << 18, (1, T))
    slot = slots(rng, T, dcp, nb, bs)
    gen = torch.Generator().manual_seed(T)
    q = torch.randn((T, Hq, dim), generator=gen).to(BF16).cuda()
    kv = torch.randn((T, dim), generator=gen).to(BF16).cuda()
    p = pools(dcp, (nb, bs, dim), BF16)
    args = [torch.from_numpy(a).cuda() for a in (pos[0], inv, slot)]
    got = lib.rope_write_mla(lib.Layout(dcp, bs, 1), q, kv, *args, p, nb)
    at = dim - rot
    y, mag = R.rotated(q.double().cpu().numpy(), pos, inv, None, at, True)
    assert (np.abs(got.double().cpu().numpy() - y) <= R.rope_tol(BF16, y, mag)).all()
    assert torch.equal(got[..., :at], q[..., :at])
    y, mag = R.rotated(kv.double().cpu().numpy(), pos, inv, None, at, True)
    tol = R.rope_tol(BF16, y, mag)
    for r in range(dcp):
        mine = slot[r] >= 0
        rows = stored(p[r], slot[r][mine], bs, True).double().cpu().numpy()
        assert (np.abs(rows - y[mine]) <= tol[mine]).all()
