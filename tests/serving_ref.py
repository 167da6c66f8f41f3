"""Plain 64-bit implementations of the calls around the decode step (drafted
token trees, rotary positions, pages, compaction) and the bounds the GPU tests
hold them to.  numpy on the host.
"""
from __future__ import annotations

import numpy as np
import torch


# largest relative rounding error of a type: half a step
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def place(x, dcp, bs, I):
    """(rank, virtual block, place in the rank's page) of token x."""
    vb, off = divmod(int(x), bs * dcp)
    run = off // I
    return run % dcp, vb, run // dcp * I + off % I


def random_tables(rng, lens, dcp, bs, spare=3, max_vb=None):
    """Block tables [dcp, B, VB] over pages placed anywhere, and the pages' number."""
    vbs = bs * dcp
    n = [-(-L // vbs) for L in lens]
    VB, nb = max(1, max(n), max_vb or 0), sum(n) + spare
    bt = np.full((dcp, len(lens), VB), -1, dtype=np.int32)
    for r in range(dcp):
        ids = rng.permutation(nb)
        at = 0
        for b, k in enumerate(n):
            bt[r, b, :k] = ids[at:at + k]
            at += k
    return bt, nb


def gather(pools, bt, b, positions, dcp, bs, I):
    """float64 rows [H, len(positions), d] of request b from pools [dcp, nb, H, bs, d]."""
    out = np.empty((pools.shape[2], len(positions), pools.shape[4]))
    for i, x in enumerate(positions):
        r, vb, loc = place(x, dcp, bs, I)
        out[:, i] = pools[r, bt[r, b, vb], :, loc]
    return out


def attend(q, k, v, seen, scale, sink=None):
    """o, lse, sum of weight * |v| and sum |q||k| * scale (for the bounds), all in
    64 bits: q [R, d], k and v [L, d], seen [R, L]."""
    R, L = seen.shape
    with np.errstate(all="ignore"):
        s = np.where(seen, (q @ np.where(np.isfinite(k), k, 0).T) * scale, -np.inf)
    if sink is not None:
        s = np.concatenate([s, np.full((R, 1), sink)], 1)
    top = s.max(1, initial=-np.inf)
    base = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - base[:, None])
    tot = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = base + np.log(tot)
    w = e[:, :L] / np.where(tot == 0, 1, tot)[:, None]
    vv = np.where(np.isfinite(v), v, 0)
    size = (np.abs(q) @ np.abs(np.where(np.isfinite(k), k, 0)).T * scale)
    size = np.where(seen, size, 0).max(1, initial=0.0)
    return w @ vv, lse, w @ np.abs(vv), size


def attend_tol(dtype, out_dtype, o, wabs, size, d, L):
    """Bound on the output error of a kernel that multiplies exactly, sums in 32
    bits, takes exp2 with 2 ulp and, for bf16 inputs, rounds the probabilities
    to bf16; rounded once to out_dtype.

    A score is off by delta <= (d + 4) 2^-24 size (a sum of d products whose
    magnitudes sum to size, then scaled), so a weight is off by 2 delta + 2^-21
    relatively, the sums over L tokens by L 2^-24, and bf16 probabilities by
    2^-8; each of these acts on terms that sum to wabs.
    """
    delta = (d + 4) * 2.0 ** -24 * size
    rel = 2 * delta + 2.0 ** -21 + 2 * L * 2.0 ** -24
    if dtype == torch.bfloat16:
        rel = rel + HALF[torch.bfloat16]
    return HALF[out_dtype] * np.abs(o) + (rel[:, None] * wabs) * 1.01 + 1e-30


def lse_tol(lse, size, d, L):
    """The same for the LSE: the score's error, the sum's and the logarithm's."""
    return (d + 4) * 2.0 ** -24 * size + L * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * np.abs(
        np.where(np.isfinite(lse), lse, 0))


def rotated(x, pos, inv_freq, axis, at, interleaved, scaling=1.0):
    """x [T, ..., d] float64 with rot entries from `at` on rotated; also the
    magnitude |a| + |b| that each rotated entry's bound goes by."""
    rot = 2 * len(inv_freq)
    turns = np.empty((x.shape[0], rot // 2))
    for i in range(rot // 2):
        ax = 0 if axis is None else int(axis[i])
        # exact integer positions times the float32 frequency: long double keeps the fraction
        a = pos[ax].astype(np.longdouble) * np.longdouble(np.float32(inv_freq[i]))
        turns[:, i] = np.float64(np.fmod(a, np.longdouble(2) * np.arccos(np.longdouble(-1))))
    c, s = np.cos(turns) * scaling, np.sin(turns) * scaling
    shape = (x.shape[0],) + (1,) * (x.ndim - 2) + (rot // 2,)
    c, s = c.reshape(shape), s.reshape(shape)
    y, mag = x.copy(), np.zeros_like(x)
    r = x[..., at:at + rot]
    if interleaved:
        ia, ib = np.arange(0, rot, 2), np.arange(1, rot, 2)
    else:
        ia, ib = np.arange(rot // 2), np.arange(rot // 2, rot)
    a, b = r[..., ia], r[..., ib]
    y[..., at + ia] = a * c - b * s
    y[..., at + ib] = b * c + a * s
    mag[..., at + ia] = mag[..., at + ib] = (np.abs(a) + np.abs(b)) * abs(scaling)
    return y, mag


def rope_tol(dtype, y, mag):
    """cos and sin are off by 2^-31 of a turn (4e-9), 2 ulp of sincospi and the
    scaling's rounding (2^-22 together), the products and the sum by 2^-23 more;
    then one rounding."""
    return HALF[dtype] * np.abs(y) + 2.0 ** -21 * mag + 1e-30


class PageModel:
    """The pages' life, one page at a time."""

    def __init__(self, dcp, bs, I, B, VB, nb, shared):
        self.dcp, self.bs, self.I, self.VB, self.nb, self.shared = dcp, bs, I, VB, nb, shared
        self.tables = 1 if shared else dcp
        self.bt = np.full((self.tables, B, VB), -1, dtype=np.int32)
        self.seq = np.zeros(B, dtype=np.int32)
        self.ref = np.zeros((self.tables, nb), dtype=np.int32)
        self.err = 0

    def bits(self):
        words = (self.nb + 31) // 32
        out = np.zeros((self.tables, words), dtype=np.uint32)
        for t in range(self.tables):
            for i in range(self.nb):
                if self.ref[t, i] == 0:
                    out[t, i // 32] |= np.uint32(1 << (i % 32))
        return out.view(np.int32)

    def blocks(self, n):
        return -(-n // (self.bs * self.dcp))

    def open(self, n, t):
        """(open page's block, its tokens) of a length on table t, or None if none is open."""
        vbs = self.bs * self.dcp
        if n % vbs == 0:
            return None
        if self.shared:
            return n // vbs, n % vbs
        have = sum(place(x, self.dcp, self.bs, self.I)[0] == t for x in range(n // vbs * vbs, n))
        return None if have == self.bs else (n // vbs, have)

    def take(self, t):
        free = np.nonzero(self.ref[t] == 0)[0]
        if len(free) == 0:
            self.err += 1
            return -1
        self.ref[t, free[0]] = 1
        return int(free[0])

    def resize(self, req, new):
        n = len(req)
        src = np.full((self.tables, n), -1, dtype=np.int32)
        dst = src.copy()
        first = {}
        for i, c in enumerate(req):
            if 0 <= c < len(self.seq):
                first.setdefault(int(c), i)
        ok = [0 <= c < len(self.seq) and first[int(c)] == i and L >= 0 and
              self.blocks(L) <= self.VB for i, (c, L) in enumerate(zip(req, new))]
        self.err += n - sum(ok)
        for t in range(self.tables):
            for i in range(n):
                if ok[i]:
                    for v in range(self.blocks(new[i]), self.blocks(self.seq[req[i]])):
                        self.ref[t, self.bt[t, req[i], v]] -= 1
                        self.bt[t, req[i], v] = -1
            before = self.ref[t].copy()
            later = []
            for i in range(n):
                if not ok[i]:
                    continue
                c, old = int(req[i]), int(self.seq[req[i]])
                at = self.open(min(old, int(new[i])), t)
                if at and before[self.bt[t, c, at[0]]] > 1:
                    page = self.bt[t, c, at[0]]
                    later.append(page)
                    self.bt[t, c, at[0]] = self.take(t)
                    if at[1] and self.bt[t, c, at[0]] >= 0:
                        src[t, i], dst[t, i] = page, self.bt[t, c, at[0]]
                for v in range(self.blocks(old), self.blocks(new[i])):
                    self.bt[t, c, v] = self.take(t)
            for page in later:
                self.ref[t, page] -= 1
        for i in range(n):
            if ok[i]:
                self.seq[req[i]] = new[i]
        return src, dst

    def fork(self, parent, child):
        n = len(parent)
        src = np.full((self.tables, n), -1, dtype=np.int32)
        dst = src.copy()
        first, B = {}, len(self.seq)
        for i, c in enumerate(child):
            if 0 <= c < B:
                first.setdefault(int(c), i)
        ok = [0 <= c < B and first[int(c)] == i and 0 <= p < B and int(p) not in first
              for i, (p, c) in enumerate(zip(parent, child))]
        self.err += n - sum(ok)
        for t in range(self.tables):
            for i in range(n):
                if ok[i]:
                    for v in range(self.blocks(self.seq[child[i]])):
                        self.ref[t, self.bt[t, child[i], v]] -= 1
                        self.bt[t, child[i], v] = -1
            for i in range(n):
                if not ok[i]:
                    continue
                p, c, L = int(parent[i]), int(child[i]), int(self.seq[parent[i]])
                at = self.open(L, t)
                if at:
                    self.bt[t, c, at[0]] = self.take(t)
                    if at[1] and self.bt[t, c, at[0]] >= 0:
                        src[t, i], dst[t, i] = self.bt[t, p, at[0]], self.bt[t, c, at[0]]
            for i in range(n):
                if not ok[i]:
                    continue
                p, c, L = int(parent[i]), int(child[i]), int(self.seq[parent[i]])
                at = self.open(L, t)
                for v in range(self.blocks(L)):
                    if not at or v != at[0]:
                        self.bt[t, c, v] = self.bt[t, p, v]
                        self.ref[t, self.bt[t, p, v]] += 1
        for i in range(n):
            if ok[i]:
                self.seq[child[i]] = self.seq[parent[i]]
        return src, dst
