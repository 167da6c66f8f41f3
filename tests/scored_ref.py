"""Plain 64-bit implementations of the 8-bit cache and of scored decode
attention, and the bounds the GPU tests hold them to.  numpy on the host.
"""
from __future__ import annotations

import numpy as np
import torch

from tests.serving_ref import HALF, place

E4M3 = torch.float8_e4m3fn


def nearest8(y):
    """The e4m3 number nearest to y, ties to even; beyond +-448 those, NaN stays."""
    y = np.clip(np.asarray(y, np.float64), -448.0, 448.0)
    size = np.maximum(np.abs(np.nan_to_num(y)), 2.0 ** -6)
    step = np.ldexp(1.0, np.frexp(size)[1] - 4)      # 8 steps to a power of two
    return np.rint(y / step) * step


def need(top):
    """Smallest power of two s >= 2^-60 with top / s <= 448."""
    s = np.ldexp(1.0, -60)
    while top / s > 448.0:
        s *= 2
    return s


def position(vb, r, loc, dcp, bs, I):
    return vb * bs * dcp + (loc // I * dcp + r) * I + loc % I


def append(pool, scale, x, table, ctx, dcp, bs, I):
    """Rows x [T, H, d] of one request at positions ctx .. into pool [dcp, nb, H, bs, d] and
    scale [dcp, nb, H] (float64, in place), page by page."""
    pages = {}
    for t in range(x.shape[0]):
        r, vb, loc = place(ctx + t, dcp, bs, I)
        pages.setdefault((r, vb), []).append((loc, t))
    nb = pool.shape[1]
    for (r, vb), places in pages.items():
        page = table[r][vb]
        if not 0 <= page < nb:
            continue
        locs = [p for p, _ in places]
        for h in range(x.shape[1]):
            rows = np.stack([x[t, h] for _, t in places])
            top = np.abs(np.where(np.isfinite(rows), rows, 0.0)).max()
            old = scale[r, page, h]
            if 0 in locs or not (np.isfinite(old) and old > 0):
                old = 0.0
            new = max(old, need(top))
            if 0 < old < new:
                for p in set(range(bs)) - set(locs):
                    pool[r, page, h, p] = nearest8(pool[r, page, h, p] * old / new)
            pool[r, page, h, locs] = nearest8(rows / new)
            scale[r, page, h] = new


def as_e4m3(x):
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(E4M3)


def seen_mask(n, window, prefix, first):
    """Which of the tokens [0, n) are seen."""
    x = np.arange(n)
    lo = max(first, 0)
    seen = x >= lo
    if window:
        seen &= (x >= n - window) | (x < lo + prefix)
    return seen


def attend(dtype, out_dtype, q, k, v, x, n, scale, cap=0.0, slope=0.0, sink=None):
    """o [d], lse, and bounds on the error of each, for one query head q [d] over the seen
    tokens (k, v [L, d] at positions x), all in 64 bits.

    The bounds are those of a kernel that multiplies exactly and sums in 32 bits:
    a score's d products, whose sizes sum to `size`, are off by (d + 4) 2^-24
    size; the cap's tanh by 2 ulp and its input by one rounding more, the bias
    by its product, the difference and the change to base 2: together at most
    2^-21 (|t| + |bias|).  A weight is off by as much as its score, relatively,
    and by exp2's 2 ulp; the sums by 2 L 2^-24.  16-bit and 8-bit caches round
    the weights for the product with the values, bf16 by 2^-8, fp16 (for 8 bits)
    by 2^-11 and by 2^-31 of the largest weight at most."""
    L, d = k.shape
    if L == 0:
        return (np.zeros(d), -np.inf if sink is None else sink, np.full(d, 1e-30),
                1e-30 if sink is None else abs(sink) * 2.0 ** -22)
    size = np.abs(k) @ np.abs(q) * abs(scale)
    t = k @ q * scale
    if cap:
        t = cap * np.tanh(t / cap)
    bias = slope * (n - 1 - x)
    off = (d + 4) * 2.0 ** -24 * size + 2.0 ** -21 * (np.abs(t) + np.abs(bias))
    e = t - bias
    all_e = e if sink is None else np.append(e, sink)
    top = all_e.max()
    lse = top + np.log(np.exp(all_e - top).sum())
    w = np.exp(e - lse)
    o = w @ v
    wabs = w @ np.abs(v)
    shift = w @ off
    rel = 2.0 ** -20 + 2 * L * 2.0 ** -24
    if dtype == torch.bfloat16:
        rel += HALF[torch.bfloat16]
    tol = HALF[out_dtype] * np.abs(o) + 1.05 * ((w * off) @ np.abs(v) + (shift + rel) * wabs) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -31 * w.max() * np.abs(v).sum(0)
    return o, lse, tol, shift * 1.05 + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * abs(lse)
