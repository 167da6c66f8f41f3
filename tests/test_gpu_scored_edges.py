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
