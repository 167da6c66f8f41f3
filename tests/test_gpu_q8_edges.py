"""The 8-bit cache at its edges."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def test_a_page_beyond_31_bits(lib):
    """One page of more than 2^31 numbers, written by one call: what lies behind 2^31 comes back."""
    bs, d = (1 << 23) + 32, 256
    N = bs - 7
    L = lib.Layout(1, bs, 1)
    kv = lib.PagedKV8.new(L, 1, 1, d, torch.zeros((1, 1, 1), dtype=torch.int32, device="cuda"))
    x = torch.randn((N, 1, d), dtype=BF16, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    err = i32([0])
    lib.q8_append_gqa(L, x, x, kv, i32([0, N]), i32([0]), err=err)
    assert err.item() == 0
    pos = torch.tensor([0, 1, 1 << 22, (1 << 23) - 1, 1 << 23, (1 << 23) + 5, N - 1], device="cuda")
    req = torch.zeros(len(pos), dtype=torch.int32, device="cuda")

    # the e4m3 number nearest to x / scale, times the scale
    scale = 2.0 ** np.ceil(np.log2(x.abs().max().item() / 448))
    want = (x[pos].float() / scale).to(E4M3).float() * scale
    for got in lib.q8_gather_gqa(L, kv, req, pos, dtype=F32):
        assert torch.equal(got, want)


def test_bad_requests_leave_the_cache_alone(lib):
    """Requests whose rows leave those given, in front or behind: nothing of them is written, and
    what the others write is as ever."""
    from tests.test_gpu_q8_cache import Cache, rows

    rng = np.random.default_rng(15)
    c = Cache(lib, rng, 2, 64, 2, 16, 1, [200] * 6)
    k, v = rows(rng, 60, 2, 64, BF16, True)
    start, ctx = [-4, 10, 10, 30, 40, 45, 70], [9, 0, 0, 0, 3, 0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(k, v, start, ctx, err=err)
    c.model(k, v, start, ctx, skip=(0, 5))
    c.check()
    assert err.item() == 2
