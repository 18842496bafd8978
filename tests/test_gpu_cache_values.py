"""Values and scales of cache_write that its other tests do not meet, codes and scales bit for bit
(oracle/cache.py)."""
import numpy as np
import pytest
import torch

from test_gpu_cache import Model

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("N", [1, 5, 40])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_infinities_without_finite_values(fa, fmt, N, dt):
    """Infinities alone, beside zeros, beside NaN, in a page of zeros, and in pages that then get values."""
    B, H, d, page = 3, 2, 64, 16
    m = Model(fa, 24, H, page, d, fmt, B, 7)
    zero = torch.zeros((B, H, N, d), dtype=dt, device="cuda")
    x, y = zero.clone(), zero.clone()
    x[0], x[1, 0, 0, :3] = INF, torch.tensor([-INF, INF, NAN])
    x[2, 1, N - 1, 60:] = torch.tensor([NAN, -INF, -0.0, INF])
    y[0], y[1], y[2] = NAN, -INF, 0.0
    m.write(fa, x, y, [0, 3, 16], None)
    m.same()
    top = 0x7e if fmt == "e4m3" else 127
    assert (m.codes["k"][int(m.table[0, 0]), 0, 0] == top).all() and m.scale["k"][int(m.table[0, 0]), 0] == 0
    m.write(fa, zero, x, [N, 3 + N, 16 + N], None)
    m.same()
    one = zero.clone()
    one[:, :, 0, 5] = 3.0
    m.write(fa, one, one, [2 * N, 3 + 2 * N, 16 + 2 * N], None)
    m.same()
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("N", [1, 5, 9, 40])
def test_pages_whose_scale_is_no_power_of_two(fa, fmt, N):
    """Tokens behind those of a pool filled elsewhere: its scale becomes the next power of two and every
    writer forms the same codes, also of values that fall between two of them."""
    B, H, d, page = 3, 2, 64, 16
    m = Model(fa, 24, H, page, d, fmt, B, 6)
    for n, s in (("k", 0.3125), ("v", 0.75)):
        m.scale[n][:] = s * 2.0 ** np.arange(-2, 0)      # few bits: moved codes are exact before their rounding
        getattr(m.cache, n + "_scale").copy_(torch.from_numpy(m.scale[n]).float())
    g = torch.Generator().manual_seed(N)
    x = torch.randint(-600, 601, (2, B, H, N, d), generator=g).to(torch.bfloat16).cuda() / 64   # ties among them
    m.write(fa, x[0], x[1], [1, 7, 15], None)
    m.same()
    m.write(fa, 8 * x[1], x[0], [1 + N, 7 + N, 15 + N], None)
    m.same()
    assert fa.device_status() == fa.FA_OK


def test_writers_agree_whatever_the_scale(fa):
    """The same token by the writer of few and by that of pages."""
    codes = []
    for N in (1, 12):
        cache = fa.KVCache.empty(2, 1, 64, dtype=torch.int8, page_size=16)
        cache.k_scale.fill_(0.3)
        cache.v_scale.fill_(0.7)
        k, v = torch.zeros((2, 1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
        k[0, 0, 0] = torch.arange(64, device="cuda") * -0.75 - 2.25 - 6   # (x * (1 / 0.3)) at half-way points
        v[0, 0, 0] = torch.arange(64, device="cuda") * -0.4375 - 1.75
        one = torch.ones(1, dtype=torch.int32, device="cuda")
        fa.cache_write(cache, k, v, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), one)
        codes.append([t[1, 0, 1].clone() for t in (cache.k, cache.v)] + [cache.k_scale[1].clone(), cache.v_scale[1].clone()])
    assert all(torch.equal(a, b) for a, b in zip(*codes))
