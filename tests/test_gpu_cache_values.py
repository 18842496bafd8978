"""Values and scales of cache_write that its other tests do not meet, codes and scales bit for bit
(oracle/cache.py)."""
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
