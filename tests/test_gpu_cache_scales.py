"""Attention over pages whose scales are not powers of two (a pool filled elsewhere; cache_write makes powers of two).

The kernels take log2 and the inverse of V's scale by the fast functions: off by 2 ulp at most, which for scales
between 2^-16 and 1 (|log2| below 16, ulp 2^-20) is 2^-19 in the exponent and 2^-22 of the inverse: each weight, in the
product and in the sum, by less than 2^-19 of itself. check_batch's bound leaves 2^-12 A for O beside its own rounding of
the weights, and its 2^-17 E for the LSE (E, the largest sum |q k| scale of a row, is above 4 here: 2^-15) more than that.
"""
import pytest
import torch

from test_gpu_cache import check_batch, queries, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,G,N,B,L", [(128, 16, 1, 1, 5, 900), (64, 64, 4, 2, 3, 3000), (128, 32, 4, 4, 4, 700), (64, 16, 4, 12, 300, 130),
                                            (128, 64, 1, 100, 2, 2100), (128, 16, 2, 100, 640, 130), (64, 128, 4, 90, 2, 6000)])
def test_attention(fa, d, page, G, N, B, L, fmt):
    W = -(-L // page)
    cache = random_cache(fa, 2 * W + 1, 2, page, d, fmt, seed=60)
    g = torch.Generator(device="cuda").manual_seed(61)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(1 + torch.rand(s.shape, generator=g, device="cuda"))
    table = torch.randint(0, 2 * W + 1, (B, W), generator=torch.Generator().manual_seed(62), dtype=torch.int32).cuda()
    lens = [L - 37 * (b % 3) for b in range(B)]
    check_batch(fa, queries(B, 2 * G, N, d, "bf16", 63), cache, table, lens, [N] * B)
