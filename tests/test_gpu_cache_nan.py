"""NaN codes in V, wherever they stand: O is NaN in the channels in which a row sees one, and
nowhere else; the LSE does not depend on V. Every kernel, by the rows of a (sequence, cache head):
up to 8, 16, 64, 128 and 256 of them in a unit (fa_cache_attn.cu's attn_plan).
"""
import pytest
import torch

from test_gpu_cache import filled, queries

pytestmark = pytest.mark.gpu

# G, N, B, d: rows of a unit 8; 16; groups of 16; a tile with its rows twice; one tile; a unit of two tiles
KERNELS = [(1, 3, 2, 64), (2, 3, 2, 128), (2, 8, 2, 128), (2, 12, 2, 64), (2, 12, 300, 64), (3, 12, 300, 128), (1, 100, 2, 128),
           (2, 60, 2, 64), (2, 100, 640, 64), (2, 100, 640, 128)]


def planted(fa, G, N, B, d, page, at, causal=True, split=True, L=None):
    """O and LSE of a cache without NaN and of the same with NaN in V at `at`: (sequence of the first two,
    head, token, channel, scale of the token's page or None for its own), and the rows that see them."""
    L = N + 90 if L is None else L
    m = filled(fa, 2, 2, page, d, "e4m3", [L, L], seed=40)
    table = torch.cat([m.table, m.table[:1].expand(B - 2, -1)]).cuda()
    q = queries(B, 2 * G, N, d, "bf16", 41)
    n = torch.full((B,), L, dtype=torch.int32, device="cuda")
    codes = m.cache.v.view(torch.uint8)
    for b, h, t, c, s in at:
        p = int(m.table[b, t // page])
        codes[p, h, t % page, c] = 0
        if s is not None:
            m.cache.v_scale[p, h] = s
    want = fa.cache_attention(q, m.cache, table, n, causal=causal, split=split)
    hit = torch.zeros_like(want[0], dtype=torch.bool)
    for b, h, t, c, _ in at:
        codes[int(m.table[b, t // page]), h, t % page, c] = 0x7f if t % 2 else 0xff
        first = max(0, t - (L - N)) if causal else 0
        for i in [b] + ([] if b else list(range(2, B))):
            hit[i, h * G:(h + 1) * G, first:, c] = True
    got = fa.cache_attention(q, m.cache, table, n, causal=causal, split=split)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    return want, got, hit


def check(want, got, hit):
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    assert torch.equal(torch.isnan(got[0]), hit)
    assert torch.equal(got[0][~hit], want[0][~hit]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -101, 2.0 ** -4])
@pytest.mark.parametrize("G,N,B,d", KERNELS)
def test_nan_that_every_row_sees(fa, G, N, B, d, scale):
    """On a page of zeros (cache_write makes one of a page whose finite values are all zero) as on any other."""
    check(*planted(fa, G, N, B, d, 16, [(1, 1, 3, 5, scale), (0, 0, 20, d - 1, scale)]))


@pytest.mark.parametrize("scale", [0.0, None])
@pytest.mark.parametrize("G,N,B,d", KERNELS)
def test_nan_that_some_rows_see(fa, G, N, B, d, scale):
    """Tokens from the first row's own to the last row's, several channels, beside the edge of what rows see."""
    L = N + 90
    at = [(1, 1, L - N + i, c, scale) for i, c in ((N // 2, 7), (N - 1, 0), (N // 3, d - 1), (0, 33), (N // 2, 8))]
    check(*planted(fa, G, N, B, d, 16, at + [(0, 0, L - 1, 15, scale), (1, 0, 2, 3, scale)]))


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,N,d", [(4, 2, 64), (2, 8, 128), (4, 12, 64), (2, 60, 128), (4, 100, 64), (4, 100, 128)])
def test_nan_in_units_that_are_cut(fa, G, N, d, causal, split):
    L = 6000
    at = [(1, 1, t, c, s) for t, c, s in ((5, 1, None), (2999, 2, 0.0), (L - N + N // 2, 3, None), (L - 1, 4, 0.0), (L - 1, 63, 0.0))]
    check(*planted(fa, G, N, 2, d, 64, at, causal=causal, split=split, L=L))


def test_nan_beside_a_page_that_was_not_read(fa):
    """A bad page's keys are masked; a NaN of the page beside it, in the same tile, is seen by every row."""
    L, G = 4000, 2
    for N in (2, 8, 60):
        m = filled(fa, 1, 1, 16, 64, "e4m3", [L], seed=42)
        table, q = m.table.cuda(), queries(1, G, N, 64, "bf16", 43)
        bad = table.clone()
        bad[0, 9] = -1
        n = torch.tensor([L], dtype=torch.int32, device="cuda")
        m.cache.v.view(torch.uint8)[int(table[0, 9])] = 0x7f      # what lies in the ring before is anything
        want = fa.cache_attention(q, m.cache, bad, n)
        m.cache.v.view(torch.uint8)[int(table[0, 8]), 0, 5, 11] = 0x7f
        got = fa.cache_attention(q, m.cache, bad, n)
        torch.cuda.synchronize()
        assert fa.device_status() == fa.FA_ERR_BAD_PAGE
        assert torch.isfinite(want[0]).all() and torch.isnan(got[0][..., 11]).all()
        keep = [c for c in range(64) if c != 11]
        assert torch.equal(got[0][..., keep], want[0][..., keep]) and torch.equal(got[1], want[1])
