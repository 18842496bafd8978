"""The paged 8-bit cache and the attention over it against their fp64 definitions
(oracle/cache.py).

Codes and scales have to be equal bit for bit: a scale is a power of two, so x / s is exact and
its rounding has one answer. A value read back is off by half a step of its type.

Attention's bounds, from what the kernel rounds (A = sum p |v|, E = sum |q k| scale, both of the
row): the weights are rounded to fp16 (2^-12 each way, in the numerator alone: 2^-12 A) or
flushed 2^-32 below the largest; a score is an fp32 sum of at most 128 exact products (128 *
2^-24 E = 2^-17 E at the very most) whose error moves every weight by that part, numerator and sum
both, plus 2^-21 for the exponential and 2^-21 for fp32's argument near 2^5; sums of n weights
add n 2^-24 at most (pairs of chunks: far less). O is rounded once: half a step. So
|dO| <= eps/2 |O| + A (2^-11 + 2 (2^-17 E + 2^-20)), |dLSE| <= 2^-17 E + 2^-19 + 2^-22 |LSE|.
"""
import numpy as np
import pytest
import torch

from _util import f64
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


class Model:
    """A cache on the GPU and the same one by the oracle."""

    def __init__(self, fa, P, H, page, d, fmt, B, W, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.page = fmt, page
        self.codes = {n: torch.randint(0, 255, (P, H, page, d), generator=g, dtype=torch.int32).to(torch.uint8) for n in "kv"}
        for n in "kv":  # leftovers of other sequences, NaN codes among them
            self.codes[n][:, :, ::3, ::5] = 0x7f
        self.scale = {n: torch.exp2(torch.randint(-8, 3, (P, H), generator=g).float()) for n in "kv"}
        self.table = torch.randperm(P, generator=g)[:B * W].reshape(B, W).to(torch.int32)
        dev = [self.codes[n].cuda().view(CODE[fmt]) for n in "kv"] + [self.scale[n].cuda() for n in "kv"]
        self.cache = fa.KVCache(*dev)
        self.codes = {n: t.numpy().copy() for n, t in self.codes.items()}
        self.scale = {n: t.double().numpy() for n, t in self.scale.items()}

    def write(self, fa, k, v, start, count, table=None):
        t = self.table if table is None else table
        dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        fa.cache_write(self.cache, k, v, t.cuda(), dev(start), dev(count))
        B, _, N, _ = k.shape
        for n, x in (("k", k), ("v", v)):
            oc.write(self.codes[n], self.scale[n], f64(x), t.numpy(), start or [0] * B,
                     [N] * B if count is None else [min(N, max(0, c)) for c in count], self.page, self.fmt)

    def same(self):
        torch.cuda.synchronize()
        for n, codes, scale in (("k", self.cache.k, self.cache.k_scale), ("v", self.cache.v, self.cache.v_scale)):
            got, s = codes.view(torch.uint8).cpu().numpy(), scale.double().cpu().numpy()
            assert np.array_equal(s, self.scale[n]), f"{n}_scale differs at {np.argwhere(s != self.scale[n])[:4].tolist()}"
            if self.fmt == "e4m3":  # NaN of either sign is one value
                got, want = np.where((got & 127) == 127, 127, got), np.where((self.codes[n] & 127) == 127, 127, self.codes[n])
            else:
                want = self.codes[n]
            assert np.array_equal(got, want), f"{n} differs at {np.argwhere(got != want)[:4].tolist()}"


def rows(B, H, N, d, dt, seed, storage="bhnd", std=1.0):
    g = torch.Generator().manual_seed(seed)
    shape = (B, H, N, d) if storage == "bhnd" else (B, N, H, d)
    x = (torch.randn(shape, generator=g) * std * torch.exp2(torch.randn(shape[:-1] + (1,), generator=g))).to(DT[dt]).cuda()
    return x if storage == "bhnd" else x.transpose(1, 2)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d,dt,storage", [(16, 64, "bf16", "bhnd"), (32, 128, "fp16", "bnhd"), (64, 64, "fp16", "bhnd"),
                                               (64, 128, "bf16", "bnhd"), (128, 128, "bf16", "bhnd"), (128, 64, "fp16", "bnhd"),
                                               (16, 128, "bf16", "bnhd"), (32, 64, "bf16", "bhnd")])
def test_write_in_pieces(fa, page, d, dt, storage, fmt):
    """A prompt, single tokens, a few tokens, a long piece: ragged counts, pages shared by old and
    new tokens, scales that grow."""
    B, H, W = 3, 2, 7
    m = Model(fa, 40, H, page, d, fmt, B, W)
    at = [0, 5, page - 1]
    for i, N in enumerate((page + 3, 1, 1, 2, 7, 8, 9, 2 * page + 1, 1)):
        k, v = rows(B, H, N, d, dt, 100 + i, storage), rows(B, H, N, d, dt, 200 + i, storage, std=2.0 ** (i % 4))
        count = [N, max(0, N - 1 - i), N - N // 2]
        m.write(fa, k, v, list(at), count)
        m.same()
        at = [a + min(N, max(0, c)) for a, c in zip(at, count)]
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("N", [1, 40])
def test_write_values_that_matter(fa, fmt, N):
    """Zeros, ties, the type's largest and smallest, infinities, NaN, a page of zeros that then gets values."""
    B, H, d, page = 2, 1, 64, 16
    m = Model(fa, 16, H, page, d, fmt, B, 6)
    z = torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    m.write(fa, z, z, [0, 3], None)
    m.same()
    x = z.clone()
    x[:, :, 0, :8] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.3e38, -1e-40, 2.0 ** -133, 1.0, -0.0])
    ties = torch.tensor([448.0, 17.0, 19.0, 0.5, 1.5, 2.5, 63.5, 127.0, 113.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10])
    y = z.clone()
    y[:, :, 0, :12] = ties
    y[:, :, N - 1, 20:32] = -ties
    m.write(fa, y, x, [N, 3 + N], None)
    m.same()
    m.write(fa, x, y, [2 * N, 3 + 2 * N], None)   # v's page after an infinity and 3e38
    m.same()


def test_write_count_zero_full_table_and_offsets(fa):
    m = Model(fa, 24, 2, 16, 64, "e4m3", 3, 2)
    k, v = rows(3, 2, 40, 64, "bf16", 1), rows(3, 2, 40, 64, "bf16", 2)
    m.write(fa, k, v, [0, 20, 32], [0, 40, 40])   # nothing; up to the table's end; wholly behind it
    m.same()
    # the kernels clamp what the host cannot see
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.cache_write(m.cache, k, v, m.table.cuda(), i32([2 ** 31 - 1, 2 ** 31 - 64, 32]), i32([40, 2 ** 31 - 1, -7]))
    m.same()
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("N", [4, 40])
def test_bad_pages_are_skipped_and_reported(fa, N):
    m = Model(fa, 24, 2, 16, 64, "int8", 2, 4)
    t = m.table.clone()
    t[0, 0], t[1, 1] = 24, -1
    k, v = rows(2, 2, N, 64, "fp16", 3), rows(2, 2, N, 64, "fp16", 4)
    m.write(fa, k, v, [0, 14], None, table=t)
    m.same()
    assert fa.device_status() == fa.FA_ERR_BAD_PAGE and fa.device_status() == fa.FA_OK
    got, _ = fa.cache_read(m.cache, t.cuda(), torch.tensor([N, N], dtype=torch.int32, device="cuda"), N)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_ERR_BAD_PAGE and not got[0, :, :min(N, 16)].any()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d,dt,N", [(16, 64, "bf16", 1), (64, 128, "fp16", 200), (32, 64, "fp16", 257), (128, 128, "bf16", 130)])
def test_read(fa, page, d, dt, N, fmt):
    B, H = 3, 2
    W = -(-(N + 40) // page) + 1
    m = Model(fa, B * W + 3, H, page, d, fmt, B, W)
    start, count = [0, 37, page], [N, max(0, N - 3), N // 2]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = [torch.full((B, N, H, d), 7.0, dtype=DT[dt], device="cuda").transpose(1, 2) for _ in "kv"]
    k, v = fa.cache_read(m.cache, m.table.cuda(), i32(count), N, start=i32(start), dtype=DT[dt], k_out=out[0], v_out=out[1])
    for n, t in (("k", k), ("v", v)):
        for b in range(B):
            want = np.zeros((H, N, d))
            want[:, :count[b]] = oc.sequence(m.codes[n], m.scale[n], m.table[b].numpy(), page, fmt, start[b], count[b])
            got = f64(t[b])
            assert np.array_equal(np.isnan(got), np.isnan(want))
            got, want = np.nan_to_num(got, nan=0.0), np.nan_to_num(want, nan=0.0)
            tol = torch.finfo(DT[dt]).eps / 2 * np.abs(want) + TINY[dt]
            assert np.all(np.abs(got - want) <= tol)
    assert fa.device_status() == fa.FA_OK


# ------------------------------------------------------------------ attention
def filled(fa, B, H, page, d, fmt, lens, seed=0, std=1.0, spread=0):
    """A cache whose sequences hold random values written by the oracle; the rest is leftovers."""
    W = max(1, -(-max(lens) // page)) + 1
    m = Model(fa, B * W + 2, H, page, d, fmt, B, W, seed)
    rng = np.random.default_rng(seed)
    for n in "kv":
        for b, L in enumerate(lens):
            x = rng.standard_normal((1, H, max(L, 1), d)) * std * np.exp2(rng.integers(-spread, spread + 1, (1, H, max(L, 1), 1)))
            oc.write(m.codes[n], m.scale[n], x, m.table[b:b + 1].numpy(), [0], [L], page, fmt)
        getattr(m.cache, n).view(torch.uint8).copy_(torch.from_numpy(m.codes[n]))
        getattr(m.cache, n + "_scale").copy_(torch.from_numpy(m.scale[n]).float())
    return m


def check_attention(fa, m, q, lens, qlens=None, causal=True, scale=None, o=None, lse=None, dt="bf16", table=None):
    B, H, N, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t = (m.table if table is None else table)
    if o is None:
        o, lse = fa.cache_attention(q, m.cache, t.cuda(), i32(lens), q_len=i32(qlens), causal=causal, scale=scale)
    torch.cuda.synchronize()
    cap = t.shape[1] * m.page
    for b in range(B):
        L, n = min(cap, max(0, lens[b])), N if qlens is None else min(N, max(0, qlens[b]))
        k = oc.sequence(m.codes["k"], m.scale["k"], t[b].numpy(), m.page, m.fmt, 0, L)
        v = oc.sequence(m.codes["v"], m.scale["v"], t[b].numpy(), m.page, m.fmt, 0, L)
        good = ~np.isnan(k[0, :, 0]) if L else np.zeros(0, bool)
        i, j = np.arange(N)[:, None], np.arange(L)[None]
        see = np.broadcast_to((i < n) & (j <= L - n + i if causal else j < L), (N, L)) & good
        wo, wl, mag, big = oc.attend(f64(q[b]), np.nan_to_num(k), np.nan_to_num(v), scale, see)
        go, gl = f64(o[b]), f64(lse[b])
        assert np.array_equal(np.isneginf(gl), np.isneginf(wl)), "rows that see no token"
        eps = torch.finfo(DT[dt]).eps
        tol = eps / 2 * np.abs(wo) + mag * (2.0 ** -11 + 2 * (2.0 ** -17 * big + 2.0 ** -20))[..., None] + TINY[dt]
        err = np.abs(go - wo)
        assert np.all(err <= tol), f"sequence {b}: O off by {np.nanmax(err / tol):.2f} bounds at {np.argwhere(~(err <= tol))[0].tolist()}"
        fin = np.isfinite(wl)
        tl = 2.0 ** -17 * big + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(fin, wl, 0))
        el = np.abs(gl[fin] - wl[fin])
        assert np.all(el <= tl[fin]), f"sequence {b}: LSE off by {np.max(el / tl[fin]):.2f} bounds"
    return o, lse


def queries(B, H, N, d, dt, seed, storage="bnhd"):
    g = torch.Generator().manual_seed(seed)
    if storage == "bhnd":
        return torch.randn((B, H, N, d), generator=g).to(DT[dt]).cuda()
    return torch.randn((B, N, H, d), generator=g).to(DT[dt]).cuda().transpose(1, 2)


@pytest.mark.parametrize("fmt,dt", [("e4m3", "bf16"), ("int8", "fp16")])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32), (128, 64), (128, 16)])
@pytest.mark.parametrize("H,HK,N", [(2, 2, 1), (8, 2, 1), (7, 1, 1), (16, 1, 1), (6, 2, 3), (4, 2, 9), (2, 2, 40), (3, 1, 150)])
def test_attention(fa, H, HK, N, d, page, fmt, dt):
    lens = [1, 33, 300, max(N, 129), 0]
    m = filled(fa, len(lens), HK, page, d, fmt, lens, seed=N, spread=2)
    check_attention(fa, m, queries(len(lens), H, N, d, dt, 5), lens, dt=dt)
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("N,G", [(1, 1), (5, 4), (1, 12), (70, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_queries(fa, N, G, causal):
    """Padded query rows, sequences shorter than their queries, lengths clamped on the device."""
    lens, qlens = [200, 3, 64, 900, 5], [N, min(N, 3), 0, N // 2, N + 7]
    m = filled(fa, 5, 2, 32, 128, "e4m3", [200, 3, 64, 160, 5], seed=1)
    lens[3] = m.table.shape[1] * 32 + 11         # past the table
    for n in "kv":                               # the whole row of pages holds values then
        p = m.table[3].long().numpy()
        m.codes[n][p] = oc.encode(np.random.default_rng(2).standard_normal(m.codes[n][p].shape) * 100, "e4m3")
        getattr(m.cache, n).view(torch.uint8).copy_(torch.from_numpy(m.codes[n]))
    check_attention(fa, m, queries(5, 2 * G, N, 128, "bf16", 6), lens, qlens, causal)
    check_attention(fa, m, queries(5, 2 * G, N, 128, "bf16", 7, "bhnd"), [-4, 0, 1, 2, 3], qlens, causal)


@pytest.mark.parametrize("d,G,N,fmt", [(128, 4, 1, "e4m3"), (64, 1, 1, "int8"), (128, 8, 2, "int8"), (64, 4, 40, "e4m3"), (128, 2, 100, "e4m3")])
def test_long_sequences_are_split_and_merged(fa, d, G, N, fmt):
    lens = [5000, 17, 2048]
    m = filled(fa, 3, 2, 64, d, fmt, lens, seed=3)
    q = queries(3, 2 * G, N, d, "bf16", 8)
    o, lse = check_attention(fa, m, q, lens)
    i32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert fa.cache_attention_workspace_bytes(m.cache, 3, 2 * G, N, m.table.shape[1]) > 0
    o2, l2 = fa.cache_attention(q, m.cache, m.table.cuda(), i32)
    assert torch.equal(o, o2) and torch.equal(lse, l2)       # no order of arrival in the result
    o3, l3 = fa.cache_attention(q, m.cache, m.table.cuda(), i32, split=False)
    check_attention(fa, m, q, lens, o=o3, lse=l3)


def test_scales_far_apart(fa):
    """Pages whose V scales differ by 2^40 and whose keys decide which of them counts, zero pages, tiny and
    huge K scales."""
    lens = [160]
    for seed, big in ((0, 0), (1, 3), (2, 4)):
        m = filled(fa, 1, 1, 32, 64, "e4m3", lens, seed=seed)
        p = m.table[0].long().numpy()
        m.scale["v"][p, 0] = np.exp2([-30.0, 10, 0, -90, 5][:5] + [0.0])[:len(p)]
        m.scale["v"][p[2], 0] = 0.0
        m.scale["k"][p, 0] = 2.0 ** -8
        m.scale["k"][p[big], 0] = 2.0 ** -3      # the keys of page `big` stand out
        for n in "kv":
            getattr(m.cache, n + "_scale").copy_(torch.from_numpy(m.scale[n]).float())
        check_attention(fa, m, queries(1, 2, 1, 64, "bf16", 9), lens, scale=1.0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,G,N,B", [(128, 1, 1, 1), (64, 6, 2, 1), (128, 8, 4, 1), (64, 2, 60, 1), (128, 4, 50, 1), (128, 4, 9, 200), (64, 4, 50, 640)])
def test_pages_of_zeros_beside_large_values(fa, d, G, N, B, fmt):
    """Tokens whose V is zero take their share of the weights whatever the other pages' scale."""
    page, W = 32, 9
    cache = random_cache(fa, W, 2, page, d, fmt, seed=31)
    cache.v_scale[:] = 2.0 ** 30
    cache.v_scale[::2] = 0.0
    cache.v_scale[1] = 2.0 ** -30
    table = torch.arange(W, dtype=torch.int32, device="cuda")[None].expand(B, -1)
    check_batch(fa, queries(B, 2 * G, N, d, "bf16", 32), cache, table, [W * page - 3] * B, [N] * B)


@pytest.mark.parametrize("mul", [2.0 ** -60, 2.0 ** 90])
def test_queries_far_from_one(fa, mul):
    """bf16 queries beyond fp16's range: the row's power of two takes them in."""
    lens = [100, 260]
    m = filled(fa, 2, 1, 16, 64, "int8", lens, seed=4)
    q = (queries(2, 4, 2, 64, "bf16", 10).float() * mul).to(torch.bfloat16)
    check_attention(fa, m, q, lens, scale=0.125 / mul)


def test_nan_and_infinite_values_stay_where_they_are(fa):
    """NaN behind a sequence's end or above the diagonal has no effect; a NaN that a row sees is its result."""
    lens = [50, 50]
    m = filled(fa, 2, 1, 16, 64, "e4m3", lens, seed=5)
    q = queries(2, 2, 4, 64, "bf16", 11)
    page, row = int(m.table[1, 3]), 1            # token 49 of sequence 1: seen by its last query row alone
    for n in "kv":
        m.codes[n][page, 0, row, 7] = 0x7f
        getattr(m.cache, n).view(torch.uint8).copy_(torch.from_numpy(m.codes[n]))
    i32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.cache_attention(q, m.cache, m.table.cuda(), i32)
    assert torch.isfinite(o[0]).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(o[1, :, 3]).all() and torch.isnan(lse[1, :, 3]).all()
    q[0, 1, 2, 0] = float("nan")
    o, lse = fa.cache_attention(q, m.cache, m.table.cuda(), i32)
    bad = torch.isnan(lse[0])
    assert bad.nonzero().tolist() == [[1, 2]] and torch.isnan(o[0, 1, 2]).all() and torch.isfinite(o[0, 0]).all()


@pytest.mark.parametrize("N", [1, 30])
def test_bad_pages_are_masked(fa, N):
    lens = [150, 90]
    m = filled(fa, 2, 2, 16, 128, "e4m3", lens, seed=6)
    t = m.table.clone()
    t[0, 2], t[0, 9], t[1, 0] = -1, 10 ** 6, m.cache.k.shape[0]
    q = queries(2, 4, N, 128, "bf16", 12)
    check_attention(fa, m, q, lens, table=t)
    assert fa.device_status() == fa.FA_ERR_BAD_PAGE
    t[:, :] = -1                                   # entries that no token needs are never looked at
    t[0, :1] = m.table[0, :1]
    check_attention(fa, m, q, [min(16, 3 + N), 0], table=t)
    assert fa.device_status() == fa.FA_OK


def test_broadcast_table_wide_rows_and_strides(fa):
    """One prefix shared by every sequence (a table row of stride 0) and outputs in another layout."""
    lens = [77]
    m = filled(fa, 1, 2, 16, 64, "int8", lens, seed=7)
    t = m.table.cuda().expand(3, -1)
    q = queries(3, 4, 1, 64, "fp16", 13)
    i32 = torch.tensor(lens * 3, dtype=torch.int32, device="cuda")
    out = torch.empty((3, 4, 1, 64), dtype=torch.float16, device="cuda")
    o, lse = fa.cache_attention(q, m.cache, t, i32, out=out)
    assert o.data_ptr() == out.data_ptr()
    m.table = m.table.expand(3, -1)
    check_attention(fa, m, q, lens * 3, o=o, lse=lse, dt="fp16")


def test_other_stream_and_graphs_that_share_a_workspace(fa):
    lens = [2700, 300]
    m = filled(fa, 2, 2, 64, 128, "e4m3", lens, seed=8)
    q = queries(2, 8, 1, 128, "bf16", 14)
    t, n = m.table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = fa.cache_attention(q, m.cache, t, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.cache_attention(q, m.cache, t, n, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = torch.empty(fa.cache_attention_workspace_bytes(m.cache, 2, 8, 1, t.shape[1]), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.cache_attention(q, m.cache, t, n, workspace=ws))
        graphs.append(g)
    assert ws.numel() > 0
    for new in ([2700, 300], [64, 1], [129, 0], [2650, 299]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        for g in graphs:
            g.replay()
        for o, lse in outs:
            check_attention(fa, m, q, new, o=o, lse=lse)
    ws.fill_(255)
    graphs[0].replay()
    check_attention(fa, m, q, new, o=outs[0][0], lse=outs[0][1])


def gpu_reference(q, cache, table, lens, qlens, causal, scale):
    """The definition in fp64 torch products for whole batches: O, LSE and the two magnitudes of the bounds."""
    B, H, N, d = q.shape
    HK, page = cache.heads, cache.page_size
    at = table.long()
    raw = lambda t: t.view(torch.uint8)[at].view(t.dtype)  # noqa: E731
    k, v = ((raw(c).double() * s[at].double()[..., None, None]).transpose(1, 2).flatten(2, 3)
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    L = k.shape[2]
    j, i = torch.arange(L, device=q.device), torch.arange(N, device=q.device)[:, None]
    lens, qlens = (torch.tensor(t, device=q.device)[:, None, None] for t in (lens, qlens))
    see = ((i < qlens) & (j <= lens - qlens + i if causal else j < lens) & (j < lens))[:, None, None]
    behind = ~(j < lens[:, 0])[:, None, :, None]
    k, v = k.masked_fill(behind, 0), v.masked_fill(behind, 0)
    qd = q.double().reshape(B, HK, H // HK * N, d)
    x = (qd @ k.transpose(2, 3) * scale).view(B, HK, H // HK, N, L).masked_fill(~see, -torch.inf)
    big = (qd.abs() @ k.abs().transpose(2, 3) * scale).view(B, HK, H // HK, N, L).masked_fill(~see, 0).amax(-1)
    m = x.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    p = (p / l.clamp(min=1e-300)).view(B, HK, H // HK * N, L)
    lse = (m + torch.log(l)).view(B, H, N)
    return (p @ v).view(B, H, N, d), lse, (p @ v.abs()).view(B, H, N, d), big.view(B, H, N)


def random_cache(fa, P, HK, page, d, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = []
    for _ in "kv":
        x = torch.randn((P, HK, page, d), generator=g, device="cuda") * 40
        codes.append((x.round() if fmt == "int8" else x).clamp(-127, 127).to(CODE[fmt]))
    return fa.KVCache(*codes, *(torch.exp2(torch.randint(-8, -4, (P, HK), generator=g, device="cuda").float()) for _ in "kv"))


def check_batch(fa, q, cache, table, lens, qlens, causal=True, **kw):
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = q.shape[3] ** -0.5
    o, lse = fa.cache_attention(q, cache, table, i32(lens), q_len=i32(qlens), causal=causal, **kw)
    wo, wl, mag, big = gpu_reference(q, cache, table, lens, qlens, causal, scale)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    eps = torch.finfo(q.dtype).eps
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    tol = eps / 2 * wo.abs() + mag * (2.0 ** -11 + 2 * (2.0 ** -17 * big + 2.0 ** -20))[..., None] + 2.0 ** -25
    err = (o.double() - wo).abs()
    assert (err <= tol).all(), f"O off by {(err / tol).max().item():.2f} bounds at {(err > tol).nonzero()[0].tolist()}"
    fin = ~torch.isneginf(wl)
    tl = 2.0 ** -17 * big + 2.0 ** -19 + 2.0 ** -22 * wl.abs()
    assert ((lse.double() - wl).abs()[fin] <= tl[fin]).all()
    return o, lse


@pytest.mark.parametrize("fmt,dt", [("e4m3", "bf16"), ("int8", "fp16")])
@pytest.mark.parametrize("d,page,H,HK,N,B,longest", [
    (64, 16, 40, 20, 9, 170, 120),      # thousands of units of one step: their descriptions wrap
    (128, 64, 40, 20, 9, 170, 128), (128, 16, 32, 16, 1, 300, 100), (64, 32, 18, 2, 16, 8, 3000),
    (128, 128, 3, 1, 341, 3, 2500), (64, 64, 2, 1, 1000, 2, 4000), (128, 16, 8, 2, 260, 2, 1500), (64, 16, 5, 1, 700, 1, 900),
    # enough steps for units of two tiles
    (128, 64, 4, 2, 400, 3, 7000), (64, 16, 6, 2, 300, 2, 12000), (128, 128, 2, 1, 900, 3, 9000), (64, 32, 4, 4, 150, 320, 200),
])
def test_many_units_and_long_chunks(fa, d, page, H, HK, N, B, longest, fmt, dt):
    g = torch.Generator().manual_seed(B + N)
    W = -(-longest // page)
    P = min(4000, B * W + 1)
    cache = random_cache(fa, P, HK, page, d, fmt, seed=N)
    table = torch.randint(0, P, (B, W), generator=g, dtype=torch.int32).cuda()   # sequences may share pages
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    lens[-1] = longest
    qlens = torch.randint(0, N + 1, (B,), generator=g).tolist()
    qlens[-1] = N
    q = queries(B, H, N, d, dt, 16)
    for causal in (True, False):
        a = check_batch(fa, q, cache, table, lens, qlens, causal)
    b = check_batch(fa, q, cache, table, lens, qlens, False, split=False)
    assert torch.isneginf(a[1]).equal(torch.isneginf(b[1]))


@pytest.mark.parametrize("G,N,B", [(1, 3, 2), (2, 12, 2), (1, 40, 2), (4, 60, 2), (1, 400, 2), (2, 12, 300), (1, 50, 300), (2, 100, 640)])
def test_nan_behind_a_row_has_no_effect_on_it(fa, G, N, B):
    """NaN in K and V at token t reaches the rows that see t, all of each of them, and no other row, in every
    kernel (the last three sizes: tiles with their rows twice, units of two tiles); rows of other heads and sequences stay as they are."""
    L = max(N, 1) + 90
    m = filled(fa, 2, 2, 16, 64, "e4m3", [L, L], seed=20)
    table = torch.cat([m.table, m.table[:1].expand(B - 2, -1)]).cuda()
    q = queries(B, 2 * G, N, 64, "bf16", 17)
    i32 = torch.full((B,), L, dtype=torch.int32, device="cuda")
    want, wl = fa.cache_attention(q, m.cache, table, i32)
    at = [L - N + N // 2, L - 1]
    for n, t in zip("vk", at):
        m.codes[n][int(m.table[1, t // 16]), 1, t % 16, 3] = 0xff
        getattr(m.cache, n).view(torch.uint8).copy_(torch.from_numpy(m.codes[n]))
    o, lse = fa.cache_attention(q, m.cache, table, i32)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[1, G:, N // 2:] = True
    assert torch.isnan(o[1, G:, N // 2:]).any(-1).all()
    assert not torch.isnan(o[~hit]).any() and not torch.isnan(lse[~hit]).any()
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])


def test_offsets_beyond_32_bits(fa):
    """A pool whose codes pass 2^32 bytes: the last pages are written, read back and attended over."""
    HK, page, d = 8, 128, 128
    P = 2 ** 32 // (HK * page * d) + 40
    cache = fa.KVCache.empty(P, HK, d, page, torch.float8_e4m3fn)
    table = torch.tensor([[P - 1, 3, P - 7], [P - 30, P - 2, 1]], dtype=torch.int32, device="cuda")
    k, v = rows(2, HK, 300, d, "bf16", 30, "bnhd"), rows(2, HK, 300, d, "bf16", 31, "bnhd")
    n = torch.tensor([300, 257], dtype=torch.int32, device="cuda")
    fa.cache_write(cache, k, v, table, None, n)
    got, _ = fa.cache_read(cache, table, n, 300)
    step = k.double().abs().amax((2, 3), keepdim=True) / 448 * 2 * 32 / 2     # half a step of the largest binade
    live = (torch.arange(300, device="cuda") < n[:, None])[:, None, :, None]
    assert ((got.double() - k.double()).abs() * live <= step).all() and not (got * ~live).any()
    for N, G in ((1, 2), (20, 2)):
        check_batch(fa, queries(2, HK * G, N, d, "bf16", 32), cache, table, [300, 257], [N, N])


def test_two_calls_at_once(fa):
    """Two streams, each with its own outputs and workspace."""
    cache = random_cache(fa, 600, 4, 64, 128, "e4m3", seed=3)
    table = torch.randperm(600, generator=torch.Generator().manual_seed(4)).to(torch.int32)[:520].reshape(4, 130).cuda()
    lens = [8000, 17, 5000, 129]
    q = [queries(4, 8, N, 128, "bf16", 40 + N) for N in (1, 30)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = [fa.cache_attention(x, cache, table, n) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = [[fa.cache_attention(x, cache, table, n, stream=s) for _ in range(4)] for x, s in zip(q, streams)]
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert torch.equal(w[0], r[0]) and torch.equal(w[1], r[1])


def test_captured_decoding_step(fa):
    """Rotary, write and attention of one token in one graph, replayed as the sequences grow."""
    B, HK, G, d, page, W = 3, 2, 4, 64, 16, 6
    m = Model(fa, B * W, HK, page, d, "e4m3", B, W, seed=21)
    rot = fa.rotary_frequencies(d)
    q, k, v = (queries(B, h, 1, d, "bf16", 60 + h) for h in (HK * G, HK, HK))
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    table, start, n = m.table.cuda(), torch.tensor([0, 15, 31], dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((B, HK * G, 1), device="cuda")

    def step():
        fa.rotary_forward(q, rot, k=k, positions=start[:, None], out=qr, k_out=kr)
        fa.cache_write(m.cache, kr, v, table, start)
        torch.add(start, 1, out=n)
        fa.cache_attention(qr, m.cache, table, n, out=o, lse=lse)

    for t in "kv":  # sequences that start at 15 and 31 hold leftovers before: make them plain values
        m.codes[t][:] = oc.encode(np.random.default_rng(5).standard_normal(m.codes[t].shape) * 50, "e4m3")
        getattr(m.cache, t).view(torch.uint8).copy_(torch.from_numpy(m.codes[t]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    at = start.tolist()
    for i in range(5):
        for t, x in enumerate((q, k, v)):
            x.copy_(queries(B, x.shape[1], 1, d, "bf16", 70 + 3 * i + t))
        graph.replay()
        torch.cuda.synchronize()
        for name, x in (("k", kr), ("v", v)):
            oc.write(m.codes[name], m.scale[name], f64(x), m.table.numpy(), at, [1] * B, page, "e4m3")
        m.same()
        at = [a + 1 for a in at]
        check_attention(fa, m, qr, at, o=o, lse=lse)
        start.add_(1)


def test_refusals(fa):
    m = filled(fa, 2, 2, 16, 64, "e4m3", [20, 30], seed=9)
    t, n = m.table.cuda(), torch.tensor([20, 30], dtype=torch.int32, device="cuda")
    q = queries(2, 4, 1, 64, "bf16", 15)
    for args, kw in [((queries(2, 3, 1, 64, "bf16", 1), m.cache, t, n), {}), ((queries(2, 4, 1, 128, "bf16", 1), m.cache, t, n), {}),
                     ((q.float(), m.cache, t, n), {}), ((q, m.cache, t.long(), n), {}), ((q, m.cache, t[:1], n), {}),
                     ((q, m.cache, t.cpu(), n), {}), ((q, m.cache, t, n.long()), {}), ((q, m.cache, t, n[:1]), {}),
                     ((q, m.cache, t, None), {}), ((q, m.cache, t.t().contiguous().t(), n), {}), ((q, None, t, n), {}),
                     ((q, m.cache, t, n), dict(out=q[:, :2])), ((q, m.cache, t, n), dict(lse=torch.zeros(2, 4, 1))),
                     ((q, m.cache, t, n), dict(q_len=n[:1]))]:
        with pytest.raises(ValueError):
            fa.cache_attention(*args, **kw)
    with pytest.raises(fa.FaError):
        fa.cache_attention(q, m.cache, t, n, out=q)
    with pytest.raises(fa.FaError):
        fa.cache_attention(q, m.cache, t, n, scale=float("nan"))
    k = rows(2, 2, 4, 64, "bf16", 1)
    for a in [(k, k.to(torch.float16)), (k, k[:, :, :3]), (k[:, :1], k[:, :1]), (k, rows(2, 2, 4, 64, "bf16", 1, "bnhd"))]:
        with pytest.raises(ValueError):
            fa.cache_write(m.cache, *a, t, n)
    with pytest.raises(ValueError):
        fa.cache_read(m.cache, t, n, 0)
    with pytest.raises(ValueError):
        fa.cache_read(m.cache, t, n, 4, k_out=k)
    with pytest.raises(ValueError):
        fa.cache_read(m.cache, t, n, 4, dtype=torch.float32)
    with pytest.raises(fa.FaError):
        fa.cache_read(m.cache, t, n, 4, k_out=k, v_out=k)
    with pytest.raises(ValueError):
        fa.KVCache(m.cache.k, m.cache.v[:, :, :8], m.cache.k_scale, m.cache.v_scale)
    with pytest.raises(ValueError):
        fa.KVCache(m.cache.k, m.cache.v, m.cache.k_scale.double(), m.cache.v_scale)


@pytest.mark.parametrize("fmt,dt,G", [("e4m3", "bf16", 4), ("int8", "fp16", 1)])
def test_serving_run(fa, fmt, dt, G):
    """As a server uses them: a prompt in two chunks, then tokens one at a time and a few drafted ones, each
    rotated, written and attended over; every step against the definitions on the kernels' own cache."""
    B, HK, d, page, W = 2, 2, 64, 16, 10
    m = Model(fa, B * W + 1, HK, page, d, fmt, B, W, seed=10)
    rot = fa.rotary_frequencies(d, scaling="linear", factor=2.0)
    lens = [0, 0]
    for step, (N, counts) in enumerate([(40, [40, 33]), (37, [20, 37]), (1, [1, 1]), (1, [1, 1]), (4, [4, 4]), (1, [1, 1])]):
        q, k, v = (queries(B, h, N, d, dt, 50 + 3 * step + i) for i, h in enumerate((HK * G, HK, HK)))
        pos = torch.tensor(lens, dtype=torch.int32)[:, None] + torch.arange(N, dtype=torch.int32)
        q, k = fa.rotary_forward(q, rot, k=k, positions=pos.cuda())
        m.write(fa, k, v, list(lens), counts)
        lens = [a + c for a, c in zip(lens, counts)]
        m.same()
        check_attention(fa, m, q, lens, counts, dt=dt)
    i32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    back, _ = fa.cache_read(m.cache, m.table.cuda(), i32, max(lens), dtype=DT[dt])
    want = oc.sequence(m.codes["k"], m.scale["k"], m.table[0].numpy(), page, fmt, 0, lens[0])
    assert np.max(np.abs(f64(back[0, :, :lens[0]]) - want)) <= torch.finfo(DT[dt]).eps / 2 * np.max(np.abs(want))
    assert fa.device_status() == fa.FA_OK
