"""The join of attention over shared prefixes where rows have many parts: rows of one call just below and from 4096
on (which a warp takes one by one or four at a time), prefixes cut into more parts than a row has lanes there,
groups of unequal prefixes and sequences without any beside each other, padded rows, NaN and infinities.

A row of 30 query rows to a sequence behind 8192 tokens: the prefix's 64 steps are shared out over nine or ten of 152 SMs,
the second group's 15 over two, and a row's own tokens are one part more. Bounds: those of test_gpu_shared.py."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import check_attention, queries
from test_gpu_shared import agree, batch, i32, upload

pytestmark = pytest.mark.gpu


def mixed(fa, B, N, HK, page, d, fmt, prefix=(8192, 2000), own=100, seed=0):
    """Six of ten sequences behind the first prefix, three behind the second, one on its own; every fifth padded. Every row sees all of
    its prefix and a token of its own at least."""
    rng = np.random.default_rng(seed + B)
    of = [0 if b % 10 < 6 else 1 if b % 10 < 9 else -1 for b in range(B)]
    m, lens = batch(fa, of, list(prefix), [N + int(x) for x in rng.integers(0, own, B)], HK, page, d, fmt, seed=seed + B)
    qlens = [int(rng.integers(0, N + 1)) if b % 5 == 0 else N for b in range(B)]
    return m, of, list(prefix), lens, qlens


def largest(m):
    return [np.max(np.abs(oc.decode(m.codes[n], m.fmt)).max(axis=(2, 3)) * m.scale[n]) for n in "kv"]


CASES = [
    (137, 6, 5, 1, 128, 64, "e4m3", "bf16"),   # 4110 rows: four a warp, not a multiple of 32
    (136, 6, 5, 1, 128, 64, "int8", "fp16"),   # 4080: one a warp
    (137, 6, 5, 1, 64, 32, "int8", "bf16"),
    (136, 6, 5, 1, 64, 32, "e4m3", "fp16"),
    (129, 2, 8, 2, 128, 16, "e4m3", "bf16"),   # 4128 rows, two cache heads, 16 rows to each
    (64, 16, 4, 1, 128, 128, "int8", "bf16"),  # 4096: own tokens in tiles
    (33, 32, 4, 1, 64, 64, "e4m3", "bf16"),    # 4224: own tokens in tiles of 128 rows
    (4095, 1, 1, 1, 64, 64, "e4m3", "bf16"),
    (4096, 1, 1, 1, 64, 64, "int8", "bf16"),
    (4097, 1, 1, 1, 128, 64, "e4m3", "fp16"),
]


@pytest.mark.parametrize("B,N,G,HK,d,page,fmt,dt", CASES)
def test_many_parts(fa, B, N, G, HK, d, page, fmt, dt):
    """All rows against cache_attention, each within its bounds; sequences of every kind against their definition."""
    m, of, prefix, lens, qlens = mixed(fa, B, N, HK, page, d, fmt)
    q, table = queries(B, HK * G, N, d, dt, 21), m.table.cuda()
    args = (i32(lens), i32(of), i32(prefix))
    o, lse = fa.cache_attention_shared(q, m.cache, table, *args, q_len=i32(qlens))
    want = fa.cache_attention(q, m.cache, table, args[0], q_len=i32(qlens))
    agree(want, (o, lse), q, d ** -0.5, *largest(m))
    step = max(1, B // 13)
    pick = sorted(set(range(0, B, step)) | {5, 6, 9, 10, B - 1})   # both groups, none, padded
    check_attention(fa, m, q[pick], [lens[b] for b in pick], [qlens[b] for b in pick], o=o[pick], lse=lse[pick], dt=dt, table=m.table[pick])
    again = fa.cache_attention_shared(q, m.cache, table, *args, q_len=i32(qlens))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("B,N,G,HK,d,page", [(137, 6, 5, 1, 128, 64), (136, 6, 5, 1, 128, 64), (137, 6, 5, 1, 64, 32), (129, 2, 8, 2, 64, 16),
                                             (64, 16, 4, 1, 128, 128)])
def test_nan_in_v(fa, B, N, G, HK, d, page):
    """A NaN in V of a prefix is in its channel for the rows of the sequences behind it, one of a sequence's own for its rows; all
    other channels and rows are as without them, to the bit."""
    m, of, prefix, lens, qlens = mixed(fa, B, N, HK, page, d, "e4m3", seed=1)
    q, table = queries(B, HK * G, N, d, "bf16", 22), m.table.cuda()
    args = (i32(lens), i32(of), i32(prefix))
    o, lse = fa.cache_attention_shared(q, m.cache, table, *args, q_len=i32(qlens))
    mark = torch.zeros((B, HK * G, N, d), dtype=torch.bool, device="cuda")
    m.codes["v"][int(m.table[0, 5000 // page]), 0, 5000 % page, 17] = 0x7f
    for b in range(B):
        if of[b] == 0:
            mark[b, :G, :qlens[b], 17] = True
    b = 6                                                # the second group's first sequence: its first token behind the prefix
    at = prefix[1] // page
    m.codes["v"][int(m.table[b, at]), HK - 1, 0, 40] = 0xff
    mark[b, (HK - 1) * G:, :qlens[b], 40] = True
    assert of[b] == 1 and qlens[b] > 0
    upload(m)
    o2, lse2 = fa.cache_attention_shared(q, m.cache, table, *args, q_len=i32(qlens))
    assert torch.equal(torch.isnan(o2), mark)
    assert torch.equal(o2[~mark], o[~mark]) and torch.equal(lse2, lse)
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("B,N,G,HK,d,page,fmt", [(137, 6, 5, 1, 128, 64, "e4m3"), (136, 6, 5, 1, 64, 64, "int8"), (64, 16, 4, 1, 64, 32, "e4m3"),
                                                 (40, 1, 4, 2, 128, 64, "int8")])
@pytest.mark.parametrize("below", ["nothing", "prefix", "all"])
def test_infinities_in_q(fa, B, N, G, HK, d, page, fmt, below):
    """Rows of q with an infinity: scores of either infinity and NaN, or (where K's channel has one sign, in the prefix or
    everywhere) of minus infinity alone. Such rows are what cache_attention makes of them, and the others are as ever."""
    m, of, prefix, lens, qlens = mixed(fa, B, N, HK, page, d, fmt, seed=2)
    if below != "nothing":
        pages = m.table[0, :prefix[0] // page].long().numpy() if below == "prefix" else slice(None)
        m.codes["k"][pages, :, :, 3] = 0xb8 if fmt == "e4m3" else 0xfb   # below zero
        upload(m)
    q, table = queries(B, HK * G, N, d, "bf16", 23).contiguous(), m.table.cuda()
    rows = [(0, 0, 0), (1, G - 1, N - 1), (B - 1 - (B - 1) % 10, 0, 0), (6, 0, N - 1), (9, G - 1, 0), (5, 0, N - 1)]  # the last one: padded
    mark = torch.zeros((B, HK * G, N), dtype=torch.bool, device="cuda")
    clean = q.clone()
    for k, at in enumerate(rows):
        q[at][3] = float("inf") if k != 1 else -float("inf")
        clean[at] = 0
        mark[at] = True
    args = (i32(lens), i32(of), i32(prefix))
    o, lse = fa.cache_attention_shared(q, m.cache, table, *args, q_len=i32(qlens))
    wo, wl = fa.cache_attention(q, m.cache, table, args[0], q_len=i32(qlens))
    assert torch.equal(torch.isnan(o), torch.isnan(wo)) and torch.equal(torch.isnan(lse), torch.isnan(wl))
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    assert not torch.isnan(lse[~mark]).any() and not torch.isnan(o[~mark]).any()
    none = torch.isneginf(lse) & mark
    assert not o[none].any()
    clear = [torch.where(mark[..., None], 0, t) for t in (o, wo)], [torch.where(mark, 0, t) for t in (lse, wl)]
    agree((clear[0][1], clear[1][1]), (clear[0][0], clear[1][0]), clean, d ** -0.5, *largest(m))
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("d,fmt,dt", [(128, "e4m3", "bf16"), (128, "int8", "fp16"), (64, "e4m3", "fp16")])
def test_more_sequences_than_the_plan_has_threads(fa, d, fmt, dt):
    """1500 sequences in three groups of several tiles of 256 rows each, one of a page, and on their own."""
    B, G = 1500, 4
    prefix = [700, 3000, 1500, 64]
    of = [(b * 7) % 5 - 1 for b in range(B)]             # -1 .. 3
    rng = np.random.default_rng(5)
    m, lens = batch(fa, of, prefix, [1 + int(x) for x in rng.integers(0, 60, B)], 1, 64, d, fmt, seed=11)
    q, table = queries(B, G, 1, d, dt, 24), m.table.cuda()
    o, lse = fa.cache_attention_shared(q, m.cache, table, i32(lens), i32(of), i32(prefix))
    want = fa.cache_attention(q, m.cache, table, i32(lens))
    agree(want, (o, lse), q, d ** -0.5, *largest(m))
    pick = list(range(0, B, 61))
    check_attention(fa, m, q[pick], [lens[b] for b in pick], o=o[pick], lse=lse[pick], dt=dt, table=m.table[pick])
    assert fa.device_status() == fa.FA_OK


def test_a_call_leaves_no_mark_of_its_plan(fa):
    """Kernels that run beside each other know by a mark in the workspace that the call's plan is made. A graph runs the same call
    again, so the mark is gone when the call ends, and what the workspace holds before a replay does not matter."""
    m, of, prefix, lens, qlens = mixed(fa, 40, 2, 2, 32, 64, "e4m3", seed=3)
    q, table, args = queries(40, 8, 2, 64, "bf16", 25), m.table.cuda(), (i32(lens), i32(of), i32(prefix))
    need = fa.cache_attention_shared_workspace_bytes(m.cache, 40, 8, 2, table.shape[1], len(prefix))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((40, 8, 2), device="cuda")
    want = fa.cache_attention_shared(q, m.cache, table, *args, workspace=ws)
    torch.cuda.synchronize()
    assert not ws[128:136].any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            fa.cache_attention_shared(q, m.cache, table, *args, out=out, lse=lse, workspace=ws)
    left = None
    for i in range(6):
        ws.fill_(0xff) if left is None or i % 2 else ws.copy_(left)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        left = ws.clone()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and not ws[128:136].any()
    assert fa.device_status() == fa.FA_OK
