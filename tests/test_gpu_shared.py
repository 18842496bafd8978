"""Attention over shared prefixes against the fp64 definition of attention over each sequence's own row of
pages (oracle/cache.py), and the page calls, the cache and both attentions used together.

The bounds are those of test_gpu_cache.py: a row's parts are joined in 32 bits by the same sums as the
parts of a cut unit there, and which rows share a tile changes nothing in what a row rounds."""
import numpy as np
import pytest
import torch

from _util import f64
from oracle import cache as oc
from test_gpu_cache import DT, Model, check_attention, queries

pytestmark = pytest.mark.gpu


def i32(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def batch(fa, of, prefix, own, HK, page, d, fmt, seed=0, spread=2, wide=True):
    """Sequences b of group of[b] (-1: none) with the whole pages of prefix[of[b]] tokens in common and own[b] tokens behind
    them; every page holds finite values. A call whose table has room for few tokens is that of cache_attention: `wide` gives it
    room for 2^18, so that all is shared that can be."""
    rng = np.random.default_rng(seed)
    shared = [p // page for p in prefix]
    lens = [own[b] + (shared[g] * page if 0 <= g < len(prefix) else 0) for b, g in enumerate(of)]
    W = (1 << 18) // page if wide else max(1, -(-max(lens) // page)) + 1
    P = sum(shared) + sum(-(-n // page) for n in own) + 5
    m = Model(fa, P, HK, page, d, fmt, 1, 1, seed)
    for n in "kv":
        m.codes[n] = oc.encode(rng.standard_normal(m.codes[n].shape) * (16 if fmt == "e4m3" else 40), fmt)
        m.scale[n] = np.exp2(rng.integers(-5 - spread, -4 + spread, (P, HK)).astype(np.float64)) / (4 if fmt == "int8" else 1)
    order, at = rng.permutation(P).tolist(), 0
    first = []
    for s in shared:
        first.append(order[at:at + s])
        at += s
    table = np.full((len(of), W), -1, np.int32)
    for b, g in enumerate(of):
        head = first[g] if 0 <= g < len(prefix) else []
        table[b, :len(head)] = head
        k = -(-own[b] // page)
        table[b, len(head):len(head) + k] = order[at:at + k]
        at += k
    m.table = torch.from_numpy(table)
    upload(m)
    return m, lens


def upload(m):
    for n in "kv":
        getattr(m.cache, n).view(torch.uint8).copy_(torch.from_numpy(m.codes[n]))
        getattr(m.cache, n + "_scale").copy_(torch.from_numpy(m.scale[n]).float())


def check_shared(fa, m, q, lens, of, prefix, qlens=None, causal=True, scale=None, dt="bf16", **kw):
    o, lse = fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(prefix), q_len=i32(qlens), causal=causal,
                                       scale=scale, **kw)
    return check_attention(fa, m, q, lens, qlens, causal, scale, o, lse, dt)


@pytest.mark.parametrize("fmt,dt", [("e4m3", "bf16"), ("int8", "fp16")])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32), (128, 64), (128, 16)])
@pytest.mark.parametrize("H,HK,N", [(2, 2, 1), (8, 2, 1), (7, 1, 1), (16, 1, 1), (6, 2, 3), (4, 2, 9), (2, 2, 40), (3, 1, 43), (3, 1, 44)])
def test_shared(fa, H, HK, N, d, page, fmt, dt):
    """A large group, a small one, one of one, sequences without any, in any order; with these, every kernel: 8 and 16
    rows, tiles with rows twice, of 128 rows and pairs of them (43 rows of 3: just not shared any more)."""
    of = [0, 1, 0, -1, 0, 2, 1, 0, 0, 7, 0]
    prefix, own = [300, 128, 40], [N + x for x in (0, 5, 33, 200, 1, 9, 130, 64, 15, 0, 17)]
    m, lens = batch(fa, of, prefix, own, HK, page, d, fmt, seed=N)
    check_shared(fa, m, queries(len(of), H, N, d, dt, 5), lens, of, prefix, dt=dt)
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("B,groups,HK,G,N,prefix,own,d,page,fmt", [
    (70, 1, 2, 4, 1, 5000, 300, 128, 64, "e4m3"),     # 280 rows to a cache head: two tiles of 256
    (33, 1, 1, 8, 1, 2000, 40, 64, 16, "int8"),       # 264 rows, one head
    (40, 20, 2, 4, 1, 600, 100, 128, 32, "e4m3"),     # pairs: few rows
    (24, 8, 3, 2, 5, 1100, 700, 64, 32, "e4m3"),      # 30 rows
    (12, 3, 2, 8, 6, 900, 200, 128, 128, "int8"),     # own tokens in tiles of 64
    (9, 2, 1, 16, 7, 700, 400, 64, 16, "e4m3"),       # 112 rows of a sequence: own tokens in tiles of 128
    (200, 3, 1, 1, 1, 500, 60, 64, 16, "int8"),
    (2, 1, 4, 3, 2, 4000, 9, 128, 16, "e4m3"),        # two sequences
    (1, 1, 4, 3, 2, 400, 9, 128, 16, "e4m3"),         # one: nothing to share
])
def test_sizes(fa, B, groups, HK, G, N, prefix, own, d, page, fmt):
    rng = np.random.default_rng(B)
    of, pre = [b % groups for b in range(B)], [prefix - 37 * g for g in range(groups)]
    m, lens = batch(fa, of, pre, [N + int(x) for x in rng.integers(0, own, B)], HK, page, d, fmt, seed=B)
    q = queries(B, HK * G, N, d, "bf16", 7, "bnhd")
    o, lse = check_shared(fa, m, q, lens, of, pre)
    o2, l2 = fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(pre))
    assert torch.equal(o, o2) and torch.equal(lse, l2)   # no order of arrival in the result
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("B,groups,N,G", [(2500, 1100, 1, 1), (2500, 3, 1, 2), (1500, 40, 6, 3)])
def test_large_batches(fa, B, groups, N, G):
    """More sequences, and more groups, than the plan has threads; every fiftieth sequence against its definition, all of them
    against cache_attention: each within its bounds, with |O| <= sum p |v| <= max |v| and E <= scale max |k| sum |q|."""
    rng = np.random.default_rng(B)
    of = rng.integers(-1, groups, B)
    prefix = (16 * rng.integers(0, 7, groups) + 5).tolist()
    own = [N + int(x) for x in rng.integers(0, 30, B)]
    m, lens = batch(fa, of.tolist(), prefix, own, 1, 16, 64, "e4m3", seed=10)
    q, table = queries(B, G, N, 64, "bf16", 15), m.table.cuda()
    o, lse = fa.cache_attention_shared(q, m.cache, table, i32(lens), i32(of), i32(prefix))
    want = fa.cache_attention(q, m.cache, table, i32(lens))
    most = {n: np.max(np.abs(oc.decode(m.codes[n], "e4m3")).max(axis=(1, 2, 3)) * m.scale[n][:, 0]) for n in "kv"}
    agree(want, (o, lse), q, 64 ** -0.5, most["k"], most["v"])
    pick = list(range(0, B, 50))
    check_attention(fa, m, q[pick], [lens[b] for b in pick], o=o[pick], lse=lse[pick], table=m.table[pick])
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("N,G", [(1, 1), (5, 4), (1, 12), (30, 3)])
@pytest.mark.parametrize("causal,wide", [(True, True), (False, True), (True, False)])
def test_any_lengths(fa, N, G, causal, wide):
    """Padded rows, sequences that end within or before their prefix, prefixes past the table or negative, no tokens at all."""
    of = [0, 0, 0, 0, 0, 0, 1, 1, 2, 2, 3, 3, -9, 99]
    prefix = [330, 10 ** 9, -5, 15]
    m, lens = batch(fa, of, [330, 64, 0, 0], [N + 20, N, 1, 40, 7, 30, N + 1, N + 1, 30, 5, 40, 41, 8, 50], 2, 32, 128, "e4m3", seed=3, wide=wide)
    m.table[7] = m.table[6]                              # group 1: the whole table is shared
    lens[7] = lens[6]
    qlens = [N, min(N, 2), N, 0, N // 2, N + 7, N, N, N, 1, N, 0, N, N]
    lens[2], lens[4], lens[5] = 200, 0, -3               # within the prefix, empty, negative
    q = queries(len(of), 2 * G, N, 128, "bf16", 6)
    check_shared(fa, m, q, lens, of, prefix, qlens, causal)
    check_shared(fa, m, q, lens, of, prefix, None, causal)
    check_shared(fa, m, q, [0] * len(of), of, prefix, qlens, causal)
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("G,N,B", [(4, 1, 3), (4, 1, 30), (3, 20, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_nothing_behind_the_prefix(fa, G, N, B, causal):
    """Sequences that end with their prefix: single tokens (and, without causality, any rows) see all of it."""
    of, prefix = [b % 2 for b in range(B)], [256, 320]
    m, lens = batch(fa, of, prefix, [0 if b % 3 else N + b for b in range(B)], 2, 64, 64, "e4m3", seed=9)
    check_shared(fa, m, queries(B, 2 * G, N, 64, "bf16", 14), lens, of, prefix, causal=causal)


def test_group_hint_of_another_size(fa):
    """`groups` far from the groups in use: all in one of 64, and as many groups as sequences."""
    B = 40
    for groups, of in ((64, [50] * B), (B, [b // 2 for b in range(B)]), (2048, [2047 - b % 3 for b in range(B)])):
        prefix = [0] * groups
        for g in set(of):
            prefix[g] = 256
        m, lens = batch(fa, of, prefix, [1 + 7 * b % 90 for b in range(B)], 2, 32, 64, "int8", seed=groups)
        check_shared(fa, m, queries(B, 8, 1, 64, "bf16", 8), lens, of, prefix)


@pytest.mark.parametrize("G,N,B", [(1, 1, 5), (4, 1, 5), (4, 1, 40), (4, 6, 6), (4, 30, 4)])
def test_nan(fa, G, N, B):
    """NaN behind the prefix's end and behind the rows has no effect; one in V of the prefix is in its channel for all that see
    it; one in K is in all of their results; one in q in its row alone."""
    of, prefix = [0] * (B - 1) + [-1], [330]
    m, lens = batch(fa, of, prefix, [N + 3] * B, 1, 32, 64, "e4m3", seed=4)
    last = int(m.table[0, lens[0] // 32])
    row = lens[0] % 32
    if row:                                              # behind sequence 0's last token
        for n in "kv":
            m.codes[n][last, 0, row:] = 0x7f
    unused = sorted(set(range(m.cache.k.shape[0])) - set(m.table.flatten().tolist()))
    for n in "kv":
        m.codes[n][unused] = 0x7f
    upload(m)
    q = queries(B, G, N, 64, "bf16", 9)
    check_shared(fa, m, q, lens, of, prefix)
    m.codes["v"][int(m.table[0, 3]), 0, 5, 17] = 0xff    # token 101 of the prefix
    upload(m)
    o, lse = fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(prefix))
    nan = torch.isnan(o)
    assert nan[:-1, ..., 17].all() and nan.sum() == (B - 1) * G * N and torch.isfinite(lse).all()
    own = int(m.table[0, 10])                            # the first page behind it, a row that every query of sequence 0 sees
    m.codes["v"][own, 0, 1, 40] = 0x7f
    upload(m)
    o, _ = fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(prefix))
    nan = torch.isnan(o)
    assert nan[0, ..., 40].all() and nan[:-1, ..., 17].all() and nan.sum() == B * G * N
    m.codes["k"][int(m.table[0, 9]), 0, 31, 0] = 0x7f    # the prefix's last token
    upload(m)
    o, lse = fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(prefix))
    assert torch.isnan(o[:-1]).all() and torch.isnan(lse[:-1]).all() and torch.isfinite(o[-1]).all()
    m.codes["k"][int(m.table[0, 9]), 0, 31, 0] = 0
    upload(m)
    q[1, G - 1, N - 1, 3] = float("nan")
    o, lse = fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(prefix))
    assert torch.isnan(lse).nonzero().tolist() == [[1, G - 1, N - 1]] and torch.isnan(o[1, G - 1, N - 1]).all()


@pytest.mark.parametrize("G,N,B", [(4, 1, 3), (4, 1, 40), (2, 30, 4)])
def test_pages_of_zeros_bad_pages_and_far_scales(fa, G, N, B):
    of, prefix = [0] * B, [512]
    m, lens = batch(fa, of, prefix, [N + 5] * B, 2, 32, 128, "e4m3", seed=5)
    m.scale["v"][m.table[0, 1:9:2].long().numpy()] = 0.0
    m.scale["v"][int(m.table[0, 2])] = 2.0 ** 30
    upload(m)
    q = queries(B, 2 * G, N, 128, "bf16", 10)
    check_shared(fa, m, q, lens, of, prefix)
    m.scale["v"][int(m.table[0, 2])] = 2.0 ** -5
    upload(m)
    m.table[:, 5], m.table[:, 6], m.table[1, 16] = -1, 10 ** 6, m.cache.k.shape[0]
    check_shared(fa, m, q, lens, of, prefix)
    assert fa.device_status() == fa.FA_ERR_BAD_PAGE


def test_outputs_workspace_and_a_table_in_a_wider_one(fa):
    of, prefix = [0, 0, 1, 0, 1], [200, 90]
    m, lens = batch(fa, of, prefix, [30, 1, 17, 64, 5], 2, 16, 64, "int8", seed=6)
    W = m.table.shape[1]
    assert W == 1 << 14
    wide = torch.full((5, W + 9), 10 ** 8, dtype=torch.int32)
    wide[:, 4:4 + W] = m.table
    q = queries(5, 6, 1, 64, "fp16", 11, "bnhd")
    out = torch.full((5, 6, 3, 64), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.empty((5, 6, 1), dtype=torch.float32, device="cuda")
    ws = torch.full((fa.cache_attention_shared_workspace_bytes(m.cache, 5, 6, 1, W, 2),), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o, l = fa.cache_attention_shared(q, m.cache, wide.cuda()[:, 4:4 + W], i32(lens), i32(of), i32(prefix), out=out[:, :, 1:2], lse=lse, workspace=ws)
        assert o.data_ptr() == out[:, :, 1:2].data_ptr() and l is lse
        check_attention(fa, m, q, lens, o=o, lse=l, dt="fp16")
        assert (out[:, :, ::2] == 7).all()
        ws.fill_(0x3c)
    with pytest.raises(fa.FaError):
        fa.cache_attention_shared(q, m.cache, m.table.cuda(), i32(lens), i32(of), i32(prefix), workspace=ws[:-16])


def test_offsets_past_32_bits(fa):
    """A pool of more than 2^32 bytes of codes, a prefix in its last pages."""
    P, HK, page, d = 40000, 8, 128, 128
    k = torch.zeros((P, HK, page, d), dtype=torch.int8, device="cuda")
    cache = fa.KVCache(k, torch.zeros_like(k), *(torch.ones((P, HK), dtype=torch.float32, device="cuda") for _ in "kv"))
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (cache.k, cache.v):
        t[P - 9:] = torch.randint(-9, 10, (9, HK, page, d), generator=g, device="cuda", dtype=torch.int8)
    table = torch.full((20, 300), -1, dtype=torch.int32)
    table[:, :7] = torch.arange(P - 7, P)
    table[:, 7] = P - 8
    table = table.cuda()
    q = queries(20, 8, 1, d, "bf16", 1)
    lens, of = [7 * page + 1 + b for b in range(20)], [0] * 20
    o, lse = fa.cache_attention_shared(q, cache, table, i32(lens), i32(of), i32([7 * page]), scale=0.01)
    m = Model(fa, 9, HK, page, d, "int8", 1, 1)
    m.codes = {n: getattr(cache, n)[P - 9:].cpu().view(torch.uint8).numpy().copy() for n in "kv"}
    m.scale = {n: np.ones((9, HK)) for n in "kv"}
    m.table = torch.where(table.cpu() >= 0, table.cpu() - (P - 9), -1)
    check_attention(fa, m, q, lens, scale=0.01, o=o, lse=lse)
    src, dst = [P - 1, P - 2], [P - 20, 3]
    fa.cache_copy(cache, i32(src), i32(dst))
    assert torch.equal(cache.k[dst], cache.k[src]) and torch.equal(cache.v[dst], cache.v[src])


def test_few_tokens_are_the_plain_attention(fa):
    """Where the table has room for few tokens, and where a sequence has more than 128 rows to a cache head, nothing is shared."""
    of, prefix = [0] * 6, [96]
    for N, wide in ((1, False), (130, True)):
        m, lens = batch(fa, of, prefix, [N + 7 * b for b in range(6)], 1, 32, 64, "e4m3", seed=8, wide=wide)
        q, table = queries(6, 1, N, 64, "bf16", 13), m.table.cuda()
        o, lse = check_shared(fa, m, q, lens, of, prefix)
        want = fa.cache_attention(q, m.cache, table, i32(lens))
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert fa.cache_attention_shared_workspace_bytes(m.cache, 6, 1, N, table.shape[1], 1) == fa.cache_attention_workspace_bytes(m.cache, 6, 1, N, table.shape[1])


# ------------------------------------------------------------------ together
def agree(a, b, q, scale, kmax, vmax):
    """Both attentions' O, LSE: each within the bounds of the same exact values, |O| <= sum p |v| <= vmax, E <= scale kmax sum |q|."""
    E = scale * kmax * q.float().abs().sum(-1).max().item()
    live = torch.isfinite(a[1])
    assert torch.equal(a[1][~live], b[1][~live])
    assert (a[1][live] - b[1][live]).abs().max() <= 2 * (2.0 ** -17 * E + 2.0 ** -19 + 2.0 ** -22 * a[1][live].abs().max().item())
    assert (a[0].float() - b[0].float()).abs().max() <= 2 * vmax * (2.0 ** -9 + 2.0 ** -11 + 2 * (2.0 ** -17 * E + 2.0 ** -20))


def test_a_serving_run(fa):
    """Prompts written, samples forked from them, tokens written and attended over by both attentions, some samples dropped, the
    pool moved together in between, in two layers: every sequence reads back what was written to it."""
    page, HK, H, d, P, S, W = 16, 2, 4, 64, 200, 12, 9000
    caches = [fa.KVCache.empty(P, HK, d, page, dtype=torch.int8) for _ in range(2)]
    table, refs = torch.full((S, W), -1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(0)
    values = {}   # token -> its constant value in every layer
    said = [[] for _ in range(S)]

    def write(start, count, first):
        n = max(count)
        ids = np.zeros((S, n), np.int64)
        for b in range(S):
            for t in range(count[b]):
                values[first] = float(rng.integers(-100, 101))
                ids[b, t] = first
                said[b].append(first)
                first += 1
        for l, c in enumerate(caches):
            x = torch.tensor([[values.get(i, 0.0) for i in row] for row in ids], device="cuda")[:, None, :, None].expand(S, HK, n, d)
            fa.cache_write(c, (x + l).to(torch.bfloat16).contiguous(), (x - l).to(torch.bfloat16).contiguous(), table, i32(start), i32(count))
        return first

    def read_back():
        lens = [len(s) for s in said]
        for l, c in enumerate(caches):
            k, v = fa.cache_read(c, table, i32(lens), max(lens))
            for b in range(S):
                want = torch.tensor([values[i] for i in said[b]], device="cuda")
                # int8 codes of values up to 101: scales of 1 at most, so that whole numbers are held exactly
                assert torch.equal(k[b, 0, :lens[b], 3].float(), want + l) and torch.equal(v[b, 1, :lens[b], 60].float(), want - l)

    def attend(of, prefix):
        lens = [len(s) for s in said]
        q = queries(S, H, 1, d, "bf16", len(values))
        for c in caches:
            a = fa.cache_attention(q, c, table, i32(lens), scale=0.001)
            b = fa.cache_attention_shared(q, c, table, i32(lens), i32(of), i32(prefix), scale=0.001)
            agree(a, b, q, 0.001, 101, 101)

    count = [100, 37] + [0] * (S - 2)
    assert fa.cache_reserve(caches, table, refs, None, i32(count)).tolist() == [1] * S
    token = write([0] * S, count, 0)
    parent = [0, 1] + [0] * 6 + [1] * 4
    fa.cache_fork(table, refs, page, parent=i32(parent))
    said = [list(said[p]) for p in parent]
    read_back()
    for step in range(40):
        start = [len(s) for s in said]
        ok = fa.cache_reserve(caches, table, refs, i32(start), 1).tolist()
        token = write(start, ok, token)
        attend(parent, [100, 37])
        if step % 7 == 3:      # sample 3 goes back to its prompt, sample 5 continues as sample 4 does
            new = list(range(S))
            new[3], new[5] = 0, 4
            keep = [W * page] * S
            keep[3] = 100
            fa.cache_fork(table, refs, page, parent=i32(new), keep=i32(keep))
            said = [list(said[p]) for p in new]
            said[3] = said[3][:100]
        if step % 11 == 5:
            _, live = fa.cache_compact(caches, table, refs)
            assert not refs[live.item():].any() and (refs[:live.item()] > 0).all()
        read_back()
    held = table[table >= 0].long()
    assert torch.equal(refs, torch.bincount(held, minlength=P).to(torch.int32))
    fa.cache_fork(table, refs, page, parent=i32([-1] * S))
    assert not refs.any() and (table == -1).all() and fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("groups", [1, 3])
def test_a_captured_step_is_replayed_with_other_lengths(fa, groups):
    """Reserve, write and attend in one graph, replayed token by token; the sequences' pages come from the pool as they grow.
    A second graph shares the workspaces and runs after the first."""
    B, HK, H, d, page, P, W = 6, 2, 8, 64, 16, 120, 9000
    cache = fa.KVCache.empty(P, HK, d, page)
    table, refs = torch.full((B, W), -1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    of = [b % groups for b in range(B)]
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    prompt = i32([70 if b < groups else 0 for b in range(B)])
    g = torch.Generator(device="cuda").manual_seed(2)
    fa.cache_reserve(cache, table, refs, None, prompt)
    kv = [torch.randn((B, HK, 70, d), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
    fa.cache_write(cache, *kv, table, None, count=prompt)
    fa.cache_fork(table, refs, page, parent=i32(of))
    start.fill_(70)
    q, k, v = (torch.zeros((B, h, 1, d), dtype=torch.bfloat16, device="cuda") for h in (H, HK, HK))
    prefix = i32([70] * groups)
    ok = torch.empty(B, dtype=torch.int32, device="cuda")
    w1 = torch.empty(fa.cache_reserve_workspace_bytes(cache, B, W), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(fa.cache_attention_shared_workspace_bytes(cache, B, H, 1, W, groups), dtype=torch.uint8, device="cuda")
    members, out, lse, kv_len = i32(of), torch.empty_like(q), torch.empty((B, H, 1), device="cuda"), torch.zeros_like(start)

    def step():
        fa.cache_reserve(cache, table, refs, start, 1, ok=ok, workspace=w1)
        fa.cache_write(cache, k, v, table, start)
        torch.add(start, 1, out=kv_len)
        fa.cache_attention_shared(q, cache, table, kv_len, members, prefix, out=out, lse=lse, workspace=w2)
        start.copy_(kv_len)

    side = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    saved = [t.clone() for t in (table, refs, start, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for gr in graphs:
        with torch.cuda.graph(gr):
            step()
    for t, s in zip((table, refs, start, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale), saved):
        t.copy_(s)
    kmax, vmax = (t.abs().max().item() for t in kv)
    for i in range(40):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graphs[i % 2].replay()
        want = fa.cache_attention(q, cache, table, kv_len)
        assert ok.tolist() == [1] * B and start.tolist() == [71 + i] * B
        kmax, vmax = (max(most, t.abs().max().item()) for most, t in zip((kmax, vmax), (k, v)))
        agree(want, (out, lse), q, 64 ** -0.5, 17 / 16 * kmax, 17 / 16 * vmax)   # held in e4m3: off by a sixteenth at most
    held = table[table >= 0].long()
    assert torch.equal(refs, torch.bincount(held, minlength=P).to(torch.int32)) and fa.device_status() == fa.FA_OK


def test_other_streams(fa):
    """Calls on a stream that is not the current one, two at a time with workspaces of their own."""
    of, prefix = [b % 2 for b in range(30)], [500, 300]
    m, lens = batch(fa, of, prefix, [1 + 9 * b for b in range(30)], 2, 16, 64, "e4m3", seed=7)
    q, args = queries(30, 8, 1, 64, "bf16", 12), (i32(lens), i32(of), i32(prefix))
    table = m.table.cuda()
    want = check_shared(fa, m, q, lens, of, prefix)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = fa.cache_attention_shared_workspace_bytes(m.cache, 30, 8, 1, table.shape[1], 2)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [(torch.empty_like(q), torch.empty_like(want[1])) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, (o, l) in zip(streams, ws, outs):
            fa.cache_attention_shared(q, m.cache, table, *args, out=o, lse=l, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
