"""The page calls against their definitions (oracle/pages.py): everything is counted or copied, so
everything has to be equal."""
import numpy as np
import pytest
import torch

from oracle import pages as op

pytestmark = pytest.mark.gpu
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def pools(fa, layers, P, H, page, d, fmt="e4m3", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(layers):
        codes = [torch.randint(0, 256, (P, H, page, d), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8).view(CODE[fmt])
                 for _ in "kv"]
        out.append(fa.KVCache(*codes, *(torch.rand((P, H), generator=g, device="cuda") for _ in "kv")))
    return out


def bits(caches):
    return [t.view(torch.uint8).clone() if t.dtype != torch.float32 else t.clone() for c in caches for t in (c.k, c.v, c.k_scale, c.v_scale)]


def moved(before, moves):
    if moves:
        src, dst = (torch.tensor(t, device="cuda") for t in zip(*moves))
        for t in before:
            t[dst] = t[src]
    return before


def same(caches, want):
    return all(torch.equal(a, b) for a, b in zip(bits(caches), want))


# ------------------------------------------------------------------ copy
@pytest.mark.parametrize("layers,P,H,page,d,fmt,n", [(1, 8, 1, 16, 64, "int8", 1), (1, 9, 12, 16, 64, "int8", 3), (3, 40, 5, 32, 128, "e4m3", 17),
                                                     (2, 16, 13, 16, 64, "e4m3", 8), (2, 30, 17, 128, 128, "int8", 12), (66, 5, 1, 16, 64, "e4m3", 2),
                                                     (4, 700, 8, 64, 128, "e4m3", 300), (1, 3, 331, 128, 128, "int8", 1)])
def test_copy(fa, layers, P, H, page, d, fmt, n):
    caches = pools(fa, layers, P, H, page, d, fmt)
    order = torch.randperm(P, generator=torch.Generator().manual_seed(n)).tolist()
    src, dst = order[:n], order[n:2 * n]
    want = moved(bits(caches), list(zip(src, dst)))
    fa.cache_copy(caches, i32(src), i32(dst))
    assert same(caches, want)
    assert fa.device_status() == fa.FA_OK


def test_copy_what_is_left_out(fa):
    caches = pools(fa, 2, 20, 2, 16, 64)
    before = bits(caches)
    fa.cache_copy(caches, i32([-1, 3, -1, 5]), i32([4, -1, -1, 5]))   # no moves, and a page onto itself
    fa.cache_copy(caches, i32([]), i32([]))
    assert same(caches, before) and fa.device_status() == fa.FA_OK
    fa.cache_copy(caches, i32([20, 1, -2, 2 ** 31 - 1, 7]), i32([6, -9, 8, 9, 10]))
    assert same(caches, moved(before, [(7, 10)])) and fa.device_status() == fa.FA_ERR_BAD_PAGE
    one = bits(caches[:1])
    fa.cache_copy(caches[0], i32([2]), i32([3]))                      # a single cache
    assert same(caches[:1], moved(one, [(2, 3)])) and same(caches[1:], before[4:])


def test_copy_same_source_twice(fa):
    caches = pools(fa, 1, 30, 3, 64, 64)
    want = moved(bits(caches), [(4, 9), (4, 11), (4, 2)])
    fa.cache_copy(caches, i32([4, 4, 4]), i32([9, 11, 2]))
    assert same(caches, want)


# ------------------------------------------------------------------ fork
def random_table(rng, B, W, P, page, shared=0.4):
    """Rows of random length; some begin with the pages of another."""
    table, refs = np.full((B, W), -1, np.int32), np.zeros(P, np.int32)
    free = list(rng.permutation(P))
    length = np.zeros(B, np.int64)
    for b in range(B):
        n = int(rng.integers(0, W + 1))
        k = 0
        if b and rng.random() < shared:
            p = int(rng.integers(0, b))
            k = min(n, int((table[p] >= 0).sum()), int(rng.integers(0, W + 1)))
            table[b, :k] = table[p, :k]
        n = min(n, k + max(0, len(free) - 4))
        for c in range(k, n):
            table[b, c] = free.pop()
        length[b] = max(0, n * page - int(rng.integers(0, page)))
        refs += np.bincount(table[b][table[b] >= 0], minlength=P).astype(np.int32)
    return table, refs, length


@pytest.mark.parametrize("B,W,P,page", [(1, 1, 1, 16), (5, 7, 40, 16), (33, 65, 900, 64), (64, 300, 4000, 32), (700, 33, 3000, 128), (16384, 3, 9000, 16)])
@pytest.mark.parametrize("kind", ["beams", "samples", "free", "trim", "mixed"])
def test_fork(fa, B, W, P, page, kind):
    rng = np.random.default_rng(B + W)
    table, refs, length = random_table(rng, B, W, P, page)
    me = np.arange(B)
    parent = {"beams": rng.integers(0, B, B), "samples": np.where(me < (B + 3) // 4, me, me % ((B + 3) // 4)),
              "free": np.where(rng.random(B) < 0.5, -1, me), "trim": None, "mixed": rng.integers(-1, B, B)}[kind]
    keep = rng.integers(-5, W * page + 40, B) if kind in ("trim", "mixed") else None
    t, r = i32(table), i32(refs)
    assert not op.fork(table, refs, page, parent, keep)
    fa.cache_fork(t, r, page, None if parent is None else i32(parent), None if keep is None else i32(keep))
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert np.array_equal(refs, np.bincount(table[table >= 0], minlength=P))
    assert fa.device_status() == fa.FA_OK


def test_fork_reverses_rows_in_a_slice_of_a_wider_table(fa):
    rng = np.random.default_rng(1)
    table, refs, _ = random_table(rng, 9, 40, 500, 16)
    whole = np.full((9, 50), 77, np.int32)
    whole[:, 5:45] = table
    t, r = i32(whole), i32(refs)
    fa.cache_fork(t[:, 5:45], r, 16, parent=i32(np.arange(9)[::-1].copy()))
    whole[:, 5:45] = table[::-1]
    assert np.array_equal(t.cpu().numpy(), whole) and np.array_equal(r.cpu().numpy(), refs)


def test_fork_out_of_range(fa):
    table, refs = np.array([[0, 9], [1, -7], [2, 3], [4, -1]], np.int32), np.array([1, 1, 1, 1, 1, 0, 0], np.int32)
    parent = np.array([0, 0, 9, -2], np.int32)
    t, r = i32(table), i32(refs)
    assert op.fork(table, refs, 16, parent)
    fa.cache_fork(t, r, 16, parent=i32(parent))
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert table.tolist() == [[0, 9], [0, -1], [2, 3], [4, -1]] and fa.device_status() == fa.FA_ERR_BAD_PAGE


# ------------------------------------------------------------------ reserve
def check_reserve(fa, caches, table, refs, page, start, count, **kw):
    t, r = i32(table), i32(refs)
    before = bits(caches)
    ok, moves, bad = op.reserve(table, refs, page, start, count)
    got = fa.cache_reserve(caches, t, r, i32(start), i32(count), **kw)
    assert np.array_equal(t.cpu().numpy(), table)
    assert np.array_equal(r.cpu().numpy(), refs)
    assert np.array_equal(got.cpu().numpy(), ok)
    assert same(caches, moved(before, moves))
    assert fa.device_status() == (fa.FA_ERR_BAD_PAGE if bad else fa.FA_OK)
    return ok, moves


@pytest.mark.parametrize("B,W,P,page,spare", [(1, 1, 2, 16, 1), (6, 9, 60, 16, 20), (64, 40, 2500, 64, 900), (40, 30, 700, 32, 0), (300, 20, 4000, 16, 30),
                                              (50, 100, 5000, 128, 60), (50, 100, 9000, 16, 30), (16384, 3, 20000, 16, 4000), (16384, 1, 8192, 16, 900), (3, 4000, 12100, 16, 9000)])
@pytest.mark.parametrize("kind", ["token", "draft", "prompt"])
def test_reserve(fa, B, W, P, page, spare, kind):
    """Rows with pages of their own and shared ones, at the start of pages and within them; enough free pages, and too few."""
    rng = np.random.default_rng(B + W + spare)
    table, refs, length = random_table(rng, B, W, max(1, P - spare), page, shared=0.6)
    refs = np.concatenate([refs, np.zeros(P - len(refs), np.int32)])
    names = rng.permutation(P).astype(np.int32)  # free pages anywhere
    table = np.where(table >= 0, names[table], -1).astype(np.int32)
    where = np.empty_like(refs)
    where[names] = refs
    refs = where
    if kind == "prompt":
        start, count = np.zeros(B, np.int64), rng.integers(-3, W * page + 9, B)
    else:
        start = np.where(rng.random(B) < 0.3, rng.integers(0, length + 1), length)  # some go back into their rows
        count = np.full(B, 1) if kind == "token" else rng.integers(0, 2 * page, B)
    caches = pools(fa, 2, P, 1, page, 64)
    check_reserve(fa, caches, table, refs, page, start, count)


@pytest.mark.parametrize("B,W,P", [(150, 64, 8192), (150, 64, 5000), (900, 50, 30000), (900, 50, 20000)])
def test_reserve_more_items_than_are_kept_on_chip(fa, B, W, P):
    """Every column of every row: some 10000 items for one CTA, 45000 for a cluster, most of them of shared pages."""
    rng = np.random.default_rng(B + P)
    page = 16
    table, refs, _ = random_table(rng, B, W, P // 3, page, shared=0.9)
    refs = np.concatenate([refs, np.zeros(P - len(refs), np.int32)])
    start, count = rng.integers(0, 20, B), np.full(B, W * page - 20)
    refs[rng.choice(np.nonzero(refs)[0], 50)] += 1    # pages that the caller holds besides
    ok, moves = check_reserve(fa, pools(fa, 1, P, 1, page, 64), table, refs, page, start, count)
    assert len(moves) > 5


def test_reserve_by_hand(fa):
    """Three rows share a partly filled page and all write on: the last one keeps it. Pages go in order."""
    caches = pools(fa, 3, 8, 2, 16, 64)
    table = np.array([[0, 5, -1], [0, 5, -1], [0, 5, -1]], np.int32)
    refs = np.array([3, 0, 0, 0, 0, 3, 0, 0], np.int32)
    ok, moves = check_reserve(fa, caches, table, refs, 16, [20, 20, 20], [1, 1, 1])
    assert table.tolist() == [[0, 1, -1], [0, 2, -1], [0, 5, -1]] and moves == [(5, 1), (5, 2)] and ok.all()
    assert refs.tolist() == [3, 1, 1, 0, 0, 1, 0, 0]


def test_reserve_without_enough_pages(fa):
    """Two free pages for three sharers and a row that needs two: who comes first is served; a row that needs none is as well."""
    caches = pools(fa, 1, 8, 1, 16, 64)
    table = np.array([[0, 5, -1], [0, 5, -1], [6, -1, -1], [0, 5, -1], [7, -1, -1]], np.int32)
    refs = np.array([4, 1, 0, 0, 1, 4, 1, 1], np.int32)   # somebody else has page 5 as well
    ok, _ = check_reserve(fa, caches, table, refs, 16, [20, 20, 16, 20, 3], [1, 1, 17, 1, 5])
    assert ok.tolist() == [1, 1, 0, 0, 1] and refs[5] == 2
    table, refs = np.array([[0], [0], [0]], np.int32), np.array([3, 1, 1, 1, 1, 1, 1, 1], np.int32)   # none at all: nothing changes
    ok, _ = check_reserve(fa, caches, table, refs, 16, [1, 1, 1], [1, 0, 1])
    assert ok.tolist() == [0, 1, 0] and refs[0] == 3
    table, refs = np.array([[0], [0], [-1]], np.int32), np.array([2, 1, 1, 1, 0, 1, 1, 1], np.int32)   # one: its sharer keeps the old page
    ok, _ = check_reserve(fa, caches, table, refs, 16, [1, 1, 0], [1, 1, 1])
    assert ok.tolist() == [1, 1, 0] and table.tolist() == [[4], [0], [-1]]


def test_reserve_rows_that_do_not_fit_and_bad_entries(fa):
    caches = pools(fa, 1, 12, 1, 16, 64)
    table = np.array([[0, 1], [2, 3], [4, -1], [99, -5], [5, -1], [-1, -1]], np.int32)
    refs = np.array([1] * 6 + [0] * 6, np.int32)
    ok, _ = check_reserve(fa, caches, table, refs, 16, [31, -1, 20, 3, 2 ** 31 - 1, 0], [2, 1, 12, 20, 2 ** 31 - 1, 0])
    assert ok.tolist() == [0, 0, 1, 1, 0, 1]


def test_reserve_without_start_one_count_and_a_workspace(fa):
    caches = pools(fa, 1, 30, 2, 32, 64)
    t, r = torch.full((5, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(30, dtype=torch.int32, device="cuda")
    ws = torch.full((fa.cache_reserve_workspace_bytes(caches[0], 5, 4),), 0xff, dtype=torch.uint8, device="cuda")
    ok = torch.empty(5, dtype=torch.int32, device="cuda")
    assert fa.cache_reserve(caches[0], t, r, None, 33, ok=ok, workspace=ws) is ok
    assert t.tolist() == [[2 * b, 2 * b + 1, -1, -1] for b in range(5)] and r.tolist() == [1] * 10 + [0] * 20 and ok.tolist() == [1] * 5


# ------------------------------------------------------------------ compact
@pytest.mark.parametrize("B,W,P,layers", [(1, 1, 1, 1), (4, 3, 2, 1), (7, 20, 200, 3), (30, 100, 5000, 1), (3, 5, 40000, 1), (200, 9, 1037, 2)])
@pytest.mark.parametrize("used", [0.0, 0.3, 1.0])
def test_compact(fa, B, W, P, layers, used):
    rng = np.random.default_rng(P + B)
    table, refs = np.full((B, W), -1, np.int32), np.zeros(P, np.int32)
    n = min(int(P * used), B * W)
    table.reshape(-1)[rng.permutation(B * W)[:n]] = rng.permutation(P)[:n]
    if n > 3:  # shared pages
        table[0, 0] = table.max()
    refs += np.bincount(table[table >= 0], minlength=P).astype(np.int32)
    if P > 20:
        refs[P - 3] += 2  # held by the caller alone
    caches = pools(fa, layers, P, 1, 16, 64)
    before, t, r = bits(caches), i32(table), i32(refs)
    held = table.copy()
    where, L, moves, _ = op.compact(table, refs)
    got, live = fa.cache_compact(caches, t, r)
    assert np.array_equal(got.cpu().numpy(), where) and live.tolist() == [L]
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert same(caches, moved(before, moves))
    assert (refs[:L] > 0).all() and not refs[L:].any() and np.array_equal(table[held >= 0], where[held[held >= 0]])
    assert fa.device_status() == fa.FA_OK


def test_compact_bad_entries_are_left(fa):
    caches = pools(fa, 1, 6, 1, 16, 64)
    table, refs = np.array([[5, 77, -1, -3]], np.int32), np.array([0, 0, 0, 0, 0, 1], np.int32)
    t, r = i32(table), i32(refs)
    where, live = fa.cache_compact(caches, t, r)
    assert t.tolist() == [[0, 77, -1, -3]] and r.tolist() == [1, 0, 0, 0, 0, 0] and where.tolist() == [-1] * 5 + [0] and live.item() == 1
    assert fa.device_status() == fa.FA_ERR_BAD_PAGE


# ------------------------------------------------------------------ streams and graphs
def test_captured_calls_follow_the_tensors(fa):
    """Fork, reserve, copy and compact in one graph, replayed with other parents, lengths and moves, on a stream of its own."""
    B, W, P, page = 8, 12, 120, 16
    rng = np.random.default_rng(3)
    caches = pools(fa, 2, P, 2, page, 64)
    table, refs, _ = random_table(rng, B, W, P // 2, page)
    refs = np.concatenate([refs, np.zeros(P - len(refs), np.int32)])
    t, r = i32(table), i32(refs)
    parent, keep, start, count, src, dst = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B, B, B, 2, 2))
    ok, where, live = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, P, 1))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (fa.cache_reserve_workspace_bytes(caches[0], B, W), fa.cache_compact_workspace_bytes(caches[0]))]

    def step():
        fa.cache_fork(t, r, page, parent=parent, keep=keep)
        fa.cache_reserve(caches, t, r, start, count, ok=ok, workspace=ws[0])
        fa.cache_copy(caches, src, dst)
        fa.cache_compact(caches, t, r, where=where, live=live, workspace=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    saved = [x.clone() for x in (t, r)]
    before = bits(caches)
    with torch.cuda.stream(side):
        src.fill_(-1)
        keep.fill_(W * page)
        parent.copy_(torch.arange(B, device="cuda"))
        step()
        with torch.cuda.graph(graph, stream=side):
            step()
        for x, y in zip((t, r), saved):
            x.copy_(y)
        for x, y in zip([x for c in caches for x in (c.k, c.v, c.k_scale, c.v_scale)], before):
            (x.view(torch.uint8) if x.dtype != torch.float32 else x).copy_(y)
        for _ in range(12):
            values = [rng.integers(-1, B, B), rng.integers(0, W * page, B), rng.integers(0, W * page, B), rng.integers(0, 40, B),
                      rng.choice(P, 2, replace=False), np.array([-1, P - 1])]
            values[4][1] = rng.choice(np.setdiff1d(np.arange(P - 1), values[4][:1]))
            for x, v in zip((parent, keep, start, count, src, dst), values):
                x.copy_(i32(v))
            graph.replay()
            op.fork(table, refs, page, values[0], values[1])
            want, moves, _ = op.reserve(table, refs, page, values[2], values[3])
            moved(before, moves)
            moved(before, [(int(values[4][1]), P - 1)])
            places, L, moves, _ = op.compact(table, refs)
            moved(before, moves)
            assert np.array_equal(ok.cpu().numpy(), want) and np.array_equal(where.cpu().numpy(), places) and live.item() == L
            assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs) and same(caches, before)
    torch.cuda.current_stream().wait_stream(side)
    assert fa.device_status() == fa.FA_OK


def test_two_tables_on_two_streams(fa):
    """Calls on streams that are not the current one, two pools at a time."""
    B, W, P, page = 20, 30, 900, 32
    rng = np.random.default_rng(4)
    streams, state = [torch.cuda.Stream() for _ in range(2)], []
    for k in range(2):
        table, refs, length = random_table(rng, B, W, P - 300, page, shared=0.7)
        refs = np.concatenate([refs, np.zeros(300, np.int32)])
        caches = pools(fa, 2, P, 1, page, 64, seed=k)
        ws = torch.empty(fa.cache_reserve_workspace_bytes(caches[0], B, W), dtype=torch.uint8, device="cuda")
        state.append([table, refs, length, caches, bits(caches), i32(table), i32(refs), ws, torch.empty(B, dtype=torch.int32, device="cuda")])
    args = [[(i32(rng.integers(0, B, B)), i32(rng.integers(0, W * page - 9, B))) for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        for s, x, a in zip(streams, state, args):
            fa.cache_fork(x[5], x[6], page, parent=a[i][0], stream=s)
            fa.cache_reserve(x[3], x[5], x[6], a[i][1], 8, ok=x[8], workspace=x[7], stream=s)
    torch.cuda.synchronize()
    for (table, refs, _, caches, before, t, r, _, ok), a in zip(state, args):
        for p, n in a:
            op.fork(table, refs, page, p.cpu().numpy())
            want, moves, _ = op.reserve(table, refs, page, n.cpu().numpy(), [8] * B)
            moved(before, moves)
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
        assert np.array_equal(ok.cpu().numpy(), want) and same(caches, before)
    assert fa.device_status() == fa.FA_OK
