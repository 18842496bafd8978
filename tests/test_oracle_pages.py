"""Pins of the page calls' definitions: small cases worked by hand, and what has to hold for any."""
import numpy as np
import pytest

from oracle import pages as op


def test_fork_by_hand():
    table, refs = np.array([[3, 1, -1], [2, -1, -1], [0, 4, 5]]), np.array([1, 1, 1, 1, 1, 1])
    assert not op.fork(table, refs, 16, parent=[0, 0, -1], keep=[48, 17, 48])
    assert table.tolist() == [[3, 1, -1], [3, 1, -1], [-1, -1, -1]] and refs.tolist() == [0, 2, 0, 2, 0, 0]
    op.fork(table, refs, 16, keep=[16, 32, 0])
    assert table.tolist() == [[3, -1, -1], [3, 1, -1], [-1, -1, -1]] and refs.tolist() == [0, 1, 0, 2, 0, 0]
    op.fork(table, refs, 16, parent=[1, 0, 2])   # rows exchanged
    assert table.tolist() == [[3, 1, -1], [3, -1, -1], [-1, -1, -1]] and refs.tolist() == [0, 1, 0, 2, 0, 0]


def test_reserve_by_hand():
    table, refs = np.array([[3, 1, -1], [3, 1, -1], [-1, -1, -1]]), np.array([0, 2, 0, 2, 0, 0])
    ok, moves, bad = op.reserve(table, refs, 16, start=[20, 32, 0], count=[13, 1, 1])
    assert table.tolist() == [[3, 0, 2], [3, 1, 4], [5, -1, -1]] and moves == [(1, 0)] and ok.tolist() == [1, 1, 1] and not bad
    assert refs.tolist() == [1, 1, 1, 2, 1, 1]
    ok, moves, _ = op.reserve(table, refs, 16, start=[0, 32, 16], count=[48, 16, 1])   # page 3 is shared, none is free
    assert ok.tolist() == [0, 1, 0] and not moves and table.tolist() == [[3, 0, 2], [3, 1, 4], [5, -1, -1]]


def test_compact_by_hand():
    table, refs = np.array([[5, 1], [5, 3], [-1, -1]]), np.array([0, 1, 0, 1, 0, 2])
    where, L, moves, _ = op.compact(table, refs)
    assert L == 3 and moves == [(3, 0), (5, 2)] and where.tolist() == [-1, 1, -1, 0, -1, 2]
    assert table.tolist() == [[2, 1], [2, 0], [-1, -1]] and refs.tolist() == [1, 1, 2, 0, 0, 0]


@pytest.mark.parametrize("seed", range(30))
def test_counts_and_contents_over_a_run(seed):
    """A run of calls: the counts stay those of the table, no row that is written shares the page it is written to, and
    every row's tokens are those that were written to it."""
    rng = np.random.default_rng(seed)
    B, W, P, page = 6, 8, 30, 16
    table, refs = np.full((B, W), -1), np.zeros(P, np.int64)
    content, length, said = np.full((P, page), -1), np.zeros(B, np.int64), [[] for _ in range(B)]
    token = 0
    for _ in range(60):
        parent, keep = np.arange(B), np.full(B, W * page)
        b = int(rng.integers(0, B))
        parent[b] = int(rng.integers(-1, B))
        if rng.random() < 0.5:
            keep[b] = int(rng.integers(0, W * page))
        new = length[parent[b]] if parent[b] >= 0 else 0
        said[b] = (said[parent[b]] if parent[b] >= 0 else [])[:keep[b]]
        length[b] = min(new, keep[b])
        op.fork(table, refs, page, parent, keep)
        count = rng.integers(0, 20, B) * (rng.random(B) < 0.6)
        ok, moves, _ = op.reserve(table, refs, page, length, count)
        for s, d in moves:
            content[d] = content[s]
        for b in range(B):
            if ok[b]:
                for n in range(int(count[b])):
                    p = table[b, length[b] // page]
                    assert refs[p] == 1
                    content[p, length[b] % page] = token
                    said[b] = said[b] + [token]
                    token += 1
                    length[b] += 1
        if rng.random() < 0.2:
            where, L, moves, _ = op.compact(table, refs)
            for s, d in moves:
                content[d] = content[s]
            assert (refs[:L] > 0).all() and not refs[L:].any()
        assert np.array_equal(refs, np.bincount(table[table >= 0], minlength=P))
        for b in range(B):
            assert [content[table[b, t // page], t % page] for t in range(length[b])] == said[b]
