"""CPU definitions of the page calls (fork, reserve, compact), entry by entry, in NumPy. Test
infrastructure: written from the definitions, with no code of the package.
"""
from __future__ import annotations

import numpy as np


def _named(entry, P):
    return 0 <= entry < P


def fork(table, refs, page, parent=None, keep=None):
    """In place; whether an entry or a parent was out of range."""
    old, P, bad = table.copy(), len(refs), False
    B, W = table.shape
    for b in range(B):
        p = b if parent is None else int(parent[b])
        if not -1 <= p < B:
            p, bad = b, True
        cols = W if keep is None else min(W, -(-max(0, int(keep[b])) // page))
        for c in range(W):
            if p == b:
                new = old[b, c] if c < cols else -1
                if c < cols:
                    continue
            else:
                new = old[p, c] if p >= 0 and c < cols else -1
                if new != -1 and not _named(new, P):
                    new, bad = -1, True
            if new == old[b, c]:
                continue
            table[b, c] = new
            if new >= 0:
                refs[new] += 1
            if _named(old[b, c], P):
                refs[old[b, c]] -= 1
            elif old[b, c] != -1:
                bad = True
    return bad


def reserve(table, refs, page, start, count):
    """In place, row by row. Returns ok, the moves [(from, to)], and whether an entry was out of range."""
    B, W = table.shape
    P, bad = len(refs), False
    free = [p for p in range(P) if refs[p] == 0]
    ok, moves, closed = np.ones(B, np.int32), [], False
    for b in range(B):
        s, n = int(start[b]), max(0, int(count[b]))
        if n == 0:
            continue
        if s < 0 or s + n > W * page:
            ok[b] = 0
            continue
        cols = range(s // page, -(-(s + n) // page))
        bad |= any(table[b, c] != -1 and not _named(table[b, c], P) for c in cols)
        r, take = refs.copy(), []  # in the order of columns: a row may name a page twice
        for c in cols:
            e = table[b, c]
            if _named(e, P) and r[e] == 1:
                continue
            if _named(e, P):
                r[e] -= 1
            take.append(c)
        if not take:
            continue
        if closed or len(take) > len(free):
            ok[b], closed = 0, True
            continue
        for c in take:
            e, new = table[b, c], free.pop(0)
            if _named(e, P):
                refs[e] -= 1
                if c == s // page and s % page:
                    moves.append((int(e), new))
            table[b, c], refs[new] = new, 1
    return ok, moves, bad


def compact(table, refs):
    """In place. Returns where, L, the moves, and whether an entry was out of range."""
    P, bad = len(refs), False
    L = int(np.count_nonzero(refs))
    where = np.array([p if refs[p] else -1 for p in range(P)], np.int32)
    holes = [p for p in range(L) if refs[p] == 0]
    moves = list(zip([p for p in range(L, P) if refs[p]], holes))
    for a, b in moves:
        where[a], refs[b], refs[a] = b, refs[a], 0
    for at, e in np.ndenumerate(table):
        if _named(e, P):
            table[at] = where[e]
        elif e != -1:
            bad = True
    return where, L, moves, bad
