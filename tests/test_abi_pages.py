"""Refusals of the page calls, before anything touches a GPU: fake pointers, never
dereferenced, on hosts without one (see test_abi.py); and what the binding refuses itself."""
import pytest
import torch

import exact_io_aware_11_gb300 as fa
from exact_io_aware_11_gb300 import _cache, _pages

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation tests run on CPU-only hosts")

A, SPAN = 1 << 20, 1 << 30
OK = 3  # past validation: no device here


@pytest.fixture(scope="module")
def L():
    from exact_io_aware_11_gb300 import build
    build.build()
    return fa.lib()


def at(i):
    return A + i * SPAN


def layers_of(a):
    pools = []
    for l in range(a["layers"]):
        c = dict(k=at(20 + 4 * l), v=at(21 + 4 * l), ks=at(22 + 4 * l), vs=at(23 + 4 * l), P=32, H=2, page=16, d=64, fmt=0)
        if l == a["layer"]:
            c.update(a["cache"])
        pools.append(_cache.CacheStruct(c["k"], c["v"], c["ks"], c["vs"], c["P"], c["H"], c["page"], c["d"], c["fmt"]))
    return b"".join(bytes(p) for p in pools) if a["pools"] else None


def table_of(a):
    return bytes(_pages.PageTableStruct(a["tab"], a["ts"], a["rows"], a["tw"], a["refs"], a["P"], a["page"])) if a["table"] else None


BASE = dict(layers=2, layer=1, cache={}, pools=True, n_layers=None, src=at(0), dst=at(1), n=5, tab=at(2), ts=8, rows=4, tw=8, refs=at(3),
            P=32, page=16, table=True, parent=at(4), keep=at(5), start=at(6), count=at(7), tokens=0, ok=at(8), where=at(9),
            live=at(10), ws=at(11), wsn=1 << 20)


def call(L, name, kw):
    a = dict(BASE)
    a.update(kw)
    n = a["layers"] if a["n_layers"] is None else a["n_layers"]
    if name == "copy":
        return L.fa_cache_copy(layers_of(a), n, a["src"], a["dst"], a["n"], None)
    if name == "fork":
        return L.fa_cache_fork(table_of(a), a["parent"], a["keep"], None)
    if name == "reserve":
        return L.fa_cache_reserve(layers_of(a), n, table_of(a), a["start"], a["count"], a["tokens"], a["ok"], a["ws"], a["wsn"], None)
    return L.fa_cache_compact(layers_of(a), n, table_of(a), a["where"], a["live"], a["ws"], a["wsn"], None)


LAYERS = [
    (dict(), OK), (dict(layers=1, layer=0), OK), (dict(layers=70), OK), (dict(pools=False), 1), (dict(n_layers=0), 1), (dict(n_layers=-1), 1),
    (dict(n_layers=1025), 1), (dict(cache=dict(k=None)), 1), (dict(cache=dict(vs=None)), 1), (dict(cache=dict(v=at(30) + 8)), 1),
    (dict(cache=dict(ks=at(30) + 2)), 1), (dict(cache=dict(H=3)), 1), (dict(cache=dict(P=33)), 1), (dict(cache=dict(page=32)), 1),
    (dict(cache=dict(d=128)), 1), (dict(cache=dict(fmt=1)), 1), (dict(cache=dict(page=48)), 2), (dict(cache=dict(d=96)), 2),
    (dict(cache=dict(fmt=2)), 2), (dict(cache=dict(P=0)), 1),
    (dict(cache=dict(k=at(20))), 1), (dict(cache=dict(v=at(20) + 16)), 1), (dict(cache=dict(vs=at(22) + 4)), 1),  # layers that share memory
    (dict(cache=dict(v=at(24))), 1),
]
TABLE = [
    (dict(table=False), 1), (dict(tab=None), 1), (dict(refs=None), 1), (dict(tab=at(2) + 2), 1), (dict(refs=at(3) + 1), 1), (dict(rows=0), 1),
    (dict(rows=16385), 1), (dict(tw=0), 1), (dict(ts=7), 1), (dict(ts=-8), 1), (dict(rows=1, ts=0), OK), (dict(ts=1 << 41), 1),
    (dict(rows=16384, tw=1 << 17, ts=1 << 17), 1), (dict(rows=1, tw=1 << 27, ts=1 << 27), 1), (dict(P=0), 1), (dict(page=8), 2),
    (dict(refs=at(2) + 64), 1),                               # the counts on the table
]


@pytest.mark.parametrize("kw,expect", LAYERS + [
    (dict(n=0), 0), (dict(n=0, src=None, dst=None), 0), (dict(n=-1), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(src=at(0) + 2), 1),
    (dict(dst=at(0)), OK),                                    # pages onto themselves: nothing to do, on the device
    (dict(src=at(20)), 1), (dict(dst=at(26)), 1),             # the lists on the pools
])
def test_copy(L, kw, expect):
    assert call(L, "copy", kw) == expect


@pytest.mark.parametrize("kw,expect", TABLE + [
    (dict(), OK), (dict(keep=None), OK), (dict(parent=None), OK), (dict(parent=None, keep=None), 1), (dict(parent=at(4) + 2), 1),
    (dict(parent=at(2)), 1), (dict(keep=at(3)), 1), (dict(parent=at(5)), OK),
])
def test_fork(L, kw, expect):
    assert call(L, "fork", kw) == expect


BOTH = LAYERS + [x for x in TABLE if x[0].get("P", 32) == 32] + [
    (dict(P=31), 1), (dict(page=32), 1),                      # another pool than the table's
    (dict(ws=None), 1), (dict(ws=at(11) + 8), 1), (dict(wsn=300), 1), (dict(ws=at(2)), 1), (dict(ws=at(3)), 1), (dict(ws=at(25)), 1),
    (dict(tab=at(20)), 1), (dict(refs=at(27)), 1),
]


@pytest.mark.parametrize("kw,expect", BOTH + [
    (dict(start=None), OK), (dict(count=None, tokens=7), OK), (dict(tokens=-1), 1), (dict(ok=None), 1), (dict(ok=at(8) + 2), 1),
    (dict(ok=at(2)), 1), (dict(ok=at(3)), 1), (dict(ok=at(6)), 1), (dict(ok=at(7) + 4), 1), (dict(start=at(3)), 1), (dict(count=at(11)), 1),
    (dict(ok=at(21)), 1), (dict(start=at(22)), 1), (dict(count=at(6)), OK),
])
def test_reserve(L, kw, expect):
    assert call(L, "reserve", kw) == expect


@pytest.mark.parametrize("kw,expect", BOTH + [
    (dict(where=None), 1), (dict(live=None), 1), (dict(where=at(9) + 1), 1), (dict(live=at(9)), 1), (dict(where=at(2)), 1), (dict(live=at(3) + 8), 1),
    (dict(where=at(11)), 1), (dict(where=at(24)), 1), (dict(live=at(23)), 1),
])
def test_compact(L, kw, expect):
    assert call(L, "compact", kw) == expect


def test_workspace_sizes(L):
    assert L.fa_cache_reserve_workspace_bytes(1, 1, 1) > 0
    assert L.fa_cache_reserve_workspace_bytes(0, 1, 1) == 0 and L.fa_cache_reserve_workspace_bytes(16385, 1, 1) == 0
    assert L.fa_cache_reserve_workspace_bytes(16384, 1 << 16, 100) < 16384 * 8 + 2048  # the list of pages ends with the pool
    assert L.fa_cache_compact_workspace_bytes(0) == 0 and L.fa_cache_compact_workspace_bytes(7) > 0


def test_the_binding_refuses_other_tensors():
    t, r = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="page_table"):
        fa.cache_fork(t, r, 16, parent=r)
    for bad in (None, [], [1], t):
        with pytest.raises(ValueError, match="caches"):
            fa.cache_copy(bad, r, r)
        with pytest.raises(ValueError, match="caches"):
            fa.cache_reserve(bad, t, r, r, 1)
        with pytest.raises(ValueError, match="caches"):
            fa.cache_compact(bad, t, r)
