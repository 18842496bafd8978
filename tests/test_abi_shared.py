"""Refusals of the attention over shared prefixes, before anything touches a GPU: fake pointers, never
dereferenced, on hosts without one (see test_abi.py); and what the binding refuses itself."""
import pytest
import torch

import exact_io_aware_11_gb300 as fa
from exact_io_aware_11_gb300 import _cache

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


def call(L, **kw):
    a = dict(ck=at(0), cv=at(1), ks=at(2), vs=at(3), P=32, H=2, page=16, cd=64, fmt=0, tab=at(4), ts=32, tw=32, kvl=at(5), ql=at(6), causal=1,
             dtype=0, scale=0.125, sq=(0, 0, 0), so=(0, 0, 0), q=at(7), o=at(8), lse=at(9), ws=at(10), wsn=1 << 24, B=4, Hq=8, N=3, of=at(11),
             pl=at(12), groups=2, cache=True, opt=True)
    a.update(kw)
    cache = bytes(_cache.CacheStruct(a["ck"], a["cv"], a["ks"], a["vs"], a["P"], a["H"], a["page"], a["cd"], a["fmt"])) if a["cache"] else None
    opt = bytes(_cache.CacheAttentionOptions(a["tab"], a["ts"], a["tw"], a["kvl"], a["ql"], a["causal"], a["dtype"], a["scale"],
                                             *a["sq"], *a["so"])) if a["opt"] else None
    return L.fa_cache_attention_shared(a["q"], a["o"], a["lse"], cache, a["B"], a["Hq"], a["N"], opt, a["of"], a["pl"], a["groups"],
                                       a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(ql=None, causal=0), OK), (dict(B=1), OK), (dict(groups=2048), OK), (dict(dtype=1, fmt=1, page=128, cd=128), OK),
    (dict(tw=1 << 20, ts=0), OK),
    (dict(cache=False), 1), (dict(opt=False), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(kvl=None), 1), (dict(tab=None), 1),
    (dict(Hq=7), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(tw=0), 1), (dict(causal=2), 1), (dict(scale=-1.0), 1), (dict(dtype=3), 2), (dict(page=8), 2),
    (dict(of=None), 1), (dict(pl=None), 1), (dict(of=at(11) + 2), 1), (dict(pl=at(12) + 1), 1), (dict(groups=0), 1), (dict(groups=2049), 1),
    (dict(tw=1 << 20, wsn=1 << 16), 1), (dict(tw=1 << 20, ws=None, wsn=0), 1), (dict(ws=at(10) + 8), 1),
    (dict(o=at(7)), 1), (dict(lse=at(8)), 1), (dict(o=at(11)), 1), (dict(lse=at(12)), 1), (dict(ws=at(11)), 1), (dict(ws=at(12)), 1),
    (dict(ws=at(7)), 1), (dict(ws=at(9)), 1), (dict(o=at(0)), 1), (dict(lse=at(5)), 1),
    (dict(of=at(5)), OK),                                     # inputs may be one tensor
])
def test_shared(L, kw, expect):
    assert call(L, **kw) == expect


def test_workspace(L):
    def need(B=4, Hq=8, N=1, tw=1 << 16, groups=2, page=16, d=64):
        c = _cache.CacheStruct(at(0), at(1), at(2), at(3), 32, 2, page, d, 0)
        return L.fa_cache_attention_shared_workspace_bytes(c, B, Hq, N, tw, groups)

    assert need() > 0 and need(groups=0) == 0 and need(groups=2049) == 0 and need(Hq=7) == 0 and need(tw=0) == 0 and need(page=8) == 0
    plain = _cache.CacheStruct(at(0), at(1), at(2), at(3), 32, 2, 16, 64, 0)
    # a table with room for few tokens, one sequence, many rows: the plain attention's
    for kw in (dict(tw=4), dict(B=1), dict(N=33)):
        a = dict(B=4, Hq=8, N=1, tw=1 << 16)
        a.update(kw)
        assert need(**kw) == L.fa_cache_attention_workspace_bytes(plain, a["B"], a["Hq"], a["N"], a["tw"])
    assert need(B=256, groups=1) > need(B=64, groups=1)


def test_the_binding_refuses():
    q, r = torch.zeros((2, 2, 1, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="KVCache"):
        fa.cache_attention_shared(q, None, r[None], r, r, r)
