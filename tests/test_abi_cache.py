"""Refusals of the rotary and cache entry points, before anything touches a GPU: fake
pointers, never dereferenced, on hosts without one (see test_abi.py)."""
import ctypes

import pytest
import torch

import exact_io_aware_11_gb300 as fa
from exact_io_aware_11_gb300 import _cache

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation tests run on CPU-only hosts")

A, SPAN = 1 << 20, 1 << 30


@pytest.fixture(scope="module")
def L():
    from exact_io_aware_11_gb300 import build
    build.build()
    return fa.lib()


def ptrs(n):
    return [A + i * SPAN for i in range(n)]


OK = 3  # past validation: no device here


def rotary(L, name="fa_rotary_fwd", **kw):
    q, qo, k, ko, turns, pos = ptrs(6)
    a = dict(q=q, qo=qo, k=k, ko=ko, B=2, Hq=4, Hk=2, N=8, d=64, r=64, inter=0, dtype=0, factor=1.0, turns=turns, pos=pos, pb=8,
             pn=1, off=0, sq=(0, 0, 0), sqo=(0, 0, 0), sk=(0, 0, 0), sko=(0, 0, 0), opt=True)
    a.update(kw)
    opt = _cache.RotaryOptions(a["r"], a["inter"], a["dtype"], a["factor"], a["turns"], a["pos"], a["pb"], a["pn"], a["off"],
                               *a["sq"], *a["sqo"], *a["sk"], *a["sko"])
    return getattr(L, name)(a["q"], a["qo"], a["k"], a["ko"], a["B"], a["Hq"], a["Hk"], a["N"], a["d"],
                            opt if a["opt"] else None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(pos=None), OK), (dict(dtype=1, inter=1, r=2), OK), (dict(k=None, ko=None, Hk=0), OK),
    (dict(qo=A), OK),                                        # in place
    (dict(qo=A + 16), 1),                                    # shifted onto its input
    (dict(ko=A + SPAN), 1),                                  # k_out on q_out
    (dict(ko=A), 1), (dict(qo=A + 2 * SPAN), 1),             # an output on the other input
    (dict(qo=A + 4 * SPAN), 1), (dict(qo=A + 5 * SPAN), 1),  # an output on the frequencies, the positions
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(Hk=0), 1), (dict(opt=False), 1),
    (dict(q=A + 8), 1), (dict(turns=None), 1), (dict(turns=A + 4), 1), (dict(pos=A + 5 * SPAN + 2), 1),
    (dict(B=0), 1), (dict(N=0), 1), (dict(Hq=0), 1), (dict(Hk=-1), 1), (dict(B=65536), 1), (dict(d=96), 2), (dict(dtype=2), 2),
    (dict(r=0), 1), (dict(r=66), 1), (dict(r=63), 1), (dict(inter=2), 1), (dict(factor=float("inf")), 1), (dict(pb=-1), 1),
    (dict(sq=(2048, 512, 60)), 1), (dict(sq=(2048, 64, 64)), 1),
    (dict(pos=None, off=2 ** 31 - 8), OK), (dict(pos=None, off=2 ** 31 - 7), 1),  # the last row's position, N = 8
    (dict(pb=2 ** 31 + 1), 1), (dict(pn=2 ** 31 + 1), 1), (dict(off=2 ** 31 - 1), OK),
])
@pytest.mark.parametrize("name", ["fa_rotary_fwd", "fa_rotary_bwd"])
def test_rotary(L, name, kw, expect):
    assert rotary(L, name, **kw) == expect


def cache_of(a):
    return _cache.CacheStruct(a["ck"], a["cv"], a["ks"], a["vs"], a["P"], a["H"], a["page"], a["cd"], a["fmt"])


def rows(L, name, **kw):
    ck, cv, ks, vs, tab, start, count, k, v = ptrs(9)
    a = dict(ck=ck, cv=cv, ks=ks, vs=vs, P=32, H=2, page=16, cd=64, fmt=0, tab=tab, ts=4, tw=4, start=start, count=count, k=k, v=v,
             B=2, N=8, dtype=0, st=(0, 0, 0), cache=True, rng=True)
    a.update(kw)
    rng = _cache.CacheRange(a["tab"], a["ts"], a["tw"], a["start"], a["count"], a["dtype"], *a["st"])
    return getattr(L, name)(cache_of(a) if a["cache"] else None, a["k"], a["v"], a["B"], a["N"], rng if a["rng"] else None, None)


COMMON = [
    (dict(), OK), (dict(start=None, count=None), OK), (dict(fmt=1, dtype=1, page=128, cd=128), OK),
    (dict(cache=False), 1), (dict(rng=False), 1), (dict(ck=None), 1), (dict(cv=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(tab=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(ck=A + 4), 1), (dict(k=A + 7 * SPAN + 2), 1),
    (dict(tab=A + 4 * SPAN + 2), 1), (dict(start=A + 5 * SPAN + 1), 1), (dict(P=0), 1), (dict(H=0), 1), (dict(B=0), 1), (dict(N=0), 1),
    (dict(tw=0), 1), (dict(ts=-1), 1), (dict(tw=1 << 28), 1), (dict(page=48), 2), (dict(page=256), 2), (dict(cd=96), 2),
    (dict(fmt=2), 2), (dict(dtype=2), 2), (dict(st=(1024, 512, 60)), 1),
    (dict(k=A), 1), (dict(v=A + 2 * SPAN), 1),               # k on the codes, v on the scales
]


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(v=A + 7 * SPAN), OK),                               # k and v may be one tensor
    (dict(cv=A), 1), (dict(ks=A), 1), (dict(vs=A + 2 * SPAN), 1),  # the pool on itself
    (dict(tab=A), 1), (dict(start=A + SPAN), 1), (dict(count=A + 3 * SPAN), 1),
])
def test_write(L, kw, expect):
    assert rows(L, "fa_cache_write", **kw) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(v=A + 7 * SPAN), 1), (dict(k=A + 4 * SPAN), 1), (dict(k=A + 5 * SPAN), 1), (dict(v=A + 6 * SPAN), 1),
])
def test_read(L, kw, expect):
    assert rows(L, "fa_cache_read", **kw) == expect


def attention(L, **kw):
    ck, cv, ks, vs, tab, kvl, ql, q, o, lse, ws = ptrs(11)
    a = dict(ck=ck, cv=cv, ks=ks, vs=vs, P=32, H=2, page=16, cd=64, fmt=0, tab=tab, ts=32, tw=32, kvl=kvl, ql=ql, causal=1, dtype=0,
             scale=0.125, sq=(0, 0, 0), so=(0, 0, 0), q=q, o=o, lse=lse, ws=ws, wsn=1 << 20, B=2, Hq=8, N=3, cache=True, opt=True)
    a.update(kw)
    opt = _cache.CacheAttentionOptions(a["tab"], a["ts"], a["tw"], a["kvl"], a["ql"], a["causal"], a["dtype"], a["scale"],
                                       *a["sq"], *a["so"])
    return L.fa_cache_attention(a["q"], a["o"], a["lse"], cache_of(a) if a["cache"] else None, a["B"], a["Hq"], a["N"],
                                opt if a["opt"] else None, a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(ql=None, causal=0), OK), (dict(ws=None, wsn=0), OK), (dict(wsn=0), OK), (dict(Hq=2), OK),
    (dict(cache=False), 1), (dict(opt=False), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(kvl=None), 1),
    (dict(tab=None), 1), (dict(Hq=7), 1), (dict(Hq=0), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(N=1 << 30), 1), (dict(tw=0), 1),
    (dict(tw=1 << 27), 1), (dict(causal=2), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=3e38), 1), (dict(dtype=3), 2),
    (dict(page=8), 2), (dict(cd=32), 2), (dict(fmt=-1), 2), (dict(ws=None), 1), (dict(ws=A + 10 * SPAN + 8), 1),
    (dict(o=A + 7 * SPAN), 1), (dict(lse=A + 8 * SPAN), 1), (dict(o=A), 1), (dict(lse=A + 4 * SPAN), 1), (dict(ws=A + 7 * SPAN), 1),
    (dict(ws=A + 9 * SPAN), 1), (dict(ws=A + SPAN), 1), (dict(o=A + 5 * SPAN), 1), (dict(lse=A + 6 * SPAN), 1),
    (dict(q=A + 7 * SPAN + 8), 1), (dict(lse=A + 9 * SPAN + 4), 1), (dict(sq=(512, 64, 60)), 1),
])
def test_attention(L, kw, expect):
    assert attention(L, **kw) == expect


def test_attention_workspace(L):
    def need(B=2, Hq=8, N=1, width=64, H=2, page=16, d=64):
        c = _cache.CacheStruct(None, None, None, None, 4, H, page, d, 0)
        return L.fa_cache_attention_workspace_bytes(c, B, Hq, N, width)
    assert need() > 0
    assert need(width=8) == 0 and need(width=32) == 0   # 512 tokens: too little to cut
    assert need(B=200, width=64) == 0           # 400 units of 1024 tokens fill the GPU whole
    assert need(Hq=7) == 0 and need(page=24) == 0 and need(width=0) == 0 and need(B=0) == 0
    # at most what a fixed number of CTAs leave behind, however long the sequences
    assert need(width=1 << 20) == need(width=1 << 22)


def test_python_refuses_cpu_tensors_and_bad_handles():
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    rot = fa.rotary_frequencies(64, device="cpu")
    with pytest.raises(ValueError):
        fa.rotary_forward(x, rot)
    codes = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        fa.KVCache(codes, codes, torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        fa.cache_attention(x, None, None, None)


def test_status_string(L):
    assert fa.FA_ERR_BAD_PAGE == 6 and fa.status_string(6) == "FA_ERR_BAD_PAGE"


def test_structs_match_the_header():
    """Field sizes by the header's order of members (no padding is left out)."""
    assert ctypes.sizeof(_cache.RotaryOptions) == 16 + 8 + 8 + 16 + 8 + 12 * 8
    assert ctypes.sizeof(_cache.CacheStruct) == 32 + 20 + 4
    assert ctypes.sizeof(_cache.CacheRange) == 8 + 8 + 8 + 16 + 8 + 24
    assert ctypes.sizeof(_cache.CacheAttentionOptions) == 8 + 8 + 8 + 16 + 16 + 48
