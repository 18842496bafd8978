"""Definitions and host-side checks of the cache's calls that need no GPU."""
import os
import warnings

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_io_aware_11_gb300 as fa
from exact_io_aware_11_gb300 import _cache
from oracle import cache as oc


@pytest.mark.parametrize("fmt,top,nan", [("e4m3", 0x7e, 0x7f), ("int8", 127, 0)])
def test_definition_of_infinities_without_finite_values(fmt, top, nan):
    codes, scale = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1))
    x = np.zeros((1, 1, 2, 64))
    x[0, 0, 0, 3], x[0, 0, 1, 4] = np.inf, np.nan
    oc.write(codes, scale, x, np.array([[0]]), [0], [2], 16, fmt)
    assert codes[0, 0, 0, 3] == top and codes[0, 0, 1, 4] == nan and scale[0, 0] == 0
    assert np.count_nonzero(codes) == 1 + (nan > 0)


class Reached(Exception):
    """The library was about to be called."""


def _calls(t, rot):
    """Each entry point's call with every tensor that it takes; t(name, dtype, shape) makes one."""
    bf16, i32 = torch.bfloat16, torch.int32
    codes = [torch.empty((9, 2, 16, 64), dtype=torch.int8, device="cuda:0") for _ in "kv"]
    cache = fa.KVCache(*codes, *(torch.empty((9, 2), device="cuda:0") for _ in "kv"))
    q, kv = (3, 4, 5, 64), (3, 2, 5, 64)

    def rotary(f):
        rot.turns = t("turns", torch.int64, (32,))
        return f(torch.empty(q, dtype=bf16, device="cuda:0"), rot, t("k", bf16, kv), t("positions", i32, (5,)), out=t("out", bf16, q),
                 k_out=t("k_out", bf16, kv))

    def table():
        return t("page_table", i32, (3, 4))

    return [lambda: rotary(fa.rotary_forward), lambda: rotary(fa.rotary_backward),
            lambda: fa.cache_write(cache, t("k", bf16, kv), t("v", bf16, kv), table(), t("start", i32, (3,)), t("count", i32, (3,))),
            lambda: fa.cache_read(cache, table(), t("count", i32, (3,)), 5, t("start", i32, (3,)), k_out=t("k_out", bf16, kv),
                                  v_out=t("v_out", bf16, kv)),
            lambda: fa.cache_attention(t("q", bf16, q), cache, table(), t("kv_len", i32, (3,)), t("q_len", i32, (3,)),
                                       out=t("out", bf16, q), lse=t("lse", torch.float32, q[:3]),
                                       workspace=t("workspace", torch.uint8, (4096,))),
            lambda: fa.cache_attention(t("q", bf16, q), cache, table(), t("kv_len", i32, (3,)), split=False)]  # outputs made by the call


def test_tensors_on_another_device_are_refused(monkeypatch):
    """Every tensor of every call, one at a time, on another GPU than the rest (fake tensors: no GPU is touched)."""
    class Lib:
        def __getattr__(self, name):
            raise Reached

    monkeypatch.setattr(_cache, "_on", lambda call, device, stream, *args: call(*args))
    monkeypatch.setattr(_cache, "lib", Lib)
    names, odd, rot = [], None, fa.rotary_frequencies(64, device="cpu")

    def make(name, dtype, shape):
        names.append(name)
        return torch.empty(shape, dtype=dtype, device="cuda:1" if name == odd else "cuda:0")

    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")  # of a fake tensor's data_ptr
        for call in _calls(make, rot):
            names, odd = [], None
            with pytest.raises(Reached):
                call()
            assert len(names) > 2
            for odd in list(names):
                with pytest.raises(ValueError):
                    call()


def test_split_false_uses_no_workspace(monkeypatch):
    """Neither one that the caller gives nor one of its own."""
    given = []

    class Lib:
        fa_cache_attention_workspace_bytes = staticmethod(lambda *a: 512)
        fa_cache_attention = staticmethod(lambda *a: given.append(a[9]) or 0)  # workspace_bytes

    monkeypatch.setattr(_cache, "_on", lambda call, device, stream, *args: call(*args))
    monkeypatch.setattr(_cache, "_raw_stream", lambda index: None)
    monkeypatch.setattr(_cache, "lib", Lib)
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")  # of a fake tensor's data_ptr
        t = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda:0")  # noqa: E731
        cache = fa.KVCache(*(t((9, 2, 16, 64), torch.int8) for _ in "kv"), *(t((9, 2), torch.float32) for _ in "kv"))
        for ws, split in ((None, True), (t((700,), torch.uint8), True), (None, False), (t((700,), torch.uint8), False)):
            fa.cache_attention(t((3, 4, 5, 64), torch.bfloat16), cache, t((3, 4), torch.int32), t((3,), torch.int32), workspace=ws, split=split)
    assert given == [512, 700, 0, 0]


def test_kernels_of_dependent_launches_read_coherently():
    """These kernels may be set up while their predecessor on the stream (a write before a read, a
    rotation in place before a write) still runs: what it writes is not read-only for their lifetime, as the
    non-coherent load (__ldg, ld.global.nc) demands."""
    csrc = os.path.join(os.path.dirname(fa.__file__), "csrc")
    names = sorted(n for n in os.listdir(csrc) if n.startswith(("fa_cache", "fa_rotary")))
    assert len(names) >= 9
    for n in names:
        with open(os.path.join(csrc, n)) as f:
            text = f.read()
        assert "__ldg" not in text and ".global.nc" not in text and "__restrict__" not in text, n
