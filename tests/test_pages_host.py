"""Checks of the page calls and of the shared attention that the binding makes, without a GPU."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_io_aware_11_gb300 as fa
from exact_io_aware_11_gb300 import _cache, _pages


class Reached(Exception):
    """The library was called."""


class Lib:
    def __getattr__(self, name):
        def call(*args):
            raise Reached
        return call


@pytest.fixture
def fakes(monkeypatch):
    """Fake tensors, no device, no library."""
    for module in (_cache, _pages):
        monkeypatch.setattr(module, "_on", lambda call, device, stream, *args: call(*args))
        monkeypatch.setattr(module, "lib", Lib)
        monkeypatch.setattr(module, "_raw_stream", lambda index: None)
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")  # of a fake tensor's data_ptr
        yield


def _calls(t):
    """Each call with every tensor that it takes; t(name, dtype, shape) makes one."""
    i32, bf16, u8 = torch.int32, torch.bfloat16, torch.uint8
    cache = fa.KVCache(*(torch.empty((9, 2, 16, 64), dtype=torch.int8, device="cuda:0") for _ in "kv"),
                       *(torch.empty((9, 2), device="cuda:0") for _ in "kv"))

    def table():
        return t("page_table", i32, (3, 4)), t("refs", i32, (9,))

    return [lambda: fa.cache_copy(cache, t("src", i32, (5,)), t("dst", i32, (5,))),
            lambda: fa.cache_fork(*table(), 16, t("parent", i32, (3,)), t("keep", i32, (3,))),
            lambda: fa.cache_reserve([cache], *table(), t("start", i32, (3,)), t("count", i32, (3,)), ok=t("ok", i32, (3,)),
                                     workspace=t("workspace", u8, (4096,))),
            lambda: fa.cache_compact((cache,), *table(), where=t("where", i32, (9,)), live=t("live", i32, (1,)),
                                     workspace=t("workspace", u8, (4096,))),
            lambda: fa.cache_attention_shared(t("q", bf16, (3, 4, 5, 64)), cache, t("page_table", i32, (3, 4)), t("kv_len", i32, (3,)),
                                              t("prefix_of", i32, (3,)), t("prefix_len", i32, (2,)), t("q_len", i32, (3,)),
                                              out=t("out", bf16, (3, 4, 5, 64)), lse=t("lse", torch.float32, (3, 4, 5)),
                                              workspace=t("workspace", u8, (4096,)))]


def test_tensors_on_another_device_are_refused(fakes):
    """Every tensor of every call, one at a time, on another GPU than the rest."""
    names, odd = [], None

    def make(name, dtype, shape):
        names.append(name)
        return torch.empty(shape, dtype=dtype, device="cuda:1" if name == odd else "cuda:0")

    for i, call in enumerate(_calls(make)):
        names, odd = [], None
        with pytest.raises(Reached):
            call()
        assert len(names) > 1
        for odd in list(names):
            if i == 1 and odd == "page_table":
                continue  # a fork's device is its page table's: then all the others are elsewhere
            with pytest.raises(ValueError):
                call()
    odd = "page_table"
    with pytest.raises(ValueError):
        _calls(make)[1]()


@pytest.mark.parametrize("size", [2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_a_page_size_beyond_32_bits_is_refused(fakes, size):
    t, refs, parent = (torch.zeros(s, dtype=torch.int32, device="cuda:0") for s in ((3, 4), (9,), (3,)))
    with pytest.raises(ValueError, match="page_size"):
        fa.cache_fork(t, refs, size, parent)
