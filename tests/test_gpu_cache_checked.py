"""The cache's calls in the checked build (-DFA_CHECKS=1, device-side checks of every TMA copy):
representative calls run with it in a child process; the device status must stay clean and the
results must equal the default build's."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_cases(fa):
    """Writes, reads and attends over small caches of every page size; CPU copies of the results."""
    out = {}
    for i, (d, page, dtype) in enumerate([(64, 16, torch.float8_e4m3fn), (128, 32, torch.int8), (64, 64, torch.int8),
                                          (128, 128, torch.float8_e4m3fn), (128, 16, torch.int8)]):
        g = torch.Generator().manual_seed(i)
        B, HK, W = 2, 2, -(-400 // page)
        cache = fa.KVCache.empty(B * W + 1, HK, d, page, dtype)
        table = torch.randperm(B * W + 1, generator=g)[:B * W].reshape(B, W).to(torch.int32).cuda()
        n = torch.tensor([400, 131], dtype=torch.int32, device="cuda")
        k, v = (torch.randn((B, HK, 400, d), generator=g).to(torch.bfloat16).cuda() for _ in "kv")
        fa.cache_write(cache, k, v, table, None, n)
        res = list(fa.cache_read(cache, table, n, 400))
        for G, N in ((1, 1), (3, 4), (2, 30), (4, 90)):
            q = torch.randn((B, HK * G, N, d), generator=g).to(torch.bfloat16).cuda()
            res += fa.cache_attention(q, cache, table, n)
        for N in (10, 50):  # tiles with their rows twice, units of two tiles
            q = torch.randn((640, HK * 4, N, d), generator=g).to(torch.bfloat16).cuda()
            many = fa.cache_attention(q, cache, table[:1].expand(640, -1), n[:1].repeat(640))
            res += [t[::71] for t in many]
        torch.cuda.synchronize()
        assert fa.device_status() == fa.FA_OK
        out[i] = [t.cpu() for t in res]
    return out


CHILD = """
import sys, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {root!r} + "/tests")
from exact_io_aware_11_gb300 import _lib
_lib._LIB_PATH = {lib!r}
import exact_io_aware_11_gb300 as fa
import test_gpu_cache_checked as T
assert fa.lib()._name == {lib!r}
torch.save(T.run_cases(fa), {out!r})
"""


def test_checked_build_matches_default(fa, tmp_path):
    from exact_io_aware_11_gb300 import build
    lib, out = build.build(checked=True), str(tmp_path / "checked.pt")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, lib=lib, out=out)], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    checked, ref = torch.load(out), run_cases(fa)
    for i in ref:
        assert all(torch.equal(a, b) for a, b in zip(checked[i], ref[i], strict=True)), i
