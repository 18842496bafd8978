"""Attention over shared prefixes and page copies in the checked build (-DFA_CHECKS=1, device-side checks of every TMA
copy): representative calls run with it in a child process; the device status must stay clean and the
results must equal the default build's."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_cases(fa):
    """Every kernel and page size: few rows, tiles with their rows twice, of 128 rows and pairs of them."""
    out = {}
    for i, (d, page, dtype) in enumerate([(64, 16, torch.float8_e4m3fn), (128, 32, torch.int8), (64, 64, torch.int8),
                                          (128, 128, torch.float8_e4m3fn), (128, 16, torch.int8)]):
        g = torch.Generator().manual_seed(i)
        HK, pages, B = 2, 400 // page, 40
        W = (1 << 18) // page
        caches = [fa.KVCache.empty(pages + B + 40, HK, d, page, dtype) for _ in range(2)]
        refs = torch.zeros(pages + B + 40, dtype=torch.int32, device="cuda")
        table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        n = torch.tensor([400 - 5] + [0] * (B - 1), dtype=torch.int32, device="cuda")
        fa.cache_reserve(caches, table, refs, None, n)
        k, v = (torch.randn((B, HK, 400, d), generator=g).to(torch.bfloat16).cuda() for _ in "kv")
        for c in caches:
            fa.cache_write(c, k, v, table, None, n)
        fa.cache_fork(table, refs, page, parent=torch.zeros(B, dtype=torch.int32, device="cuda"))
        n[:] = n[0].clone()
        assert fa.cache_reserve(caches, table, refs, n, 3).all()
        for c in caches:
            fa.cache_write(c, k[:, :, :3], v[:, :, 3:6], table, n)
        n += 3
        res = [table, refs] + [t.view(torch.uint8) for c in caches for t in (c.k, c.v)]
        prefix = torch.tensor([395, 300, 200], dtype=torch.int32, device="cuda")
        for G, N in ((1, 1), (3, 4), (2, 30), (4, 30)):
            q = torch.randn((B, HK * G, N, d), generator=g).to(torch.bfloat16).cuda()
            for groups in (1, 3):
                of = (torch.arange(B, device="cuda") % (8 * groups) // 8).to(torch.int32)
                res += fa.cache_attention_shared(q, caches[1], table, n, of, prefix[:groups])
        _, live = fa.cache_compact(caches, table, refs)
        torch.cuda.synchronize()
        assert fa.device_status() == fa.FA_OK
        out[i] = [t.cpu() for t in res + [table, refs, live]]
    return out


CHILD = """
import sys, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {root!r} + "/tests")
from exact_io_aware_11_gb300 import _lib
_lib._LIB_PATH = {lib!r}
import exact_io_aware_11_gb300 as fa
import test_gpu_shared_checked as T
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
