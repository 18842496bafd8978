"""The README's Python examples run, one after another, and leave the device without an error."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_examples(fa):
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) == 3
    names = {}
    for b in blocks:
        exec(b, names)
        torch.cuda.synchronize()
        assert fa.device_status() == fa.FA_OK
    assert names["ok"].all() and torch.isfinite(names["lse"]).all() and names["live"].item() == int((names["refs"] > 0).sum()) == 16
