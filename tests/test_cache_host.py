"""Definitions and host-side checks of the cache's calls that need no GPU."""
import numpy as np
import pytest

from oracle import cache as oc


@pytest.mark.parametrize("fmt,top,nan", [("e4m3", 0x7e, 0x7f), ("int8", 127, 0)])
def test_definition_of_infinities_without_finite_values(fmt, top, nan):
    codes, scale = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1))
    x = np.zeros((1, 1, 2, 64))
    x[0, 0, 0, 3], x[0, 0, 1, 4] = np.inf, np.nan
    oc.write(codes, scale, x, np.array([[0]]), [0], [2], 16, fmt)
    assert codes[0, 0, 0, 3] == top and codes[0, 0, 1, 4] == nan and scale[0, 0] == 0
    assert np.count_nonzero(codes) == 1 + (nan > 0)
