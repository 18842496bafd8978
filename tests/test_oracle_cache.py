"""Pins of the fp64 definitions in oracle/cache.py, and the host side of the rotary
frequencies and the cache handle (no GPU)."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_11_gb300 as fa
from oracle import attention as oracle_attention  # noqa: F401
from oracle import cache as oc


def test_e4m3_values_match_torch():
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    got = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, oc.e4m3_values(), equal_nan=True)


def test_encode_matches_torch_on_ties_and_edges():
    pos = oc.e4m3_values()[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), [448.0, 2.0 ** -10, 2.0 ** -11]])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float32)
    same = want.double().numpy() == x      # values fp32 holds
    assert same.sum() > 500
    got = oc.encode(x, "e4m3")
    assert np.array_equal(got[same], want.to(torch.float8_e4m3fn).view(torch.uint8).numpy()[same])
    assert oc.encode(np.array([1e9, -np.inf, np.nan]), "e4m3").tolist() == [0x7e, 0xfe, 0x7f]
    assert oc.encode(np.array([2.5, 3.5, -0.5, 200.0, np.nan]), "int8").view(np.int8).tolist() == [2, 4, 0, 127, 0]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_smallest_power_of_two(fmt):
    for a in (1e-30, 0.1, 1.0, oc.QMAX[fmt], oc.QMAX[fmt] * 1.0001, 3e38):
        s = oc.scale_for(a, fmt)
        assert math.frexp(s)[0] == 0.5 and a <= s * oc.QMAX[fmt]
        assert s == 2.0 ** -126 or a > s / 2 * oc.QMAX[fmt]
    assert oc.scale_for(0.0, fmt) == 0.0


def test_write_moves_older_rows_when_the_scale_grows():
    codes, scale = np.zeros((2, 1, 16, 64), np.uint8), np.zeros((2, 1))
    table = np.array([[1]])
    x = np.full((1, 1, 1, 64), 0.5)
    oc.write(codes, scale, x, table, [0], [1], 16, "e4m3")
    oc.write(codes, scale, x * 1024, table, [1], [1], 16, "e4m3")
    got = oc.sequence(codes, scale, table[0], 16, "e4m3", 0, 2)
    assert np.array_equal(got[0, 0], np.full(64, 0.5)) and np.array_equal(got[0, 1], np.full(64, 512.0))
    assert not codes[0].any() and not codes[1, 0, 2:].any()


def test_rotate_is_an_isometry_and_its_own_inverse():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 64))
    pos = np.array([[0, 1, 2, 1000, -7], [5, 6, 7, 8, 2 ** 30]])
    for inter in (False, True):
        for r in (64, 20, 2):
            w = 10000.0 ** (-2 * np.arange(r // 2) / r)
            y = oc.rotate(x, w, pos, 1.0, inter)
            assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
            assert np.allclose(oc.rotate(y, w, pos, 1.0, inter, back=True), x, atol=1e-12)
            assert np.array_equal(y[..., r:], x[..., r:])
    # scores of rotated rows depend on the distance alone
    w = 10000.0 ** (-2 * np.arange(32) / 64)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    dot = lambda a, b: (oc.rotate(q, w, np.array([[a]]), 1, False) * oc.rotate(k, w, np.array([[b]]), 1, False)).sum()  # noqa: E731
    assert abs(dot(10, 3) - dot(1010, 1003)) < 1e-9


def test_attend_matches_the_dense_oracle():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 2, 9, 64))
    see = np.tril(np.ones((9, 9), bool))
    o, lse, mag, big = oc.attend(q, k, v, 0.125, see)
    o2, lse2 = oracle_attention.forward(*(t[None] for t in (q, k, v)), 0.125, causal=True)
    assert np.allclose(o, o2[0], atol=1e-12) and np.allclose(lse, lse2[0], atol=1e-12)
    assert np.all(mag >= np.abs(o) - 1e-12) and np.all(big > 0)
    o, lse, _, _ = oc.attend(q, k, v, 0.125, np.zeros((9, 9), bool))
    assert not o.any() and np.all(np.isneginf(lse))


# ------------------------------------------------------------------ frequencies and handles
def _angles_back(rot):
    """Radians per position from the 64-bit fractions of a turn."""
    return np.array([(t & (2 ** 64 - 1)) / 2.0 ** 64 * 2 * math.pi for t in rot.turns.tolist()])


@pytest.mark.parametrize("r", [2, 20, 64, 128])
def test_frequencies_unscaled(r):
    rot = fa.rotary_frequencies(r, device="cpu")
    want = 10000.0 ** (-2 * np.arange(r // 2) / r)
    assert np.allclose(_angles_back(rot), want, rtol=1e-13) and rot.factor == 1.0 and rot.rotary_dim == r


def test_frequencies_scaled():
    r = 64
    w = 10000.0 ** (-2 * np.arange(r // 2) / r)
    lin = fa.rotary_frequencies(r, scaling="linear", factor=8.0, device="cpu")
    assert np.allclose(_angles_back(lin), w / 8, rtol=1e-13)
    ntk = _angles_back(fa.rotary_frequencies(r, scaling="ntk", factor=8.0, device="cpu"))
    assert np.isclose(ntk[0], 1.0) and np.isclose(ntk[-1], w[-1] / 8, rtol=1e-12)
    rot = fa.rotary_frequencies(r, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    y = _angles_back(rot)
    turns = 4096 * w / (2 * math.pi)
    assert np.allclose(y[turns > 40], w[turns > 40], rtol=1e-12)
    assert np.allclose(y[turns < 0.7], w[turns < 0.7] / 4, rtol=1e-12)
    assert np.all(y <= w * (1 + 1e-12)) and np.all(y >= w / 4 * (1 - 1e-12))
    assert math.isclose(rot.factor, 0.1 * math.log(4.0) + 1.0)


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=64, scaling="other"),
                                dict(rotary_dim=64, base=0.0), dict(rotary_dim=64, scaling="linear", factor=float("nan")),
                                dict(rotary_dim=64, scaling="yarn", factor=4.0), dict(rotary_dim=2, scaling="ntk", factor=2.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        fa.rotary_frequencies(device="cpu", **kw)


def test_turns_of_far_positions_are_exact():
    rot = fa.rotary_frequencies(64, device="cpu")
    for t, a in zip(rot.turns.tolist(), rot.angles.tolist()):
        for p in (1, 131071, 2 ** 30):
            got = ((t * p) % 2 ** 64) / 2.0 ** 64
            want = math.fmod(p * (a / (2 * math.pi)), 1.0)
            d = abs(got - want)
            assert min(d, 1 - d) <= p * 2.0 ** -52
