"""Overlaps of the rotary call's tensors, refused exactly: q, k and v may be views of one packed
projection [B, N, Hq + 2 Hk, d] and be rotated in place. Fake pointers, never dereferenced, on hosts
without a GPU (see test_abi.py)."""
import itertools
import random

import pytest

from test_abi_cache import A, OK, L, pytestmark, rotary  # noqa: F401


def packed(Hq, Hk, N=8, d=64, B=2, **kw):
    """In-place rotation of q and k of a packed buffer; sizes of bytes from A."""
    row = (Hq + 2 * Hk) * d
    st = (N * row, d, row)
    a = dict(q=A, qo=A, k=A + 2 * Hq * d, ko=A + 2 * Hq * d, Hq=Hq, Hk=Hk, N=N, d=d, B=B, sq=st, sqo=st, sk=st, sko=st)
    a.update(kw)
    return a


@pytest.mark.parametrize("name", ["fa_rotary_fwd", "fa_rotary_bwd"])
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (4, 2), (8, 1), (1, 1), (2, 6)])
def test_in_place_on_a_packed_projection(L, name, Hq, Hk):  # noqa: F811
    d = 64
    assert rotary(L, name, **packed(Hq, Hk)) == OK
    assert rotary(L, name, **packed(Hq, Hk, N=1)) == OK
    assert rotary(L, name, **packed(Hq, Hk, B=1)) == OK
    last = A + 2 * (Hq - 1) * d                                       # q's last head
    assert rotary(L, name, **packed(Hq, Hk, k=last, ko=last)) == 1
    assert rotary(L, name, **packed(Hq, Hk, ko=last)) == 1
    assert rotary(L, name, **packed(Hq, Hk, ko=A + 2 * Hq * d + 16)) == 1   # k shifted onto itself
    assert rotary(L, name, **packed(Hq, Hk, ko=A + 2 * (Hq + Hk) * d)) == OK  # k into v's place
    assert rotary(L, name, **packed(Hq, Hk, ko=A + 2 * (Hq + Hk) * d + 16)) == 1  # onto the next row's q


def test_overlaps_by_counting(L):  # noqa: F811
    """Random views against the sets of their elements' places (in units of 8 elements)."""
    rng = random.Random(5)
    met = 0
    for _ in range(3000):
        B, Hq, Hk, N, u = rng.choice((1, 2)), rng.choice((1, 2, 3)), rng.choice((1, 2, 3)), rng.choice((1, 2, 3)), 8
        H = max(Hq, Hk)
        pad = [rng.choice((0, 0, 1, 3, 8, 17)) for _ in range(3)]
        order = rng.choice(list(itertools.permutations("bhn")))
        size, st = dict(b=B, h=H, n=N), {}
        step = u + pad[0]
        for i, ax in enumerate(order):
            st[ax] = step
            step = step * size[ax] + (pad[i + 1] if i < 2 else 0)
        stride = tuple(8 * st[a] for a in "bhn")

        def places(at, heads):
            return {at + b * st["b"] + h * st["h"] + n * st["n"] + c  # noqa: B023
                    for b in range(B) for h in range(heads) for n in range(N) for c in range(u)}  # noqa: B023

        at = rng.randrange(0, 2 * step)
        q, k = places(0, Hq), places(at, Hk)
        far = A + (1 << 26)
        got = rotary(L, q=far, qo=A, k=far + (1 << 26), ko=A + 16 * at, B=B, Hq=Hq, Hk=Hk, N=N, d=64, sq=stride, sqo=stride, sk=stride,
                     sko=stride, turns=far + (1 << 28), pos=None)
        assert got == (1 if q & k else OK), (B, Hq, Hk, N, st, at)
        met += bool(q & k)
    assert 300 < met < 2700
