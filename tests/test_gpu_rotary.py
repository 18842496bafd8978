"""Rotary positions against their fp64 definition (oracle/cache.py).

Bound of an output y of the pair (a, b): half a step of its type (eps / 2 of |y|, and half the
smallest subnormal), plus what fp32 leaves before it: the angle is off by at most 2^-25 half
turns (pi 2^-25 < 2^-23), sine and cosine by 2 ulp (2^-23), products and sum by three
roundings (3 * 2^-24): together less than (|a| + |b|) factor 2^-21.
"""
import numpy as np
import pytest
import torch

from _util import f64
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


def make(shape, dt, seed, storage="bhnd"):
    B, H, N, d = shape
    g = torch.Generator().manual_seed(seed)
    if storage == "bhnd":
        return torch.randn(shape, generator=g).to(DT[dt]).cuda()
    if storage == "bnhd":
        return torch.randn((B, N, H, d), generator=g).to(DT[dt]).cuda().transpose(1, 2)
    return torch.randn((B, N, 3, H, d), generator=g).to(DT[dt]).cuda()[:, :, 1].transpose(1, 2)  # a slice of a packed tensor


def check(y, x, rot, pos, dt, back=False, tag=""):
    want = oc.rotate(f64(x), rot.angles.numpy(), np.broadcast_to(pos, (x.shape[0], x.shape[2])), rot.factor, rot.interleaved, back)
    r = rot.rotary_dim
    xa = np.abs(f64(x))
    mag = np.zeros_like(xa)
    if rot.interleaved:
        s = xa[..., 0:r:2] + xa[..., 1:r:2]
        mag[..., 0:r:2] = mag[..., 1:r:2] = s
    else:
        s = xa[..., :r // 2] + xa[..., r // 2:r]
        mag[..., :r // 2] = mag[..., r // 2:r] = s
    tol = torch.finfo(DT[dt]).eps / 2 * np.abs(want) * (1 + 2.0 ** -10) + mag * rot.factor * 2.0 ** -21 + TINY[dt]
    err = np.abs(f64(y) - want)
    assert np.all(err <= tol), f"{tag} off by {np.max(err / tol):.2f} bounds"
    assert np.array_equal(f64(y)[..., r:], f64(x)[..., r:])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,HK,N,d,r,storage", [
    (1, 1, 1, 1, 64, 64, "bhnd"), (3, 4, 2, 7, 64, 64, "bnhd"), (2, 5, 1, 33, 128, 128, "packed"), (2, 3, 3, 5, 128, 64, "bnhd"),
    (1, 2, 1, 9, 64, 20, "bhnd"), (2, 2, 2, 4, 128, 2, "packed"), (1, 3, 2, 130, 64, 48, "bnhd"), (2, 16, 4, 600, 128, 96, "bhnd"),
    # several heads to a thread, their number not a multiple of it
    (2, 16, 3, 2100, 128, 96, "bhnd"), (2, 13, 2, 2100, 128, 128, "bnhd"), (1, 13, 2, 1500, 64, 20, "bnhd"),
    (2, 5, 2, 40, 128, 100, "packed"), (1, 11, 1, 70, 64, 62, "bnhd"), (3, 1, 1, 5, 128, 126, "bhnd"), (2, 4, 4, 9, 64, 34, "bhnd"),
    (2, 13, 2, 2100, 128, 100, "bnhd"), (4, 30, 3, 1100, 64, 62, "bhnd"),
])
def test_forward_and_backward(fa, B, H, HK, N, d, r, storage, interleaved, dt):
    rot = fa.rotary_frequencies(r, interleaved=interleaved)
    q, k = make((B, H, N, d), dt, 1, storage), make((B, HK, N, d), dt, 2, storage)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-50, 131072, (B, N), generator=g, dtype=torch.int32)
    y, z = fa.rotary_forward(q, rot, k=k, positions=pos.cuda())
    check(y, q, rot, pos.numpy(), dt, tag="q")
    check(z, k, rot, pos.numpy(), dt, tag="k")
    dq, dk = fa.rotary_backward(q, rot, dk=k, positions=pos.cuda())
    check(dq, q, rot, pos.numpy(), dt, back=True, tag="dq")
    check(dk, k, rot, pos.numpy(), dt, back=True, tag="dk")


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_scaled_frequencies(fa, scaling):
    rot = fa.rotary_frequencies(64, scaling=scaling, factor=4.0, original_length=4096)
    q = make((2, 3, 40, 64), "fp16", 4)
    pos = torch.arange(16000, 16040, dtype=torch.int32)
    check(fa.rotary_forward(q, rot, positions=pos.cuda()), q, rot, pos.numpy()[None], "fp16")
    check(fa.rotary_backward(q, rot, positions=pos.cuda()), q, rot, pos.numpy()[None], "fp16", back=True)


@pytest.mark.parametrize("first", [0, 5, -3, 2 ** 20, 2 ** 30])
def test_offset_and_far_positions(fa, first):
    rot = fa.rotary_frequencies(128)
    q = make((2, 2, 6, 128), "fp16", 5)
    pos = np.arange(first, first + 6)[None]
    a = fa.rotary_forward(q, rot, offset=first)
    check(a, q, rot, pos, "fp16")
    b = fa.rotary_forward(q, rot, positions=torch.from_numpy(pos[0].astype(np.int32)).cuda())
    assert torch.equal(a, b)


def test_position_strides(fa):
    rot = fa.rotary_frequencies(64)
    q = make((3, 2, 4, 64), "bf16", 6)
    wide = torch.randint(0, 1000, (4, 3), dtype=torch.int32, generator=torch.Generator().manual_seed(7)).cuda()
    pos = wide.t()                                            # [3, 4], strides (1, 3)
    assert torch.equal(fa.rotary_forward(q, rot, positions=pos), fa.rotary_forward(q, rot, positions=pos.contiguous()))


@pytest.mark.parametrize("interleaved,r", [(False, 64), (False, 20), (True, 36)])
def test_in_place(fa, interleaved, r):
    rot = fa.rotary_frequencies(r, interleaved=interleaved)
    q, k = make((2, 4, 9, 64), "bf16", 8, "packed"), make((2, 2, 9, 64), "bf16", 9, "bnhd")
    y, z = fa.rotary_forward(q, rot, k=k, offset=3)
    y2, z2 = fa.rotary_forward(q, rot, k=k, offset=3, out=q, k_out=k)
    assert y2.data_ptr() == q.data_ptr() and torch.equal(y, q) and torch.equal(z, k)


def test_gradient_is_the_transpose_and_matches_differences(fa):
    """<dy, R x> = <R' dy, x>: fp16 rounds each side's elements by 2^-11, so the sums of n
    products differ by at most 2 * 2^-11 * sum |dy| |x| * 2; and R is linear, so a difference
    quotient along v is R v itself."""
    rot = fa.rotary_frequencies(48, scaling="yarn", factor=2.0, original_length=64)
    x, dy = make((2, 3, 11, 64), "fp16", 10), make((2, 3, 11, 64), "fp16", 11)
    y, dx = fa.rotary_forward(x, rot), fa.rotary_backward(dy, rot)
    lhs, rhs = (f64(dy) * f64(y)).sum(), (f64(dx) * f64(x)).sum()
    norms = np.linalg.norm(f64(dy)) * np.linalg.norm(f64(x)) * rot.factor
    assert abs(lhs - rhs) <= 2 * 2.0 ** -11 * norms
    # differences of L(x) = <dy, R x> (fp64 definition) against the kernel's gradient
    pos = np.broadcast_to(np.arange(11), (2, 11))
    loss = lambda a: (f64(dy) * oc.rotate(a, rot.angles.numpy(), pos, rot.factor, False)).sum()  # noqa: E731
    for at in [(0, 0, 0, 0), (1, 2, 10, 23), (0, 1, 5, 47), (1, 0, 3, 60)]:
        e = np.zeros(x.shape)
        e[at] = 0.5
        d = loss(f64(x) + e) - loss(f64(x) - e)
        assert abs(d - f64(dx)[at]) <= 2.0 ** -11 * abs(d) + 2.0 ** -19 * 8


def test_non_finite_rows_stay_in_their_pairs(fa):
    rot = fa.rotary_frequencies(64)
    x = make((1, 1, 3, 64), "bf16", 12)
    x[0, 0, 1, 5] = float("nan")
    x[0, 0, 2, 40] = float("inf")
    y = fa.rotary_forward(x, rot, offset=1)
    bad = ~torch.isfinite(y)
    assert set(map(tuple, bad.nonzero()[:, 2:].tolist())) == {(1, 5), (1, 37), (2, 8), (2, 40)}


def test_graph_replays_with_new_positions(fa):
    rot = fa.rotary_frequencies(64)
    q, pos = make((2, 2, 1, 64), "bf16", 13), torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    fa.rotary_forward(q, rot, positions=pos, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.rotary_forward(q, rot, positions=pos, out=out)
    for p in (3, 70000):
        pos.fill_(p)
        g.replay()
        torch.cuda.synchronize()
        check(out, q, rot, np.full((2, 1), p), "bf16")


def test_refusals(fa):
    rot = fa.rotary_frequencies(64)
    q, k = make((2, 2, 4, 64), "bf16", 14), make((2, 2, 4, 64), "fp16", 15)
    for kw in [dict(k=k), dict(k=q[:, :, :3]), dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(positions=torch.zeros(4, dtype=torch.int64, device="cuda")), dict(positions=torch.zeros(4, dtype=torch.int32)),
               dict(out=q[:, :, :3]), dict(k_out=q), dict(offset=2 ** 31), dict(out=torch.empty_like(k))]:
        with pytest.raises(ValueError):
            fa.rotary_forward(q, rot, **kw)
    with pytest.raises(ValueError):
        fa.rotary_forward(q.expand(2, 2, 4, 64)[..., ::2], rot)
    with pytest.raises(ValueError):
        fa.rotary_forward(q[:1, :1, :1].expand(2, 2, 4, 64), rot)
    with pytest.raises(fa.FaError):                      # more channels than the head has
        fa.rotary_forward(q, fa.rotary_frequencies(128))
    with pytest.raises(fa.FaError):                      # overlapping, not in place
        buf = torch.zeros(2 * 2 * 4 * 64 + 64, dtype=torch.bfloat16, device="cuda")
        fa.rotary_forward(buf[:1024].view(2, 2, 4, 64), rot, out=buf[64:1088].view(2, 2, 4, 64))


def test_training_step_with_attention(fa):
    """Rotary, attention, and both backward passes, against the chain in fp64 on the kernels' own
    rounded intermediates (the bars of tests/_util.py)."""
    import oracle
    from _util import check_fwd, check_grads
    rot = fa.rotary_frequencies(64)
    q, k, v, do = (make((2, 3, 200, 64), "bf16", 20 + i) for i in range(4))
    qr, kr = fa.rotary_forward(q, rot, k=k)
    o, lse = fa.forward(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.backward(qr, kr, v, o, do, lse, causal=True)
    dq, dk = fa.rotary_backward(dqr, rot, dk=dkr)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    pos = np.broadcast_to(np.arange(200), (2, 200))
    turn = lambda x, back=False: oc.rotate(x, rot.angles.numpy(), pos, 1.0, False, back)  # noqa: E731
    o_ref, l_ref = oracle.forward(turn(f64(q)), turn(f64(k)), f64(v), 0.125, causal=True)
    err = np.max(np.abs(f64(o) - o_ref))
    assert err <= 2.5e-2, err          # O's own bar (1e-2) plus q, k rounded once more: scores off by 2^-8
    g = oracle.backward(turn(f64(q)), turn(f64(k)), f64(v), f64(do), 0.125, causal=True)
    check_grads((dq, dk, dv), (turn(g[0], True), turn(g[1], True), g[2]))
    check_fwd(o, lse, *oracle.forward(f64(qr), f64(kr), f64(v), 0.125, causal=True))
