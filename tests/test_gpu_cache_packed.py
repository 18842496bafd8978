"""q, k and v as views of one packed projection [B, N, (Hq + 2 Hk) d], grouped heads: rotated in place,
written and attended over, against the definitions."""
import numpy as np
import pytest
import torch

from _util import f64
from oracle import cache as oc
from test_gpu_cache import Model, check_attention
from test_gpu_rotary import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dt", [("e4m3", "bf16"), ("int8", "fp16")])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 64), (8, 1, 128), (3, 3, 64)])
def test_serving_on_a_packed_projection(fa, Hq, Hk, d, fmt, dt):
    B, page, W = 2, 16, 8
    m = Model(fa, B * W + 1, Hk, page, d, fmt, B, W, seed=50)
    rot = fa.rotary_frequencies(d)
    lens = [0, 0]
    for step, (N, counts) in enumerate([(33, [33, 20]), (1, [1, 1]), (5, [5, 5]), (1, [1, 1])]):
        g = torch.Generator().manual_seed(step)
        x = torch.randn((B, N, (Hq + 2 * Hk) * d), generator=g).to({"bf16": torch.bfloat16, "fp16": torch.float16}[dt]).cuda()
        was = x.clone()
        q, k, v = (t.unflatten(2, (-1, d)).transpose(1, 2) for t in x.split([Hq * d, Hk * d, Hk * d], 2))
        pos = torch.tensor(lens, dtype=torch.int32)[:, None] + torch.arange(N, dtype=torch.int32)
        y, z = fa.rotary_forward(q, rot, k=k, positions=pos.cuda(), out=q, k_out=k)
        assert y.data_ptr() == q.data_ptr() and z.data_ptr() == k.data_ptr()
        check(q, was[..., :Hq * d].unflatten(2, (-1, d)).transpose(1, 2), rot, pos.numpy(), dt)
        check(k, was[..., Hq * d:(Hq + Hk) * d].unflatten(2, (-1, d)).transpose(1, 2), rot, pos.numpy(), dt)
        assert torch.equal(x[..., (Hq + Hk) * d:], was[..., (Hq + Hk) * d:])
        m.write(fa, k, v, list(lens), counts)
        m.same()
        lens = [a + c for a, c in zip(lens, counts)]
        check_attention(fa, m, q, lens, counts, dt=dt)
    assert fa.device_status() == fa.FA_OK
    # reading back into views of one buffer
    i32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.zeros((B, max(lens), 2 * Hk * d), dtype=x.dtype, device="cuda")
    k, v = (t.unflatten(2, (-1, d)).transpose(1, 2) for t in out.split(Hk * d, 2))
    fa.cache_read(m.cache, m.table.cuda(), i32, max(lens), dtype=x.dtype, k_out=k, v_out=v)
    for n, t in (("k", k), ("v", v)):
        want = oc.sequence(m.codes[n], m.scale[n], m.table[1].numpy(), page, fmt, 0, lens[1])
        assert np.all(np.abs(f64(t[1, :, :lens[1]]) - want) <= torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -25)


def test_backward_in_place_on_packed_gradients(fa):
    rot = fa.rotary_frequencies(64)
    x = torch.randn((2, 9, 8 * 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q, k = (t.unflatten(2, (-1, 64)).transpose(1, 2) for t in x.split([4 * 64, 2 * 64, 2 * 64], 2)[:2])
    want = fa.rotary_backward(q.clone(), rot, dk=k.clone())
    fa.rotary_backward(q, rot, dk=k, out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
