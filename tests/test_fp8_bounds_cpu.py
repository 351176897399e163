"""The decode's bounds can fail: they are small beside the outputs, and wrong
outputs lie outside them.  (The mistakes are planted in the expected values.)"""
import pytest
import torch

from tests import fp8_bounds as fb
from tests import fp8_util as fu


def request(n, hq, hkv, d, seed, device="cpu"):
    """q and the quantised keys and values of one request of n keys."""
    g = torch.Generator(device=device).manual_seed(seed)
    q = fu.rows((1, hq, d), g, device)
    rows = [fu.rows((n, hkv, d), g, device) for _ in "kv"]
    out = [q]
    for r in rows:
        c, e = fu.quantise(r)
        out += [c.float().to(fu.E4M3), (e + 127).to(fu.U8).view(fu.E8M0)]
    return out


@pytest.mark.parametrize("n", [1, 300, 2049, 5000])
@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (8, 8, 64), (16, 8, 256)])
def test_bounds_are_small_and_wrong_outputs_break_them(n, hq, hkv, d):
    q, kc, ks, vc, vs = request(n, hq, hkv, d, n + d)
    out, tol, lse, lse_tol = fb.decode_bounds(q, kc, ks, vc, vs)
    rms = out.square().mean().sqrt()
    assert tol.median() < 0.02 * rms
    fu.check(out.bfloat16(), lse.float(), out, tol, lse, lse_tol)
    with pytest.raises(AssertionError):  # zeros
        fu.check(torch.zeros_like(out), lse, out, tol, lse, lse_tol)
    if n > 128:  # a block of 128 keys left out, one after the other
        x = torch.einsum("hd,khd->hk", q[0].double(),
                         fu.cache_values(kc, ks).repeat_interleave(hq // hkv, 1)) * d ** -0.5
        p = torch.softmax(x, -1)
        v = fu.cache_values(vc, vs).repeat_interleave(hq // hkv, 1)
        worst = 0
        for a in range(0, n, 128):
            kept = p.clone()
            kept[:, a:a + 128] = 0
            other = torch.einsum("hk,khd->hd", kept, v) / kept.sum(-1, keepdim=True)
            worst = max(worst, int(((other - out[0]).abs() > tol[0]).any()))
            if p[:, a:a + 128].sum(-1).max() > 0.02:
                assert ((other - out[0]).abs() > tol[0]).any(), a
        assert worst


@pytest.mark.parametrize("s", [20, 60])
def test_a_large_row_nobody_attends_does_not_widen_the_bounds(s):
    q, kc, ks, vc, vs = request(500, 4, 2, 64, 7)
    q[..., 0] = 8.0
    kc[13], ks.view(fu.U8)[13] = 0, 127
    kc[13, :, 0] = -448.0  # a score of -448: a weight below 2^-500
    before = fb.decode_bounds(q, kc, ks, vc, vs)
    vs.view(fu.U8)[13] += s
    after = fb.decode_bounds(q, kc, ks, vc, vs)
    assert torch.allclose(before[0], after[0], rtol=1e-9)
    assert (after[1] <= before[1] * 1.02).all()
