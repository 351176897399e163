"""64-bit decode over an 8-bit cache and the bounds its kernel is held to,
from the number formats alone (no share of it grows with a value that the
query does not attend)."""
from __future__ import annotations

import torch

from tests import fp8_util as fu

PART = 512  # keys that share a weight grid, counted from their tile's first key


def decode_bounds(q, k_codes, k_scale, v_codes, v_scale, split=1024):
    """One request: q [1, Hq, D]; codes [n, Hkv, D] e4m3 and scales [n, Hkv]
    e8m0 of its keys in order.  Returns (out, tol, lse, lse_tol).

    fu.attention_bounds states the bounds of the scores, of weights held to 8
    significant bits (off by at most 2^-8 relative), of the fp32 sums and of
    the bf16 output.  What is added here is the grid under them.  A key's
    weight is p * 2^ev (p its softmax weight, 2^ev its value row's scale), and
    the largest W of a part's weights is brought into (2^7, 2^8] by a power of
    two.  There it is held as hi + lo/16, both e4m3: e4m3's last place is 2^-9
    and lo's 2^-13, so that a weight is off by at most 2^-8 of itself while it
    is at least 2^-6, and by at most half a place, 2^-14, below: 2^-21 * W.  It
    multiplies the row's codes, so every key adds at most 2^-21 * W * |code|
    (1.01: the roundings of W).
    """
    k, v = fu.cache_values(k_codes, k_scale), fu.cache_values(v_codes, v_scale)
    out, tol, lse, lse_tol = fu.attention_bounds(q, k, v)
    n, hkv, d = k.shape
    hq = q.shape[1]
    x = torch.einsum("hd,khd->hk", q[0].double(), k.repeat_interleave(hq // hkv, 1)) * d ** -0.5
    ev = (v_scale.view(fu.U8).double() - 127).T.repeat_interleave(hq // hkv, 0)  # [Hq, n]
    weight = torch.exp2((x - lse.T) / torch.log(torch.tensor(2.0, dtype=fu.F64)) + ev)
    codes = v_codes.double().abs().repeat_interleave(hq // hkv, 1)  # [n, Hq, D]
    for tile in range(0, n, split):
        for a in range(tile, min(tile + split, n), PART):
            e = min(a + PART, tile + split, n)
            top = weight[:, a:e].amax(-1)
            tol = tol + 1.01 * 2.0 ** -21 * top[None, :, None] * codes[a:e].sum(0)[None]
    return out, tol, lse, lse_tol
