"""Windowed calls over very many keys. Where the weights are alike a running fp32 sum loses what each key adds
to it, so ranges of more than 65536 keys are cut into states; more sinks than that make one range with the
window."""
import math

import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests.window_util import Batch

pytestmark = pytest.mark.gpu

KEYS, NEW, HKV, MOST = (1 << 20) + 77, 8, 4, 2**31 - 1
RUN = 2 * 65536  # keys of a state at most: the sinks that stand apart and a split tile


def check_bias(call, d, page, window, sinks, new):
    """Values near a base of each column, weights of one size: what is lost would be lost by every output.

    Each output is near its column's base, so its rounding (2^-9 of it at most, uniform) has no sign over the
    4 d >= 256 columns: their mean is within 6 * 2^-9 / sqrt(3 * 256) < 2^-11 of zero. The weights' roundings
    (2^-9, independent from key to key) vanish over 65536 keys. A tensor core step adds 16 keys and loses up to
    a unit in the last place, 2^-23 of the sum: n / 16 * 2^-23 for a state of n keys, 2^-10 for RUN. The mean over a
    tile's course is half of that."""
    gen = torch.Generator(device="cuda").manual_seed(d + page)
    n_pages = -(-KEYS // page)
    shape, kw = (n_pages, page, HKV, d), dict(generator=gen, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(shape, **kw) * 0.1
    v = torch.rand(shape, **kw) * 0.25 + torch.rand(HKV, d, **kw) + 1
    q = torch.randn(new, 2 * HKV, d, generator=gen, device="cuda").bfloat16()
    desc = bia.make_desc(2 * HKV, HKV, d, page)
    kvp, last = torch.tensor([0, n_pages]).int(), torch.tensor([KEYS - (n_pages - 1) * page]).int()
    out, lse = torch.empty_like(q), torch.empty(new, 2 * HKV, device="cuda")
    call(desc, q, k, v, torch.arange(n_pages, device="cuda").int(), kvp, last, out, lse)
    p, j = torch.arange(KEYS - new, KEYS, device="cuda")[:, None], torch.arange(KEYS, device="cuda")[None]
    hidden = (j > p) | ((j <= p - window) & (j >= sinks))
    rel, lse_err = [], 0.0
    for h in range(2 * HKV):
        kk, vv = (x.view(-1, HKV, d)[:KEYS, h // 2].double() for x in (k, v))
        x = (q[:, h].double() @ kk.T * d ** -0.5).masked_fill(hidden, -math.inf)
        l = torch.logsumexp(x, -1)
        y = torch.exp(x - l[:, None]) @ vv
        rel.append((out[:, h].double() - y) / y)
        lse_err = max(lse_err, float((lse[:, h].double() - l).abs().max()))
    bias = float(torch.stack(rel).mean())
    assert abs(bias) <= 2.0 ** -11 + 2.0 ** -11, bias
    # 512 + 16 sums a state and 16 or 256 states joined, half a unit each; scores below 2 in fp32
    assert lse_err <= 2.0 ** -13, lse_err


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 1), (256, 16)])
@pytest.mark.parametrize("window,sinks,split", [(1024, MOST, 0), (1024, 65536, 0), (1024, 600000, 0), (MOST, 0, 1 << 24),
                                                (300000, 100000, 1 << 24)])
def test_extend_loses_nothing(d, page, window, sinks, split):
    def call(desc, q, k, v, pages, kvp, last, out, lse):
        qo = torch.tensor([0, NEW]).int()
        need = bia.bia_prefill_window_workspace_size(desc, window, sinks, qo, kvp, last, split)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        bia.bia_prefill_paged_window(desc, window, sinks, q, k, v, qo.cuda(), kvp.cuda(), pages, last.cuda(), qo, kvp, last,
                                     ws, out, lse, split)
        assert bia.bia_read_status(ws) == 0
    check_bias(call, d, page, window, sinks, NEW)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 1), (256, 16)])
@pytest.mark.parametrize("window,sinks,split", [(MOST, 0, 1 << 30), (300000, 600000, 1 << 20), (MOST, 0, 0)])
def test_decode_loses_nothing(d, page, window, sinks, split):
    def call(desc, q, k, v, pages, kvp, last, out, lse):
        need = bia.bia_decode_window_workspace_size(desc, window, sinks, kvp, last, split)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        bia.bia_decode_paged_window(desc, window, sinks, q, k, v, kvp.cuda(), pages, last.cuda(), kvp, last, ws, out, lse, split)
        assert bia.bia_read_status(ws) == 0
    check_bias(call, d, page, window, sinks, 1)


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 64, 16), (4, 4, 128, 16), (8, 1, 128, 1), (4, 1, 96, 8), (4, 2, 256, 16),
                                           (2, 1, 256, 2)])
@pytest.mark.parametrize("split", [0, 1024, 1 << 24])
def test_many_sinks(hq, hkv, d, page, split):
    """Sinks past 65536 that the window has left behind, what lies between NaN on pages that do not exist."""
    c = Batch([150000, 900, 66000], [130, 7, 40], hq, hkv, d, page, 300, 70001, seed=split % 1000 + d)
    ws = c.extend(split)
    assert bia.bia_read_status(ws) == 0
    c.check()


def test_many_sinks_folded_in_the_kernel():
    c = Batch([150000], [2304], 16, 16, 64, 16, 300, 70001, seed=3)
    ws = c.extend(1 << 24)
    per_row = 2304 * 3 * 16 * 65 * 4  # a state for each row and split, had they been merged
    assert bia.bia_read_status(ws) == 0 and ws.numel() < per_row
    c.check(rows=[0, 1, 127, 128, 300, 1000, 2047, 2303])
