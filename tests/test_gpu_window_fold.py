"""Windowed extends whose CTAs fold a pair's states themselves: against the definition in 64 bits, and against
the states of chunks, which a kernel of their own merges. Which way a call takes shows in its workspace."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests.window_util import Batch

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def states_of(rows, hq, d):
    return rows * hq * (d + 1) * 4


def folds(c, split):
    """Whether the call's workspace is that of a running state per CTA (152 of them) and not of one for each row."""
    d, hq = c.desc.head_dim, c.desc.num_qo_heads
    per_cta = (1 if d == 256 else 2) * 128 * (64 if d == 64 else 128 if d < 256 else 256)
    want = states_of(-(-152 * per_cta // (hq * d)), hq, d)
    need = bia.bia_prefill_window_workspace_size(c.desc, c.window, c.sinks, c.qo, c.kvp, c.last, split)
    return 0 <= need - want < 4096


# heads, width, page, tokens, window, sinks, split: 440 to 600 items and more than one split
CASES = [(32, 8, 128, 16, 3500, 600, 70, 128), (32, 8, 128, 16, 3500, 600, 70, 512), (32, 8, 128, 1, 3500, 100, 0, 128),
         (16, 16, 64, 1, 6900, 600, 70, 128), (16, 16, 64, 16, 6900, 2000, 300, 512), (16, 16, 96, 16, 6900, 600, 70, 256),
         (16, 8, 256, 16, 3500, 600, 70, 128), (16, 8, 256, 16, 3500, 1500, 1, 512), (16, 8, 256, 2, 3500, 300, 200, 256),
         (64, 8, 128, 16, 1800, 600, 70, 256), (16, 16, 64, 16, 9000, 5000, 4, 0), (32, 8, 128, 16, 9000, 4500, 64, 0),
         (16, 8, 256, 16, 9000, 2**31 - 1, 0, 0)]


@pytest.mark.parametrize("hq,hkv,d,page,n,window,sinks,split", CASES)
def test_folded_states(hq, hkv, d, page, n, window, sinks, split):
    group = 128 * hkv // hq
    c = Batch([n, 50], [n, 50], hq, hkv, d, page, window, sinks, seed=n % 97 + d, spoil=False)
    assert folds(c, split)
    ws = c.extend(split)
    assert bia.bia_read_status(ws) == 0
    edges = [0, 1, group, 2 * group - 1, 2 * group, 4095, 4096, n - 1] + [x + y for x in (window, sinks, window + sinks)
                                                                        for y in (-1, 0, 1, 127, 128)]
    some = torch.randint(0, n, (100,), generator=torch.Generator().manual_seed(1)).tolist()
    c.check([0], rows=[r for r in edges if 0 <= r < n] + some)
    c.check([1])
    whole = c.out.clone(), c.lse.clone()
    tiles = -(-n // group)
    for first, last in ((0, 2), (2, 3), (tiles // 2, tiles // 2 + 1), (tiles // 2 + 1, tiles // 2 + 4), (tiles - 3, tiles)):
        a, b = first * group, min(last * group, n)
        pages = -(-b // page)
        host = (torch.tensor([0, b - a]).int(), torch.tensor([0, pages]).int(), torch.tensor([b - (pages - 1) * page]).int())
        need = bia.bia_prefill_window_workspace_size(c.desc, window, sinks, *host, split)
        assert first < tiles // 2 or need >= states_of(2 * (b - a), hq, d)  # merged, a state for each row and split
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(c.out[a:b]), torch.empty_like(c.lse[a:b])
        bia.bia_prefill_paged_window(c.desc, window, sinks, c.q[a:b].contiguous(), c.k_cache, c.v_cache, host[0].cuda(),
                                     host[1].cuda(), c.dev[1], host[2].cuda(), *host, ws, out, lse, split)
        assert torch.equal(bits(out), bits(whole[0][a:b])) and torch.equal(bits(lse), bits(whole[1][a:b])), (a, b)


@pytest.mark.parametrize("d,hq,hkv", [(64, 16, 16), (128, 16, 16), (256, 32, 16)])
def test_folded_over_a_prefix_of_other_lengths(d, hq, hkv):
    """Chunks of several requests, no two of which have their windows' splits in step; what is not seen is NaN."""
    tile = 128 * hkv // hq
    new = [5 * tile + 3, 6 * tile, 1, 4 * tile - 1, 2 * tile + 60, 10 * tile] * (2 if d < 256 else 1)
    keys = [n + 777 * (i + 1) % 3001 for i, n in enumerate(new)]
    c = Batch(keys, new, hq, hkv, d, 16, 700, 130, seed=d)
    assert folds(c, 256)
    ws = c.extend(256)
    assert bia.bia_read_status(ws) == 0
    c.check()


def test_folded_rows_with_large_scores():
    """Running maxima far apart from split to split."""
    c = Batch([3500, 50], [3500, 50], 32, 8, 128, 16, 600, 70, seed=8, spread=20.0, spoil=False)
    assert folds(c, 128)
    ws = c.extend(128)
    assert bia.bia_read_status(ws) == 0
    c.check([0], rows=list(range(0, 3500, 37)))
    c.check([1])
