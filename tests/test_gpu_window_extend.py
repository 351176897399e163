"""Extend with a window and sinks against the definition in 64 bits. Whatever the call does not see is NaN
in the cache, and its pages' entries do not exist (tests/window_util.py)."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu
from tests.window_util import Batch

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


SHAPES = [(4, 4, 64, 1), (8, 4, 128, 16), (32, 8, 128, 1), (8, 1, 128, 256), (2, 1, 96, 8), (16, 4, 64, 32), (4, 2, 256, 16),
          (3, 3, 128, 4), (8, 1, 256, 2), (4, 1, 96, 64), (8, 1, 64, 16), (2, 2, 256, 128), (1, 1, 128, 2)]
LENGTHS = [([1], [1]), ([130], [130]), ([700, 0, 5, 1300, 129], [3, 0, 5, 200, 129]), ([2000, 64, 1], [1, 64, 1])]


@pytest.mark.parametrize("keys,new", LENGTHS, ids=range(len(LENGTHS)))
@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (128, 0), (100, 4), (1000, 130), (300, 500), (2**31 - 1, 3),
                                          (500, 2**31 - 1)])
def test_against_the_definition(keys, new, hq, hkv, d, page, window, sinks):
    c = Batch(keys, new, hq, hkv, d, page, window, sinks, seed=window % 1000 + d)
    ws = c.extend()
    assert bia.bia_read_status(ws) == 0
    c.check()


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 128, 16), (4, 4, 64, 1), (8, 4, 256, 16), (16, 2, 96, 4)])
@pytest.mark.parametrize("split", [128, 256, 1024])
@pytest.mark.parametrize("window,sinks", [(90, 3), (700, 200), (2000, 0)])
def test_splits(hq, hkv, d, page, split, window, sinks):
    """Right at every split size, with the states merged."""
    c = Batch([3000, 33, 900], [150, 33, 290], hq, hkv, d, page, window, sinks, seed=split + window)
    ws = c.extend(split)
    assert bia.bia_read_status(ws) == 0
    c.check()


@pytest.mark.parametrize("hq,hkv,d,page,n", [(32, 8, 128, 16, 2500), (16, 16, 64, 1, 5000), (16, 8, 256, 16, 2450)])
@pytest.mark.parametrize("split", [128, 512])
def test_folded_in_the_kernel_and_any_batch(hq, hkv, d, page, n, split):
    """A long prompt's states are folded by the CTAs, a chunk's on the q-tile grid are merged: the same bits,
    alone and in a batch."""
    window, sinks, group = 600, 70, 128 * hkv // hq
    assert -(-n // group) * hkv // (1 if d == 256 else 2) >= 304
    c = Batch([n, 50], [n, 50], hq, hkv, d, page, window, sinks, seed=4, spoil=False)
    c.extend(split)
    c.check([0], rows=[0, 1, 127, 128, 600, 601, 669, 670, 671, 800, n - 1])
    c.check([1])
    whole = c.out.clone(), c.lse.clone()
    for a, b in ((0, 2 * group), (2 * group, 3 * group), (n // group // 2 * group, n // group // 2 * group + 5)):
        pages = -(-b // page)
        host = torch.tensor([0, b - a]).int(), torch.tensor([0, pages]).int(), torch.tensor([b - (pages - 1) * page]).int()
        ws = torch.empty(bia.bia_prefill_window_workspace_size(c.desc, window, sinks, *host, split), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(c.out[a:b]), torch.empty_like(c.lse[a:b])
        bia.bia_prefill_paged_window(c.desc, window, sinks, c.q[a:b].contiguous(), c.k_cache, c.v_cache, host[0].cuda(),
                                     host[1].cuda(), c.dev[1], host[2].cuda(), *host, ws, out, lse, split)
        assert torch.equal(bits(out), bits(whole[0][a:b])) and torch.equal(bits(lse), bits(whole[1][a:b]))


def test_repeats_have_the_same_bits():
    c = Batch([5000, 3000], [2000, 3000], 32, 8, 128, 16, 1024, 4, seed=6, spoil=False)
    c.extend(256)
    want = c.out.clone(), c.lse.clone()
    for _ in range(5):
        c.out.fill_(0), c.lse.fill_(0)
        c.extend(256)
        assert torch.equal(bits(want[0]), bits(c.out)) and torch.equal(bits(want[1]), bits(c.lse))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_requests_large_scores_and_no_lse(d):
    keys = [1 + 37 * b % 700 for b in range(700)]
    new = [min(k, b % 9) for b, k in enumerate(keys)]
    c = Batch(keys, new, 4, 2, d, 16, 200, 20, seed=5, spread=20.0)
    ws = c.extend()
    assert bia.bia_read_status(ws) == 0
    c.check()
    out = torch.empty_like(c.out)
    c.extend(out=out, lse=None)
    assert torch.equal(bits(out), bits(c.out))


@pytest.mark.parametrize("d,page", [(64, 1), (128, 16), (256, 16), (96, 8)])
def test_bad_pages(d, page):
    """A page that does not exist reads as zeros and is noted."""
    c = Batch([700, 90], [40, 90], 8, 2, d, page, 200, 20, seed=6, spoil=False)
    c.dev[1][int(c.kvp[1]) - 3] = c.n_pages
    c.dev[1][int(c.kvp[1]) + 1] = -7
    ws = c.extend()
    assert bia.bia_read_status(ws) == 1
    at = int(c.kvp[1] - c.kvp[0]) - 3
    for x in (c.rows_k, c.rows_v):
        x[0][at * page:(at + 1) * page] = 0
        x[1][page:2 * page] = 0
    c.check()


def test_bad_arrays_compute_nothing():
    c = Batch([700, 90, 300], [40, 90, 7], 8, 2, 128, 16, 200, 20, seed=7, spoil=False)
    good = [x.clone() for x in c.dev]
    qo = c.qo.clone()
    # kv_indptr [0, 44, 50, 69], last pages, qo_indptr [0, 40, 130, 137]: no table entry past the last is asked for
    for which, at, value in ((0, 1, 46), (0, 0, -1), (0, 3, 50), (2, 0, 17), (2, 1, 0), (0, 2, 44), (3, 1, 39), (3, 2, 200),
                             (3, 0, 1), (3, 1, 137)):
        for x, y in zip(c.dev, good):
            x.copy_(y)
        c.qo = qo.clone()
        if which < 3:
            c.dev[which][at] = value
        c.out.fill_(0), c.lse.fill_(0)
        need = bia.bia_prefill_window_workspace_size(c.desc, 200, 20, qo, c.kvp, c.last)
        ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
        dev_qo = qo.cuda()
        if which == 3:
            dev_qo[at] = value
        bia.bia_prefill_paged_window(c.desc, 200, 20, c.q, c.k_cache, c.v_cache, dev_qo, *c.dev, qo, c.kvp, c.last, ws, c.out, c.lse)
        assert bia.bia_read_status(ws) == 2 and bool(c.out.isnan().all()) and bool(c.lse.isnan().all()), (which, at, value)


def test_captured_twice_over_one_workspace():
    """Two captured calls that share a workspace, replayed in turn, and the arrays changing between replays."""
    c = Batch([900, 600], [64, 40], 8, 2, 128, 16, 300, 10, seed=8, spoil=False)
    d = Batch([500, 1000], [64, 40], 8, 2, 128, 16, 300, 10, seed=9, spoil=False)
    need = max(bia.bia_prefill_window_workspace_size(x.desc, 300, 10, x.qo, x.kvp, x.last, 128) for x in (c, d))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    graphs = []
    for x in (c, d):
        x.args = (x.qo.cuda(), *x.dev)
        g = torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=stream):
            bia.bia_prefill_paged_window(x.desc, 300, 10, x.q, x.k_cache, x.v_cache, *x.args, x.qo, x.kvp, x.last, ws, x.out,
                                         x.lse, 128)
        graphs.append(g)
    for _ in range(3):
        for x, g in zip((c, d), graphs):
            x.out.fill_(0)
            g.replay()
    for x in (c, d):
        x.check()
    # request 0 grows shorter: 20 keys fewer, the same number of tokens
    c.args[3][0] = c.last[0] - 3
    c.keys = [897, 600]
    c.rows_k[0], c.rows_v[0] = c.rows_k[0][:897], c.rows_v[0][:897]
    graphs[0].replay()
    assert bia.bia_read_status(ws) == 0
    c.check()


def test_rows_behind_and_another_stream():
    """Rows of out past the call's tokens stay as they were; the call runs on the stream that it is given."""
    c = Batch([300, 80], [100, 30], 8, 4, 128, 16, 90, 4, seed=10)
    out = torch.full((140, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = c.extend(out=out[:130], stream=s)
    assert bia.bia_read_status(ws, s) == 0
    s.synchronize()
    c.out = out[:130]
    c.check()
    assert bool((out[130:] == 7).all())


def test_no_token():
    c = Batch([30, 16], [0, 0], 8, 4, 128, 16, 90, 4, seed=10)
    ws = torch.full((4096,), 9, dtype=torch.uint8, device="cuda")
    c.extend(ws=ws)
    assert bool((ws == 9).all())


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements whose last pages are read."""
    for page in (16, 1):
        c = Batch([900, 300], [70, 300], 8, 8, 128, page, 500, 4, seed=9)
        pages = (1 << 31) // (page * 8 * 128) + 64 * 16 // page
        pages = max(pages, c.n_pages + pages)
        big = [torch.zeros(pages, page, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for b, x in zip(big, (c.k_cache, c.v_cache)):
            b[-c.n_pages:] = x
        table = torch.where((c.pages >= 0) & (c.pages < c.n_pages), c.pages + (pages - c.n_pages), -1).int()
        c.extend()
        want = c.out.clone()
        c.k_cache, c.v_cache = big
        c.dev = (c.dev[0], table.cuda(), c.dev[2])
        c.out.fill_(0)
        c.extend()
        assert torch.equal(bits(want), bits(c.out))
        del big, c
