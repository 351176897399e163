"""Decode with a window and sinks against the definition in 64 bits. Whatever a query does not see is NaN
in the cache, and its pages' entries do not exist (tests/window_util.py)."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu
from tests.window_util import Batch

pytestmark = pytest.mark.gpu
I32 = torch.int32


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


SIZES = [1, 2, 127, 128, 129, 1023, 3000]


@pytest.mark.parametrize("hq,hkv,d,page", [(4, 4, 64, 1), (8, 4, 128, 16), (32, 8, 128, 1), (8, 1, 128, 256),
                                           (2, 1, 96, 8), (16, 4, 64, 32), (16, 8, 256, 16), (3, 3, 128, 4),
                                           (8, 1, 256, 2), (4, 1, 96, 64), (8, 1, 64, 16), (2, 2, 256, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (128, 0), (100, 4), (1000, 130), (517, 2000), (2**31 - 1, 3),
                                          (2000, 2**31 - 1)])
def test_against_the_definition(hq, hkv, d, page, window, sinks):
    c = Batch(SIZES, [1] * len(SIZES), hq, hkv, d, page, window, sinks, seed=window % 1000 + d)
    ws = c.decode()
    assert bia.bia_read_status(ws) == 0
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 4, 64), (8, 8, 256), (16, 2, 96)])
@pytest.mark.parametrize("split", [128, 256, 1024, 4096])
def test_splits_and_batches(hq, hkv, d, split):
    """Right at every split size, and a request has the same bits alone and in any batch."""
    sizes = [5000, 33, 700, 1, 2500]
    c = Batch(sizes, [1] * 5, hq, hkv, d, 16, 1500, 70, seed=split)
    c.decode(split)
    c.check()
    for b in (0, 2, 3):
        one = [torch.tensor([0, int(c.kvp[b + 1] - c.kvp[b])]).int(), c.pages[int(c.kvp[b]):int(c.kvp[b + 1])], c.last[b:b + 1]]
        ws = torch.empty(bia.bia_decode_window_workspace_size(c.desc, 1500, 70, one[0], one[2], split), dtype=torch.uint8,
                         device="cuda")
        out, lse = torch.empty_like(c.out[:1]), torch.empty_like(c.lse[:1])
        bia.bia_decode_paged_window(c.desc, 1500, 70, c.q[b:b + 1].contiguous(), c.k_cache, c.v_cache,
                                    *(x.cuda() for x in one), one[0], one[2], ws, out, lse, split)
        assert torch.equal(bits(out), bits(c.out[b:b + 1])) and torch.equal(bits(lse), bits(c.lse[b:b + 1]))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_window_over_everything_is_the_plain_decode(d):
    sizes = [4000, 1, 513, 2048]
    c = Batch(sizes, [1] * 4, 8, 2, d, 16, 4000, 5, seed=3)
    c.decode(512)
    ws = torch.empty(bia.bia_decode_workspace_size(c.desc, c.kvp, c.last, 512), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    bia.bia_decode_paged(c.desc, c.q, c.k_cache, c.v_cache, *c.dev, c.kvp, c.last, ws, out, lse, split_size=512)
    assert torch.equal(bits(out), bits(c.out)) and torch.equal(bits(lse), bits(c.lse))


@pytest.mark.parametrize("d", [64, 128])
def test_many_requests_large_scores_and_no_lse(d):
    sizes = [1 + 37 * b % 1500 for b in range(900)]
    c = Batch(sizes, [1] * 900, 4, 2, d, 16, 300, 20, seed=5, spread=20.0)
    c.decode()
    c.check()
    out = torch.empty_like(c.out)
    c.decode(out=out, lse=None)
    assert torch.equal(bits(out), bits(c.out))


@pytest.mark.parametrize("d", [96, 128])
def test_bad_pages_and_bad_arrays(d):
    """A page that does not exist reads as zeros and is noted; a request whose arrays break a rule is NaN
    and noted, the others are not touched by it."""
    sizes = [700, 50, 900, 64]
    c = Batch(sizes, [1] * 4, 8, 2, d, 16, 200, 20, seed=6, spoil=False)
    fine = c.decode()
    assert bia.bia_read_status(fine) == 0
    good = c.out.clone()
    pages = c.dev[1].clone()
    c.dev[1][int(c.kvp[2]) + 900 // 16] = c.n_pages  # request 2's last page
    c.dev[2][1] = 17
    ws = c.decode()
    assert bia.bia_read_status(ws) == 1 | 2
    assert bool(c.out[1].isnan().all()) and bool(c.lse[1].isnan().all())
    for b in (0, 3):
        assert torch.equal(bits(c.out[b]), bits(good[b]))
    page = 900 // 16 * 16
    c.rows_k[2][page:], c.rows_v[2][page:] = 0, 0
    c.check([2])
    c.dev[1].copy_(pages)
    for arrays in ([0, 44, 44, 105, 109], [0, 44, 43, 105, 109], [-1, 44, 48, 105, 109]):  # no page, falling, negative
        kvp = torch.tensor(arrays).int()
        c.dev[0].copy_(kvp)
        c.dev[2].copy_(c.last)
        ws = c.decode()
        assert bia.bia_read_status(ws) & 2
        bad = [b for b in range(4) if kvp[b + 1] <= kvp[b] or kvp[b] < 0]
        for b in bad:
            assert bool(c.out[b].isnan().all())


def bounded_call(c, bounds, ws, split=0):
    bia.bia_decode_paged_window_bounded(c.desc, bounds, c.window, c.sinks, c.q, c.k_cache, c.v_cache, *c.dev, ws, c.out,
                                        c.lse, split)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 4, 64)])
def test_bounded_and_captured(hq, hkv, d):
    """The bounded call has the exact call's bits; captured once, it follows growing lengths."""
    final = [2100, 700, 1500]
    c = Batch(final, [1] * 3, hq, hkv, d, 8, 600, 40, seed=8, spoil=False)
    bounds = bia.make_bounds(max_kv_len=4000)
    ws = torch.empty(bia.bia_decode_window_bounded_workspace_size(c.desc, bounds, 600, 40, 3), dtype=torch.uint8, device="cuda")
    c.decode()
    want = c.out.clone(), c.lse.clone()
    c.out.fill_(0), c.lse.fill_(0)
    bounded_call(c, bounds, ws)
    assert torch.equal(bits(want[0]), bits(c.out)) and torch.equal(bits(want[1]), bits(c.lse))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        bounded_call(c, bounds, ws)
    rows = c.rows_k, c.rows_v
    for now in ([1, 1, 1], [500, 600, 601], [640, 641, 1300], final):
        count = [-(-n // 8) for n in now]
        at = torch.cat([c.pages[int(c.kvp[b]):int(c.kvp[b]) + n] for b, n in enumerate(count)])
        c.dev[0].copy_(fu.indptr_of(count))
        c.dev[1][:len(at)].copy_(at)
        c.dev[2].copy_(torch.tensor([n - (k - 1) * 8 for n, k in zip(now, count)]).int())
        graph.replay()
        assert bia.bia_read_status(ws) == 0
        c.keys = now
        c.rows_k, c.rows_v = ([r[:n] for r, n in zip(x, now)] for x in rows)
        c.check()
    c.dev[2][0] = 8
    c.dev[0].copy_(torch.tensor([0, 501, 502, 503]).int())  # 4008 keys: above the bound
    graph.replay()
    assert bia.bia_read_status(ws) == 2
    assert bool(c.out[0].isnan().all()) and not bool(c.out[1:].isnan().any())


def test_offsets_past_32_bits_and_another_stream():
    """A cache of more than 2^31 elements whose last pages are read, on a stream of the caller's."""
    c = Batch([900, 300], [1, 1], 8, 8, 128, 16, 500, 4, seed=9)
    pages = (1 << 31) // (16 * 8 * 128) + 64
    big = [torch.zeros(pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, x in zip(big, (c.k_cache, c.v_cache)):
        b[-c.n_pages:] = x
    table = torch.where((c.pages >= 0) & (c.pages < c.n_pages), c.pages + (pages - c.n_pages), -1).int()
    c.decode()
    want = c.out.clone()
    c.k_cache, c.v_cache = big
    c.dev = (c.dev[0], table.cuda(), c.dev[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    ws = c.decode(stream=s)
    assert bia.bia_read_status(ws, s) == 0
    s.synchronize()
    assert torch.equal(bits(want), bits(c.out))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_split_tile_longer_than_every_request(d):
    """Whatever its size: 32-bit arithmetic on it must not wrap."""
    c = Batch([900, 3], [1, 1], 8, 4, d, 16, 500, 4, seed=12)
    c.decode(1024)
    want = c.out.clone(), c.lse.clone()
    c.check()
    for split in (1 << 30, 2**31 - 128):
        c.out.fill_(7), c.lse.fill_(7)
        c.decode(split)
        assert torch.equal(bits(want[0]), bits(c.out)) and torch.equal(bits(want[1]), bits(c.lse))
    e = Batch([900, 300], [40, 300], 8, 4, d, 16, 500, 4, seed=13)
    e.extend(1024)
    want = e.out.clone()
    e.extend(1 << 24)
    e.check()
    assert torch.equal(bits(want), bits(e.out))
