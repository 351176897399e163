"""The rotation and windowed calls as a server runs them together: projections normed, rotated and appended,
prompts extended in chunks, tokens decoded from a captured step; and the same over the 8-bit cache."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu
from tests import rope_util as ru
from tests import window_util as wu
from tests.fp8_bounds import decode_bounds

pytestmark = pytest.mark.gpu
BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def ints(x):
    return torch.tensor(x, dtype=I32)


class Server:
    """Requests on a pool of scattered pages; `lens` keys each so far."""

    def __init__(self, batch, hq, hkv, d, page, window, sinks, most, seed):
        self.gen = torch.Generator().manual_seed(seed)
        self.batch, self.hq, self.hkv, self.d, self.page = batch, hq, hkv, d, page
        self.window, self.sinks = window, sinks
        self.desc = bia.make_desc(hq, hkv, d, page)
        self.rope, self.fa = ru.make(d, most + 1)
        self.table = ru.table_of(most + 1, d).cuda()
        self.qw, self.kw = ru.weights(d, self.gen)
        per = -(-most // page)
        self.ids = torch.randperm(batch * per, generator=self.gen).int().view(batch, per)
        self.k = torch.full((batch * per, page, hkv, d), float("nan"), dtype=BF16, device="cuda")
        self.v = self.k.clone()
        self.lens = [0] * batch

    def arrays(self, new):
        """append_indptr and page table once new[b] tokens more are there, host and device."""
        self.lens = [a + b for a, b in zip(self.lens, new)]
        count = [-(-n // self.page) for n in self.lens]
        host = (fu.indptr_of(new), fu.indptr_of(count), ints([n - (c - 1) * self.page if c else 0 for n, c in zip(self.lens, count)]))
        pages = torch.cat([self.ids[b, :c] for b, c in enumerate(count)])
        return host, (host[0].cuda(), host[1].cuda(), pages.cuda(), host[2].cuda())

    def chunk(self, rows, new, split=0):
        """Appends and extends: rows [sum(new), hq + 2 hkv, d] of the fused projection."""
        host, dev = self.arrays(new)
        hq, hkv = self.hq, self.hkv
        q = torch.empty(rows.shape[0], hq, self.d, dtype=BF16, device="cuda")
        bia.bia_append_paged_kv_rope(self.desc, self.rope, self.table, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:],
                                     self.k, self.v, *dev, *host, q, None, self.qw, self.kw)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        ws = torch.empty(bia.bia_prefill_window_workspace_size(self.desc, self.window, self.sinks, *host, split), dtype=U8,
                         device="cuda")
        bia.bia_prefill_paged_window(self.desc, self.window, self.sinks, q, self.k, self.v, *dev, *host, ws, out, lse, split)
        assert bia.bia_read_status(ws) == 0
        return q, out, lse

    def rows_of(self, b, n):
        p = torch.arange(n)
        slots = (self.ids[b].long()[p // self.page] * self.page + p % self.page).cuda()
        return self.k.flatten(0, 1)[slots], self.v.flatten(0, 1)[slots]


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 128, 16), (4, 4, 64, 1), (4, 2, 256, 8)])
def test_chunks_and_steps(hq, hkv, d, page):
    """Prompts appended and extended in chunks have the bits of whole ones; decode steps from one captured
    graph, the append among them, are right; what left the window may be given up."""
    tile, window, sinks, n, steps = 128 * hkv // hq, 150, 5, [5 * 128, 200], 6
    most = max(n) + steps
    whole, cut = (Server(2, hq, hkv, d, page, window, sinks, most, 3) for _ in range(2))
    rows = [ru.rows((x, hq + 2 * hkv, d), whole.gen) for x in n]
    q, out, lse = whole.chunk(torch.cat(rows), n)
    at = [0, 0]
    got = [[], []]
    for size in ([3 * tile, tile], [tile, 200 - tile], [n[0] - 4 * tile, 0]):
        size = [min(s, x - a) for s, x, a in zip(size, n, at)]
        part = torch.cat([r[a:a + s] for r, a, s in zip(rows, at, size)])
        _, o, _ = cut.chunk(part, size)
        for b in range(2):
            got[b].append(o[:size[0]] if b == 0 else o[size[0]:])
        at = [a + s for a, s in zip(at, size)]
    assert at == n
    assert torch.equal(bits(torch.cat(got[0])), bits(out[:n[0]])) and torch.equal(bits(torch.cat(got[1])), bits(out[n[0]:]))
    assert torch.equal(bits(whole.k), bits(cut.k)) and torch.equal(bits(whole.v), bits(cut.v))
    s0 = 0
    for b in range(2):
        k, v = whole.rows_of(b, n[b])
        y, slack = ru.reference(rows[b][:, hq:hq + hkv], whole.kw, whole.rope, whole.fa, whole.table.cpu(),
                                torch.arange(n[b])[None].int())
        ru.check_bf16(k, y, slack)
        seen = wu.seen_of(n[b], n[b], window, sinks).cuda()
        fu.check(out[s0:s0 + n[b]], lse[s0:s0 + n[b]], *wu.bounds(q[s0:s0 + n[b]], k, v, seen))
        s0 += n[b]
    # give up what no later token sees
    for b in range(2):
        for p in range(-(-sinks // page), (n[b] + 1 - window) // page):
            whole.k[whole.ids[b, p].long()] = float("nan")
            whole.v[whole.ids[b, p].long()] = float("nan")
    # one captured step: append, then decode
    host, dev = whole.arrays([1, 1])
    dev = (dev[0], dev[1], torch.cat([whole.ids[0], whole.ids[1]]).cuda(), dev[3])
    step_rows = torch.empty(2, hq + 2 * hkv, d, dtype=BF16, device="cuda")
    q1 = torch.empty(2, hq, d, dtype=BF16, device="cuda")
    o1, l1 = torch.empty_like(q1), torch.empty(2, hq, device="cuda")
    bounds = bia.make_bounds(max_kv_len=most)
    ws = torch.empty(bia.bia_decode_window_bounded_workspace_size(whole.desc, bounds, window, sinks, 2), dtype=U8, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        bia.bia_append_paged_kv_rope(whole.desc, whole.rope, whole.table, step_rows[:, :hq], step_rows[:, hq:hq + hkv],
                                     step_rows[:, hq + hkv:], whole.k, whole.v, *dev, *host, q1, None, whole.qw, whole.kw)
        bia.bia_decode_paged_window_bounded(whole.desc, bounds, window, sinks, q1, whole.k, whole.v, *dev[1:], ws, o1, l1)
    for step in range(steps):
        if step:
            host, now = whole.arrays([1, 1])
            dev[1].copy_(now[1]), dev[3].copy_(now[3])
            dev[2][:len(now[2])].copy_(now[2])
        else:
            dev[2][:int(host[1][-1])].copy_(torch.cat([whole.ids[b, :int(host[1][b + 1] - host[1][b])] for b in range(2)]))
        step_rows.copy_(ru.rows(step_rows.shape, whole.gen))
        graph.replay()
        assert bia.bia_read_status(ws) == 0
        pos = torch.tensor([[x - 1 for x in whole.lens]]).int()
        ru.check_bf16(q1, *ru.reference(step_rows[:, :hq], whole.qw, whole.rope, whole.fa, whole.table.cpu(), pos))
        for b in range(2):
            k, v = whole.rows_of(b, whole.lens[b])
            seen = wu.seen_of(1, whole.lens[b], window, sinks).cuda()
            fu.check(o1[b:b + 1], l1[b:b + 1], *wu.bounds(q1[b:b + 1], k, v, seen))


def test_the_8_bit_cache():
    """Prompt: append with rotation, attention over the rotated rows; then a token: append, 8-bit decode."""
    hq, hkv, d, page, n = 8, 2, 128, 16, [300, 77]
    gen = torch.Generator().manual_seed(5)
    desc, (rope, fa) = bia.make_desc(hq, hkv, d, page), ru.make(d, 400)
    table, (qw, kw) = ru.table_of(400, d).cuda(), ru.weights(d, gen)
    kvp, pages, last, ids, n_pages = fu.page_table([x + 1 for x in n], page, 1)
    codes = [torch.zeros(n_pages, page, hkv, d, dtype=U8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(n_pages, page, hkv, dtype=U8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(2)]

    def append(rows, keys, new):
        count = [-(-x // page) for x in keys]
        host = fu.indptr_of(new), fu.indptr_of(count), ints([x - (c - 1) * page for x, c in zip(keys, count)])
        at = torch.cat([i[:c] for i, c in zip(ids, count)])
        dev = host[0].cuda(), host[1].cuda(), at.cuda(), host[2].cuda()
        q, k = (torch.empty(rows.shape[0], h, d, dtype=BF16, device="cuda") for h in (hq, hkv))
        bia.bia_append_paged_kv_fp8_rope(desc, rope, table, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], *codes, *scales,
                                         *dev, *host, q, k, None, qw, kw)
        return q, k, host, dev

    rows = ru.rows((sum(n), hq + 2 * hkv, d), gen)
    q, k, host, _ = append(rows, n, n)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    v = rows[:, hq + hkv:]
    ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, host[0], host[0]), dtype=U8, device="cuda")
    bia.bia_prefill_ragged(desc, q, k, v, host[0].cuda(), host[0].cuda(), host[0], host[0], ws, out, lse)
    for b, a in ((0, 0), (1, n[0])):
        e = a + n[b]
        fu.check(out[a:e], lse[a:e], *fu.attention_bounds(q[a:e], k[a:e], v[a:e], first=1))
    rows = ru.rows((2, hq + 2 * hkv, d), gen)
    keys = [x + 1 for x in n]
    q, k, host, dev = append(rows, keys, [1, 1])
    ws = torch.empty(bia.bia_decode_fp8_workspace_size(desc, host[1], host[2]), dtype=U8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    bia.bia_decode_paged_fp8(desc, q, *codes, *scales, *dev[1:], host[1], host[2], ws, out, lse)
    for b in range(2):
        p = torch.arange(keys[b])
        slots = (ids[b].long()[p // page] * page + p % page).cuda()
        take = [x.view(U8).flatten(0, 1)[slots].view(x.dtype) for x in (codes[0], scales[0], codes[1], scales[1])]
        fu.check(out[b:b + 1], lse[b:b + 1], *decode_bounds(q[b:b + 1], *take))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scale_of_the_scores(d):
    c = wu.Batch([700, 90], [40, 90], 8, 4, d, 16, 200, 20, seed=6)
    c.desc = bia.make_desc(8, 4, d, 16, 0.3)
    c.extend()
    c.check(sm_scale=0.3)
    c = wu.Batch([700, 90], [1, 1], 8, 4, d, 16, 200, 20, seed=6)
    c.desc = bia.make_desc(8, 4, d, 16, 0.3)
    c.decode()
    c.check(sm_scale=0.3)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_values_that_are_not_finite(what, d):
    """They reach the rows that see them, no row of another head or request; a NaN query its own row alone."""
    for call, split in (("extend", 0), ("extend", 128), ("decode", 0), ("decode", 128)):
        new = [60, 50] if call == "extend" else [1, 1]
        c = wu.Batch([500, 50], new, 8, 2, d, 16, 200, 5, seed=2, spoil=False)
        getattr(c, call)(split)
        good, row = c.out.clone(), new[0] - 1
        if what == "q":
            c.q[row, 3, 7] = float("nan")
        else:
            cache = c.k_cache if what == "k" else c.v_cache
            cache[int(c.pages[int(c.kvp[1]) - 1]), int(c.last[0]) - 1, 0, 9] = float("nan")
        getattr(c, call)(split)
        for h in [3] if what == "q" else range(4):
            seen = c.out[row, h].isnan()
            assert bool(seen[9] if what == "v" else seen.all()), (call, split, h)
            assert what == "v" or bool(c.lse[row, h].isnan())
        assert torch.equal(bits(good[:, 4:]), bits(c.out[:, 4:]))
        assert torch.equal(bits(good[new[0]:]), bits(c.out[new[0]:]))
        if what == "q":
            assert torch.equal(bits(good[:row]), bits(c.out[:row]))
            assert torch.equal(bits(good[row, :3]), bits(c.out[row, :3]))
