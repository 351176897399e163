"""Attention of packed sequences over contiguous keys and values against 64
bits, its strides, masks and invariance, and the 8-bit cache's calls run
together."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu
from tests.gpu_util import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(q, k, v, q_lens, kv_lens, causal=True, split=0, lse=True, sm_scale=0.0, stream=None):
    hq, d = q.shape[1:]
    desc = bia.make_desc(hq, k.shape[1], d, 1, sm_scale)
    qo, kv = fu.indptr_of(q_lens), fu.indptr_of(kv_lens)
    ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, qo, kv, causal, split),
                     dtype=torch.uint8, device=DEV)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    l = torch.full(q.shape[:2], float("nan"), device=DEV) if lse else None
    bia.bia_prefill_ragged(desc, q, k, v, qo.to(DEV), kv.to(DEV), qo, kv, ws, out, l, causal=causal,
                           split_size=split, stream=stream)
    assert bia.bia_read_status(ws, stream) == 0
    return out, l


def check(q, k, v, q_lens, kv_lens, out, lse, causal=True, sm_scale=None):
    qa = ka = 0
    for ql, kl in zip(q_lens, kv_lens):
        if ql:
            want = fu.attention_bounds(q[qa:qa + ql], k[ka:ka + kl], v[ka:ka + kl],
                                       kl - ql + 1 if causal else None, sm_scale)
            fu.check(out[qa:qa + ql], lse[qa:qa + ql], *want)
        qa, ka = qa + ql, ka + kl


def draw(hq, hkv, d, q_lens, kv_lens, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (fu.rows((sum(q_lens), hq, d), g), fu.rows((sum(kv_lens), hkv, d), g),
            fu.rows((sum(kv_lens), hkv, d), g))


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (4, 1), (16, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_against_64_bits(d, hq, hkv, causal):
    q_lens = [1, 17, 128, 0, 129, 300, 513, 5]
    kv_lens = [1, 17, 128, 0, 129, 300, 700, 400]
    q, k, v = draw(hq, hkv, d, q_lens, kv_lens, d + hq)
    out, lse = run(q, k, v, q_lens, kv_lens, causal)
    check(q, k, v, q_lens, kv_lens, out, lse, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_without_keys(d):
    q_lens, kv_lens = [5, 200, 3], [0, 130, 0]
    q, k, v = draw(4, 2, d, q_lens, kv_lens)
    out, lse = run(q, k, v, q_lens, kv_lens, causal=False)
    check(q, k, v, q_lens, kv_lens, out, lse, False)
    out, lse = run(q[:5], k[:0], v[:0], [5], [0], causal=False)
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("d,split", [(64, 128), (128, 256), (128, 4096), (256, 256), (96, 384)])
def test_long_keys_in_splits(d, split):
    q_lens, kv_lens = [40, 300, 1], [5000, 1300, 4500]
    q, k, v = draw(8, 2, d, q_lens, kv_lens, 3)
    for causal in (True, False):
        out, lse = run(q, k, v, q_lens, kv_lens, causal, split)
        check(q, k, v, q_lens, kv_lens, out, lse, causal)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_slices_of_a_fused_projection(d):
    hq, hkv, lens = 8, 2, [100, 1, 333]
    g = torch.Generator(device=DEV).manual_seed(9)
    rows = fu.rows((sum(lens), hq + 2 * hkv, d), g)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    out, lse = run(q, k, v, lens, lens)
    o2, l2 = run(q.contiguous(), k.contiguous(), v.contiguous(), lens, lens)
    assert same_bits(out, o2) and same_bits(lse, l2)
    check(q, k, v, lens, lens, out, lse)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_neighbour_does_not_reach_a_request(d, bad):
    # requests 0 and 2 hold nothing finite; request 1's rows keep their bits
    q_lens, kv_lens = [70, 150, 40], [70, 150, 300]
    q, k, v = draw(4, 2, d, q_lens, kv_lens, 5)
    for causal in (True, False):
        want, wl = run(q[70:220], k[70:220], v[70:220], [150], [150], causal)
        for t in (k, v):
            t[:70], t[220:] = bad, bad
        q[:70], q[220:] = bad, bad
        out, lse = run(q, k, v, q_lens, kv_lens, causal)
        assert same_bits(out[70:220], want) and same_bits(lse[70:220], wl)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_row_has_its_bits_in_any_batch_and_chunking(d):
    hq, hkv, n = 8, 2, 700
    q, k, v = draw(hq, hkv, d, [n], [n], 6)
    want, wl = run(q, k, v, [n], [n], split=256)
    q2, k2, v2 = draw(hq, hkv, d, [300, 90], [310, 1000], 7)
    out, lse = run(torch.cat([q2[:300], q, q2[300:]]), torch.cat([k2[:310], k, k2[310:]]),
                   torch.cat([v2[:310], v, v2[310:]]), [300, n, 90], [310, n, 1000], split=256)
    assert same_bits(out[300:300 + n], want) and same_bits(lse[300:300 + n], wl)
    for chunk in (32, 100, 129, 1):  # on the q-tile grid and off it, one token too
        for a in range(0, n, max(chunk, 150) if chunk == 1 else chunk):
            e = min(n, a + chunk)
            o, l = run(q[a:e], k[:e], v[:e], [e - a], [e], split=256)
            assert same_bits(o, want[a:e]) and same_bits(l, wl[a:e]), (chunk, a)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_more_items_than_sms(d, causal):
    """Several items a CTA, of every size from a row to eight blocks, each
    with a V tail of its own: against 64 bits, and bit for bit as alone."""
    g = torch.Generator().manual_seed(d)
    q_lens = torch.randint(0, 130, (60,), generator=g).tolist()
    extra = torch.randint(0, 900, (60,), generator=g).tolist()
    kv_lens = [x + (e if i % 3 else 0) for i, (x, e) in enumerate(zip(q_lens, extra))]
    q, k, v = draw(8, 4, d, q_lens, kv_lens, d)
    out, lse = run(q, k, v, q_lens, kv_lens, causal)
    check(q, k, v, q_lens, kv_lens, out, lse, causal)
    qa = ka = 0
    for i, (x, y) in enumerate(zip(q_lens, kv_lens)):
        if i % 7 == 0 and x:
            one, l = run(q[qa:qa + x], k[ka:ka + y], v[ka:ka + y], [x], [y], causal)
            assert same_bits(one, out[qa:qa + x]) and same_bits(l, lse[qa:qa + x])
        qa, ka = qa + x, ka + y


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_splits_folded_in_the_cta_have_the_merge_s_bits(d, causal):
    """A batch with enough q tiles folds each row's splits where they are
    computed; one request of it alone has them merged by a kernel."""
    hq, hkv, split = 32, 8, 256
    q_lens, kv_lens = [1500, 700, 1, 64, 0, 1100, 900, 1500], [1500, 2900, 1300, 64, 7, 1101, 900, 1700]
    q, k, v = draw(hq, hkv, d, q_lens, kv_lens, 5)
    desc = bia.make_desc(hq, hkv, d, 1)
    need = [bia.bia_prefill_ragged_workspace_size(desc, fu.indptr_of(a), fu.indptr_of(b), causal, split)
            for a, b in ((q_lens, kv_lens), (q_lens[1:2], kv_lens[1:2]))]
    assert need[0] < need[1]  # one state a CTA, not one a row and split
    out, lse = run(q, k, v, q_lens, kv_lens, causal, split)
    qa = ka = 0
    for x, y in zip(q_lens, kv_lens):
        if x:
            one, l = run(q[qa:qa + x], k[ka:ka + y], v[ka:ka + y], [x], [y], causal, split)
            assert same_bits(one, out[qa:qa + x]) and same_bits(l, lse[qa:qa + x])
        qa, ka = qa + x, ka + y
    for i in (1, 2, 5):
        qa, ka = sum(q_lens[:i]), sum(kv_lens[:i])
        x, y = q_lens[i], kv_lens[i]
        check(q[qa:qa + x], k[ka:ka + y], v[ka:ka + y], [x], [y], out[qa:qa + x], lse[qa:qa + x], causal)


def test_rows_past_32_bits_and_more_requests_than_a_plan_s_chunk():
    """2700 requests, q and out of more than 2^31 elements: as each alone."""
    hq, hkv, d = 64, 8, 128
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 201, (2700,), generator=g).tolist()
    assert sum(lens) * hq * d > 2 ** 31
    gd = torch.Generator(device=DEV).manual_seed(4)
    q, k, v = (torch.empty((sum(lens), h, d), dtype=torch.bfloat16, device=DEV).normal_(generator=gd)
               for h in (hq, hkv, hkv))
    out, lse = run(q, k, v, lens, lens)
    at = fu.indptr_of(lens).tolist()
    for i in (0, 1, 511, 512, 1024, 1500, 2698, 2699):
        a, b = at[i], at[i + 1]
        if a == b:
            continue
        one, l = run(q[a:b], k[a:b], v[a:b], lens[i:i + 1], lens[i:i + 1])
        assert same_bits(one, out[a:b]) and same_bits(l, lse[a:b])
    a, b = at[2690], at[2700]
    check(q[a:b], k[a:b], v[a:b], lens[2690:], lens[2690:], out[a:b], lse[a:b])
    assert torch.isfinite(lse).all()


def test_scale_stream_and_lse():
    lens = [257, 64]
    q, k, v = draw(4, 4, 128, lens, lens, 8)
    out, lse = run(q, k, v, lens, lens, sm_scale=0.3)
    check(q, k, v, lens, lens, out, lse, sm_scale=0.3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o2, l2 = run(q, k, v, lens, lens, sm_scale=0.3)
    st.synchronize()
    assert same_bits(out, o2) and same_bits(lse, l2)
    assert same_bits(run(q, k, v, lens, lens, sm_scale=0.3, lse=False)[0], out)


def test_captured_prompt_replays():
    lens = [300, 5000]
    q, k, v = draw(8, 2, 128, lens, lens, 10)
    want, wl = run(q, k, v, lens, lens)
    desc = bia.make_desc(8, 2, 128, 1)
    ip = fu.indptr_of(lens)
    dev = ip.to(DEV)
    ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, ip, ip), dtype=torch.uint8,
                     device=DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bia.bia_prefill_ragged(desc, q, k, v, dev, dev, ip, ip, ws, out, lse)
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want) and same_bits(lse, wl)
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    check(q, k, v, lens, lens, out, lse)


def two_calls():
    """A call that folds its splits in the CTAs and one that merges them."""
    calls = []
    for i, (hq, hkv, q_lens, kv_lens) in enumerate((
            (32, 8, [2000, 1500], [2000, 6000]), (8, 2, [100, 1, 300], [5000, 4500, 300]))):
        calls.append((hq, hkv, q_lens, kv_lens, draw(hq, hkv, 128, q_lens, kv_lens, 20 + i)))
    return calls


def enqueue(hq, hkv, q_lens, kv_lens, rows, ws=None):
    desc = bia.make_desc(hq, hkv, 128, 1)
    qo, kv = fu.indptr_of(q_lens), fu.indptr_of(kv_lens)
    if ws is None:
        ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, qo, kv), dtype=torch.uint8,
                         device=DEV)
    out, lse = torch.empty_like(rows[0]), torch.empty(rows[0].shape[:2], device=DEV)
    dev = qo.to(DEV), kv.to(DEV)

    def call():
        bia.bia_prefill_ragged(desc, *rows, *dev, qo, kv, ws, out, lse)
    return call, out, lse, ws


def test_two_graphs_share_one_workspace():
    calls = two_calls()
    want = [run(*rows, ql, kl) for _, _, ql, kl, rows in calls]
    ws = torch.empty(max(enqueue(*c)[3].numel() for c in calls), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for c in calls:
        call, out, lse, _ = enqueue(*c, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, call))
        outs.append((out, lse))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert same_bits(o, wo) and same_bits(l, wl)


def test_calls_on_two_streams_with_their_own_workspaces():
    calls = two_calls()
    want = [run(*rows, ql, kl) for _, _, ql, kl, rows in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            call, out, lse, ws = enqueue(*calls[i % 2])
            call()
            got.append((out, lse, ws))
    torch.cuda.synchronize()
    for i, (o, l, _) in enumerate(got):
        assert same_bits(o, want[i % 2][0]) and same_bits(l, want[i % 2][1])


@pytest.mark.parametrize("d", [64, 96, 128])
def test_calls_with_and_without_a_plan_take_the_same_bits(d):
    """32 requests find their units themselves, 33 and more have them planned,
    as have calls with more items than SMs: the same rows either way."""
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 40, (33,), generator=g).tolist()
    lens[0], lens[5], lens[31], lens[32] = 0, 300, 0, 9
    kv_lens = [x + 50 * (i % 4) for i, x in enumerate(lens)]
    q, k, v = draw(4, 2, d, lens, kv_lens, 6)
    out, lse = run(q, k, v, lens, kv_lens)  # planned
    n, m = sum(lens[:32]), sum(kv_lens[:32])
    one, l = run(q[:n], k[:m], v[:m], lens[:32], kv_lens[:32])  # not
    assert same_bits(one, out[:n]) and same_bits(l, lse[:n])
    check(q, k, v, lens, kv_lens, out, lse)
    launches = []
    for count in (32, 33):
        before = bia.bia_launch_count()
        a, b = sum(lens[:count]), sum(kv_lens[:count])
        run(q[:a], k[:b], v[:b], lens[:count], kv_lens[:count])
        launches.append(bia.bia_launch_count() - before)
    assert launches == [1, 2]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("which", ["q", "kv"])
def test_device_lengths_that_end_elsewhere_compute_nothing(d, which):
    """Device arrays that count the same tiles and splits as the host's but end
    at another row: the buffers are as long as the host's say."""
    lens = [100, 100]
    q, k, v = draw(4, 2, d, lens, lens, 1)
    desc = bia.make_desc(4, 2, d, 1)
    ip = fu.indptr_of(lens)
    other = fu.indptr_of([100, 99])
    ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, ip, ip), dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    qo, kv = ((other, ip) if which == "q" else (ip, other))
    bia.bia_prefill_ragged(desc, q, k, v, qo.to(DEV), kv.to(DEV), ip, ip, ws, out, lse,
                           causal=which == "q")
    assert bia.bia_read_status(ws) != 0
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("d,hq,hkv,page", [(128, 32, 8, 16), (64, 8, 1, 1), (256, 4, 2, 32)])
def test_a_server_with_an_8_bit_cache(d, hq, hkv, page):
    """Prompts in two chunks (the second over the prefix read back), then
    tokens one at a time, all from the 8-bit cache."""
    desc = bia.make_desc(hq, hkv, d, page)
    g = torch.Generator(device=DEV).manual_seed(21)
    total = [150, 37, 400]
    first = [100, 37, 256]  # the first chunk
    steps = 4
    full = [n + steps for n in total]
    indptr_f, _, _, pages, n_pages = fu.page_table(full, page, 3)
    proj = [fu.rows((n, hq + 2 * hkv, d), g) for n in full]  # each request's fused rows
    kc, vc, ks, vs = fu.make_cache([p[:0, :hkv] for p in proj], [p[:0, :hkv] for p in proj],
                                   [x[:0] for x in pages], page, n_pages)

    def table(lens):
        count = [-(-n // page) for n in lens]
        ip = fu.indptr_of(count)
        ids = torch.cat([pages[i][:c] for i, c in enumerate(count)])
        last = torch.tensor([n - (c - 1) * page for n, c in zip(lens, count)], dtype=torch.int32)
        return ip, ids, last

    def values(b, n):  # what the cache has to hold of request b
        c = []
        for s in (slice(hq, hq + hkv), slice(hq + hkv, None)):
            codes, e = fu.quantise(proj[b][:n, s])
            c.append(codes * torch.exp2(e.double())[..., None])
        return c

    def put(lo, hi):
        ip, ids, last = table(hi)
        rows = torch.cat([p[a:e] for p, a, e in zip(proj, lo, hi)])
        ap = fu.indptr_of([e - a for a, e in zip(lo, hi)])
        bia.bia_append_paged_kv_fp8(desc, rows[:, hq:hq + hkv], rows[:, hq + hkv:], kc, vc, ks, vs,
                                    ap.to(DEV), ip.to(DEV), ids.to(DEV), last.to(DEV), ap, ip, last)
        return rows[:, :hq], ip, ids, last

    lo = [0, 0, 0]
    for hi in (first, total):
        q, ip, ids, last = put(lo, hi)
        kv = fu.indptr_of(hi)
        k = torch.empty(sum(hi), hkv, d, dtype=torch.bfloat16, device=DEV)
        v = torch.empty_like(k)
        bia.bia_gather_paged_kv_fp8(desc, kc, vc, ks, vs, k, v, kv.to(DEV), ip.to(DEV), ids.to(DEV),
                                    last.to(DEV), kv, ip, last)
        q_lens = [e - a for a, e in zip(lo, hi)]
        out, lse = run(q, k, v, q_lens, hi)
        at = 0
        for b in range(3):
            kb, vb = values(b, hi[b])
            assert torch.equal(k[kv[b]:kv[b + 1]].double(), kb)
            n = q_lens[b]
            if n:
                fu.check(out[at:at + n], lse[at:at + n],
                         *fu.attention_bounds(q[at:at + n], kb, vb, lo[b] + 1))
            at += n
        lo = hi
    for _ in range(steps):
        hi = [n + 1 for n in lo]
        q, ip, ids, last = put(lo, hi)
        q = q.contiguous()
        ws = torch.empty(bia.bia_decode_fp8_workspace_size(desc, ip, last), dtype=torch.uint8,
                         device=DEV)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        bia.bia_decode_paged_fp8(desc, q, kc, vc, ks, vs, ip.to(DEV), ids.to(DEV), last.to(DEV), ip,
                                 last, ws, out, lse)
        for b in range(3):
            kb, vb = values(b, hi[b])
            want = fu.attention_bounds(q[b:b + 1], kb, vb)
            # weights under the 8-bit terms' last place: 2^-19 of the largest
            # weight (at most 1) for every key, at the largest value
            tol = want[1] + 2.0 ** -18 * hi[b] * vb.abs().max()
            fu.check(out[b:b + 1], lse[b:b + 1], want[0], tol, want[2], want[3])
        lo = hi
