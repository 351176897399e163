"""The 8-bit paged cache: append and gather against the 64-bit plain form.
Both are exact: a code is the nearest e4m3 value and a value read back is
exact in bf16, so codes, scales and values are compared for equality."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def empty_cache(n_pages, page, hkv, d):
    codes = [torch.full((n_pages, page, hkv, d), 0x7F, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.full((n_pages, page, hkv), 255, dtype=torch.uint8, device=DEV) for _ in "kv"]
    return [c.view(fu.E4M3) for c in codes], [s.view(fu.E8M0) for s in scales]


def append(desc, k, v, kc, vc, ks, vs, new, table, status=None, stream=None):
    indptr, idx, last = table[:3]
    ap = fu.indptr_of(new)
    bia.bia_append_paged_kv_fp8(desc, k, v, kc, vc, ks, vs, ap.to(DEV), indptr.to(DEV), idx.to(DEV),
                                last.to(DEV), ap, indptr, last, status=status, stream=stream)


def slots_of(pages, page, lo, hi):
    p = torch.arange(lo, hi)
    return (pages.long()[p // page] * page + p % page).to(DEV)


def expect(cache, scale, slots, rows):
    codes, e = fu.quantise(rows)
    hkv, d = cache.shape[2:]
    got = cache.view(torch.uint8).view(-1, hkv, d)[slots].view(fu.E4M3).double()
    assert torch.equal(got.nan_to_num(999.0), codes.nan_to_num(999.0))
    assert torch.equal(scale.view(torch.uint8).view(-1, hkv)[slots].int(), (e + 127).int())


@pytest.mark.parametrize("hkv,d,page,lens,new", [
    (8, 128, 16, [40, 1, 300, 16], [40, 1, 7, 0]),
    (1, 64, 1, [5, 900], [5, 900]),
    (2, 96, 8, [17, 64], [16, 33]),
    (4, 256, 256, [257, 3], [200, 2]),
    (8, 128, 1, list(range(1, 70)), [1] * 69),
])
@pytest.mark.parametrize("fused", [False, True])
def test_append_writes_the_nearest_codes(hkv, d, page, lens, new, fused):
    g = torch.Generator(device=DEV).manual_seed(11)
    table = fu.page_table(lens, page, 5)
    (kc, vc), (ks, vs) = empty_cache(table[4], page, hkv, d)
    proj = fu.rows((sum(new), 3 * hkv, d), g)
    k, v = proj[:, hkv:2 * hkv], proj[:, 2 * hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    before = [t.view(torch.uint8).clone() for t in (kc, vc, ks, vs)]
    status = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    append(bia.make_desc(hkv, hkv, d, page), k, v, kc, vc, ks, vs, new, table, status)
    assert status.item() == 0
    touched, at = [], 0
    for b, n in enumerate(new):
        s = slots_of(table[3][b], page, lens[b] - n, lens[b])
        expect(kc, ks, s, k[at:at + n])
        expect(vc, vs, s, v[at:at + n])
        touched.append(s)
        at += n
    keep = torch.ones(table[4] * page, dtype=torch.bool, device=DEV)
    keep[torch.cat(touched)] = False  # every other slot keeps its bytes
    for t, old in zip((kc, vc, ks, vs), before):
        now = t.view(torch.uint8).flatten(0, 1)
        assert torch.equal(now[keep], old.flatten(0, 1)[keep])


def test_append_takes_the_smallest_scale_at_every_border():
    # magnitudes at, just below and just above 448 * 2^e, subnormals, zeros,
    # the largest bf16 and non-finite elements
    vals = [0.0, 448.0, 450.0, 446.0, 447.0, 1.75, 1.7578125, 3.3895313892515355e38, 1e-38, 2.0 ** -133,
            2.0 ** -127, 2.0 ** -112, float("inf"), float("nan"), -448.0, 2.0 ** -120 * 448]
    x = torch.zeros(len(vals), 2, 64, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    noise = torch.rand(len(vals), 2, 64, generator=g, device=DEV) * 2 - 1
    for i, a in enumerate(vals):
        if a == a and abs(a) != float("inf"):
            x[i] = (noise[i] * abs(a)).bfloat16()
        x[i, :, 5] = a
    table = fu.page_table([len(vals)], 4, 1)
    (kc, vc), (ks, vs) = empty_cache(table[4], 4, 2, 64)
    append(bia.make_desc(2, 2, 64, 4), x, x.flip(0).contiguous(), kc, vc, ks, vs, [len(vals)], table)
    s = slots_of(table[3][0], 4, 0, len(vals))
    expect(kc, ks, s, x)
    expect(vc, vs, s, x.flip(0))


@pytest.mark.parametrize("hkv,d,page,lens,take", [
    (8, 128, 16, [40, 1, 300, 16], [40, 1, 123, 0]),
    (1, 64, 1, [5, 900], [5, 900]),
    (2, 96, 8, [17, 64], [16, 33]),
    (4, 256, 256, [257, 3], [200, 3]),
])
def test_gather_reads_back_exactly(hkv, d, page, lens, take):
    g = torch.Generator(device=DEV).manual_seed(12)
    table = fu.page_table(lens, page, 6)
    rk = [fu.rows((n, hkv, d), g) for n in lens]
    rv = [fu.rows((n, hkv, d), g) for n in lens]
    kc, vc, ks, vs = fu.make_cache(rk, rv, table[3], page, table[4])
    op = fu.indptr_of(take)
    ko = torch.full((sum(take), hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vo = torch.full_like(ko, float("nan"))
    status = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    indptr, idx, last = table[:3]
    bia.bia_gather_paged_kv_fp8(bia.make_desc(hkv, hkv, d, page), kc, vc, ks, vs, ko, vo, op.to(DEV),
                                indptr.to(DEV), idx.to(DEV), last.to(DEV), op, indptr, last,
                                status=status)
    assert status.item() == 0
    for b, n in enumerate(take):
        for out, r in ((ko, rk), (vo, rv)):
            c, e = fu.quantise(r[b][:n])
            want = c * torch.exp2(e.double())[..., None]
            assert torch.equal(out[op[b]:op[b] + n].double(), want)


def test_a_cache_past_32_bits():
    """Codes on both sides of byte 2^32 of the cache and at its end: what is
    appended there reads back, and decodes to the bits a small cache gives."""
    hkv, d, page, n_pages = 8, 128, 16, 300_000  # 4.9 GB of codes each
    at = 2 ** 32 // (page * hkv * d)
    far = torch.tensor([at - 1, at, n_pages - 1, 0], dtype=torch.int32)
    lens = [60]
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v, q = fu.rows((60, hkv, d), g), fu.rows((60, hkv, d), g), fu.rows((1, 32, d), g)
    desc = bia.make_desc(32, hkv, d, page)
    indptr, last = fu.indptr_of([4]), torch.tensor([12], dtype=torch.int32)
    got = []
    for pages, ids in ((n_pages, far), (4, torch.arange(4, dtype=torch.int32))):
        cache = [torch.empty((pages, page, hkv, d), dtype=torch.uint8, device=DEV).view(fu.E4M3)
                 for _ in "kv"]
        scale = [torch.empty((pages, page, hkv), dtype=torch.uint8, device=DEV).view(fu.E8M0)
                 for _ in "kv"]
        append(desc, k, v, *cache, *scale, lens, (indptr, ids, last))
        slots = slots_of(ids, page, 0, 60)
        for c, e, r in zip(cache, scale, (k, v)):
            expect(c, e, slots, r)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        op, dev = fu.indptr_of(lens), (indptr.to(DEV), ids.to(DEV), last.to(DEV))
        bia.bia_gather_paged_kv_fp8(desc, *cache, *scale, ko, vo, op.to(DEV), *dev, op, indptr, last)
        ws = torch.empty(bia.bia_decode_fp8_workspace_size(desc, indptr, last), dtype=torch.uint8,
                         device=DEV)
        out, lse = torch.empty_like(q), torch.empty((1, 32), device=DEV)
        bia.bia_decode_paged_fp8(desc, q, *cache, *scale, *dev, indptr, last, ws, out, lse)
        assert bia.bia_read_status(ws) == 0
        got.append((ko, vo, out, lse))
        del cache, scale
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_a_whole_code_table_reads_back_exactly():
    # every code under every scale byte that append can write, and the e8m0
    # bytes 0 and 255 of a foreign cache
    scales = list(range(7, 248)) + [255]
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(1, 1, 1, 256)
    kc = codes.repeat(len(scales), 1, 1, 1).view(fu.E4M3)
    ks = torch.tensor(scales, dtype=torch.uint8, device=DEV).view(-1, 1, 1).view(fu.E8M0)
    n = len(scales)
    ip, last = fu.indptr_of([n]), torch.tensor([1], dtype=torch.int32)
    idx = torch.arange(n, dtype=torch.int32, device=DEV)
    ko = torch.empty(n, 1, 256, dtype=torch.bfloat16, device=DEV)
    vo = torch.empty_like(ko)
    bia.bia_gather_paged_kv_fp8(bia.make_desc(1, 1, 256, 1), kc, kc, ks, ks, ko, vo, ip.to(DEV),
                                ip.to(DEV), idx, last.to(DEV), ip, ip, last)
    want = fu.cache_values(kc, ks).view(n, 1, 256)
    want[-1] = float("nan")
    # codes 256 .. 448 under 2^120 are 2^128 and more, past bf16's largest
    # value (255 * 2^120): infinities; every other value is a bf16 number
    want = torch.where(want.abs() >= 2.0 ** 128, want.sign() * float("inf"), want)
    assert torch.equal(torch.isnan(want), torch.isnan(ko))
    assert torch.equal(ko.double().nan_to_num(0.0), want.nan_to_num(0.0))
    assert torch.equal(ko.view(torch.int16), vo.view(torch.int16))


def test_a_bad_page_is_skipped_and_reported():
    hkv, d, page, lens = 2, 128, 16, [50, 40]
    g = torch.Generator(device=DEV).manual_seed(2)
    indptr, idx, last, pages, total = fu.page_table(lens, page, 8)
    idx[1], idx[5] = total, -4  # request 0 keys 16..31, request 1 keys 16..31
    rk = fu.rows((sum(lens), hkv, d), g)
    (kc, vc), (ks, vs) = empty_cache(total, page, hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = bia.make_desc(hkv, hkv, d, page)
    table = (indptr, idx, last)
    append(desc, rk, rk, kc, vc, ks, vs, lens, table, status)
    assert bia.bia_read_status(status) == 1
    op = fu.indptr_of(lens)
    ko = torch.full((sum(lens), hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    bia.bia_gather_paged_kv_fp8(desc, kc, vc, ks, vs, ko, vo, op.to(DEV), indptr.to(DEV),
                                idx.to(DEV), last.to(DEV), op, indptr, last, status=status)
    assert bia.bia_read_status(status) == 1
    c, e = fu.quantise(rk)
    want = c * torch.exp2(e.double())[..., None]
    want[16:32] = 0
    want[lens[0] + 16:lens[0] + 32] = 0
    assert torch.equal(ko.double(), want) and torch.equal(vo.double(), want)


def test_append_on_another_stream_follows_that_stream():
    hkv, d, page, n = 8, 128, 16, 4000
    g = torch.Generator(device=DEV).manual_seed(4)
    table = fu.page_table([n], page, 2)
    (kc, vc), (ks, vs) = empty_cache(table[4], page, hkv, d)
    x = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device=DEV)
    src = fu.rows((n, hkv, d), g)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(20):
            x.mul_(0.5)
        x.copy_(src)
        append(bia.make_desc(hkv, hkv, d, page), x, x, kc, vc, ks, vs, [n], table)
    st.synchronize()
    expect(kc, ks, slots_of(table[3][0], page, 0, n), src)
