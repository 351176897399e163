"""Norm and rotation of queries and keys, to rows and into the paged caches, against the definition in
64 bits (tests/rope_util.py derives the bounds) and against the calls they join."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import rope_util as ru

pytestmark = pytest.mark.gpu
BF16, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

# head counts, head_dim, rot_dim, axes, interleaved, norm
SHAPES = [
    (32, 8, 128, 128, 1, False, True),
    (32, 8, 128, 64, 3, True, True),
    (4, 1, 64, 64, 1, False, False),
    (8, 8, 64, 32, 2, False, True),
    (16, 2, 96, 96, 1, False, True),
    (6, 3, 96, 48, 3, True, False),
    (1, 1, 96, 16, 1, True, True),
    (16, 8, 256, 256, 1, False, True),
    (8, 1, 256, 128, 4, True, True),
    (5, 5, 128, 16, 1, False, False),
]


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else U8)


@pytest.mark.parametrize("hq,hkv,d,rot,axes,inter,norm", SHAPES)
@pytest.mark.parametrize("total", [1, 2, 77, 1300])
def test_rows(hq, hkv, d, rot, axes, inter, norm, total):
    gen = torch.Generator().manual_seed(total * d + hq)
    top = 40000 if total == 77 else 300
    desc = bia.make_desc(hq, hkv, d, 16)
    rope, fa = ru.make(rot, top, axes, inter, "blocks" if total == 77 else "turns")
    table = ru.table_of(top, rot)
    positions = torch.randint(0, top, (axes, total), generator=gen).int()
    positions[0, 0], positions[-1, -1] = 0, top - 1
    fused = ru.rows((total, hq + 2 * hkv, d), gen)
    q, k = fused[:, :hq], fused[:, hq:hq + hkv]
    qw, kw = ru.weights(d, gen, norm)
    qo, ko = (torch.full((total, h, d), float("nan"), dtype=BF16, device="cuda") for h in (hq, hkv))
    args = (desc, rope, table.cuda(), positions.cuda())
    bia.bia_norm_rope(*args, q, k, qo, ko, qw, kw)
    ru.check_bf16(qo, *ru.reference(q, qw, rope, fa, table, positions))
    ru.check_bf16(ko, *ru.reference(k, kw, rope, fa, table, positions))
    # a slice of the calls' tokens, dense rows, queries or keys alone: the same bits
    a, b = total // 3, max(total // 3 + 1, total * 2 // 3)
    q2, k2 = torch.empty_like(qo[a:b]), torch.empty_like(ko[a:b])
    at = positions[:, a:b].contiguous().cuda()
    bia.bia_norm_rope(*args[:3], at, q[a:b].contiguous(), None, q2, None, qw, kw)
    bia.bia_norm_rope(*args[:3], at, None, k[a:b].contiguous(), None, k2, qw, kw)
    assert torch.equal(bits(q2), bits(qo[a:b])) and torch.equal(bits(k2), bits(ko[a:b]))
    # in place, the values' columns left as they were
    v = fused[:, hq + hkv:].clone()
    bia.bia_norm_rope(*args, q, k, q, k, qw, kw)
    assert torch.equal(bits(q), bits(qo)) and torch.equal(bits(k), bits(ko))
    assert torch.equal(bits(fused[:, hq + hkv:]), bits(v))


def test_positions_outside_the_table():
    gen = torch.Generator().manual_seed(1)
    desc, (rope, fa) = bia.make_desc(4, 2, 128, 16), ru.make(64, 50, 2)
    table = ru.table_of(50, 64)
    positions = torch.tensor([[3, 50, 7, 2**31 - 1, 9], [4, 5, -1, 6, 49]], dtype=I32)
    q, k = ru.rows((5, 4, 128), gen), ru.rows((5, 2, 128), gen)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    status = torch.full((1,), 77, dtype=I32, device="cuda")
    bia.bia_norm_rope(desc, rope, table.cuda(), positions.cuda(), q, k, qo, ko, status=status)
    assert bia.bia_read_status(status) == 8
    fine = torch.tensor([0, 4])
    y, slack = ru.reference(q[fine], None, rope, fa, table, positions[:, fine])
    ru.check_bf16(qo[fine.cuda()], y, slack)
    for t, axis in ((1, 0), (2, 1), (3, 0)):
        off = torch.tensor([f for f in range(32) if fa[f] == axis]).cuda()
        assert bool(qo[t][:, off].isnan().all()) and bool(qo[t][:, off + 32].isnan().all())
        assert torch.equal(bits(qo[t][:, 64:]), bits(q[t][:, 64:]))
    bia.bia_norm_rope(desc, rope, table.cuda(), positions.clamp(0, 49).cuda(), q, k, qo, ko, status=status)
    assert bia.bia_read_status(status) == 0


def test_nothing_to_do_and_values_that_are_not_finite():
    gen = torch.Generator().manual_seed(2)
    desc, (rope, fa) = bia.make_desc(4, 2, 128, 16), ru.make(128, 50)
    table = ru.table_of(50, 128).cuda()
    none = lambda h: torch.empty(0, h, 128, dtype=BF16, device="cuda")
    at = torch.empty(1, 0, dtype=I32, device="cuda")
    status = torch.full((1,), 5, dtype=I32, device="cuda")
    bia.bia_norm_rope(desc, rope, table, at, none(4), none(2), none(4), none(2), status=status)
    assert bia.bia_read_status(status) == 0
    # a head with an infinity or a NaN does not reach its neighbours, a zero head stays zero
    q, k = ru.rows((3, 4, 128), gen), ru.rows((3, 2, 128), gen)
    q[1, 2, 5], q[1, 1, 7], q[2, 0] = float("inf"), float("nan"), 0
    qw, kw = ru.weights(128, gen)
    at = torch.tensor([[1, 2, 3]], dtype=I32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    bia.bia_norm_rope(desc, rope, table, at.cuda(), q, k, qo, ko, qw, kw)
    clean = torch.where(q.isfinite(), q, 0)
    clean[1, 1:3] = 0
    y, slack = ru.reference(clean, qw, rope, fa, table.cpu(), at)
    ok = torch.ones(3, 4, dtype=torch.bool)
    ok[1, 1:3] = False
    ru.check_bf16(qo.cpu()[ok], y[ok], slack[ok])
    assert bool(qo[1, 1].isnan().all()) and bool(qo[1, 2, [5, 69]].isnan().all())
    assert bool((qo[2, 0] == 0).all())


def append_case(keys, new, hq, hkv, d, rot, axes, inter, norm, page, seed, fp8):
    gen = torch.Generator().manual_seed(seed)
    c = type("Case", (), {})()
    c.desc, top = bia.make_desc(hq, hkv, d, page), max(keys) + 1
    c.rope, c.fa = ru.make(rot, top, axes, inter)
    c.table = ru.table_of(top, rot)
    c.kvp, c.last, c.pages, c.n_pages = ru.page_table(keys, page, gen)
    c.ap = torch.tensor([0] + new).cumsum(0).int()
    total = int(c.ap[-1])
    c.fused = ru.rows((total, hq + 2 * hkv, d), gen)
    c.q, c.k, c.v = c.fused[:, :hq], c.fused[:, hq:hq + hkv], c.fused[:, hq + hkv:]
    c.qw, c.kw = ru.weights(d, gen, norm)
    c.text = torch.cat([torch.arange(a - n, a) for a, n in zip(keys, new)]).int().expand(axes, total).contiguous()
    c.positions = torch.randint(0, top, (axes, total), generator=gen).int()
    c.slots = ru.slots_of(keys, new, page, c.kvp, c.pages)
    shape = (c.n_pages, page, hkv, d)
    if fp8:
        old = lambda s: torch.randint(0, 120, s, generator=gen, dtype=U8).cuda()
        c.caches = [old(shape).view(E4M3), old(shape).view(E4M3), old(shape[:3]).view(E8M0), old(shape[:3]).view(E8M0)]
    else:
        c.caches = [ru.rows(shape, gen), ru.rows(shape, gen)]
    c.dev = tuple(x.cuda() for x in (c.ap, c.kvp, c.pages, c.last))
    c.arrays = (*c.dev, c.ap, c.kvp, c.last)
    return c


LENGTHS = [
    ([5], [5]), ([1], [1]), ([300], [17]),
    ([40, 1, 0, 257, 16, 999], [40, 1, 0, 1, 16, 70]),
    ([7 + 3 * b % 50 for b in range(1100)], [b % 3 for b in range(1100)]),
    ([100 + b for b in range(33)], [1] * 33),
]


@pytest.mark.parametrize("keys,new", LENGTHS, ids=range(len(LENGTHS)))
@pytest.mark.parametrize("shape,page", list(zip(SHAPES, [16, 1, 8, 256, 32, 2, 64, 16, 4, 128])),
                         ids=lambda x: str(x).replace(" ", ""))
@pytest.mark.parametrize("fp8", [False, True])
def test_append(keys, new, shape, page, fp8):
    hq, hkv, d, rot, axes, inter, norm = shape
    c = append_case(keys, new, hq, hkv, d, rot, axes, inter, norm, page, len(keys) * 7 + d, fp8)
    before = [bits(x).clone() for x in c.caches]
    qo = torch.full(c.q.shape, float("nan"), dtype=BF16, device="cuda")
    status = torch.full((1,), 3, dtype=I32, device="cuda")
    table, ko = c.table.cuda(), torch.full(c.k.shape, float("nan"), dtype=BF16, device="cuda")
    if fp8:
        bia.bia_append_paged_kv_fp8_rope(c.desc, c.rope, table, c.q, c.k, c.v, *c.caches, *c.arrays, qo, ko,
                                         c.positions.cuda(), c.qw, c.kw, status)
    else:
        bia.bia_append_paged_kv_rope(c.desc, c.rope, table, c.q, c.k, c.v, *c.caches, *c.arrays, qo,
                                     c.positions.cuda(), c.qw, c.kw, status)
    assert bia.bia_read_status(status) == 0
    slots = c.slots.cuda()
    got = [x.view(U8 if fp8 else BF16).flatten(0, 1)[slots] for x in c.caches]
    yk, slack = ru.reference(c.k, c.kw, c.rope, c.fa, c.table, c.positions)
    # the rows are the ones that the rotation alone gives
    q1, k1 = torch.empty_like(qo), torch.empty_like(ko)
    if qo.shape[0]:
        bia.bia_norm_rope(c.desc, c.rope, table, c.positions.cuda(), c.q, c.k, q1, k1, c.qw, c.kw)
    assert torch.equal(bits(qo), bits(q1))
    if fp8:
        ru.check_codes(got[0].view(E4M3), got[2], yk, slack)
        assert torch.equal(bits(ko), bits(k1))
    else:
        assert torch.equal(bits(got[0]), bits(k1))
        ru.check_bf16(got[0], yk, slack)
    # values, and everything else in the caches, are what the plain append leaves
    plain = [b.view(x.dtype).view(x.shape).clone() for b, x in zip(before, c.caches)]
    if fp8:
        bia.bia_append_paged_kv_fp8(c.desc, c.k, c.v, *plain, *c.arrays)
        assert torch.equal(bits(plain[1]), bits(c.caches[1])) and torch.equal(bits(plain[3]), bits(c.caches[3]))
    else:
        bia.bia_append_paged_kv(c.desc, k1, c.v.contiguous(), *plain, *c.arrays)
        assert torch.equal(bits(plain[0]), bits(c.caches[0])) and torch.equal(bits(plain[1]), bits(c.caches[1]))
    rest = torch.ones(c.n_pages * page, dtype=torch.bool, device="cuda")
    rest[slots] = False
    for b, x in zip(before, c.caches):
        assert torch.equal(b.flatten(0, 1)[rest], bits(x).flatten(0, 1)[rest])


@pytest.mark.parametrize("fp8", [False, True])
def test_key_positions_and_no_queries(fp8):
    c = append_case([40, 300, 0, 17], [3, 300, 0, 1], 8, 4, 128, 128, 1, False, True, 16, 5, fp8)
    table, more = c.table.cuda(), [x.clone() for x in c.caches]
    q1, q2 = (torch.empty(c.q.shape, dtype=BF16, device="cuda") for _ in range(2))
    if fp8:
        call = lambda q, caches, qo, at: bia.bia_append_paged_kv_fp8_rope(
            c.desc, c.rope, table, q, c.k, c.v, *caches, *c.arrays, qo, None, at, c.qw, c.kw)
    else:
        call = lambda q, caches, qo, at: bia.bia_append_paged_kv_rope(
            c.desc, c.rope, table, q, c.k, c.v, *caches, *c.arrays, qo, at, c.qw, c.kw)
    call(c.q, c.caches, q1, None)
    call(c.q, more, q2, c.text.cuda())
    assert torch.equal(bits(q1), bits(q2))
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(c.caches, more))
    more = [torch.zeros_like(x.view(U8)).view(x.dtype) if fp8 else torch.zeros_like(x) for x in more]
    call(None, more, None, None)
    slots = c.slots.cuda()
    for a, b in zip(c.caches, more):
        assert torch.equal(bits(a).flatten(0, 1)[slots], bits(b).flatten(0, 1)[slots])


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_bad_positions(fp8):
    """A token without a page is skipped and noted, its query is not; a position outside the table is NaN."""
    c = append_case([48, 20], [48, 4], 8, 4, 64, 64, 1, False, False, 16, 9, fp8)
    c.pages[1], c.pages[4] = c.n_pages, -1
    c.dev[2].copy_(c.pages)
    c.positions[0, 3] = c.rope.num_positions
    before = [bits(x).clone() for x in c.caches]
    qo, status = torch.empty(c.q.shape, dtype=BF16, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    if fp8:
        bia.bia_append_paged_kv_fp8_rope(c.desc, c.rope, c.table.cuda(), c.q, c.k, c.v, *c.caches, *c.arrays, qo, None,
                                         c.positions.cuda(), status=status)
    else:
        bia.bia_append_paged_kv_rope(c.desc, c.rope, c.table.cuda(), c.q, c.k, c.v, *c.caches, *c.arrays, qo,
                                     c.positions.cuda(), status=status)
    assert bia.bia_read_status(status) == 1 | 8
    ok = torch.ones(52, dtype=torch.bool)
    ok[16:32] = ok[48:] = False  # request 0's second page, request 1's last
    y, slack = ru.reference(c.k, None, c.rope, c.fa, c.table, c.positions.clamp(max=c.rope.num_positions - 1))
    yq, qslack = ru.reference(c.q, None, c.rope, c.fa, c.table, c.positions.clamp(max=c.rope.num_positions - 1))
    fine = torch.ones(52, dtype=torch.bool)
    fine[3] = False
    ru.check_bf16(qo.cpu()[fine], yq[fine], qslack[fine])
    assert bool(qo[3].isnan().all())
    pages = c.pages.clone()
    pages[1] = pages[4] = 0
    slots = ru.slots_of([48, 20], [48, 4], 16, c.kvp, pages)
    rows = c.caches[0].view(U8 if fp8 else BF16).flatten(0, 1)[slots.cuda()]
    if fp8:
        scale = c.caches[2].view(U8).flatten(0, 1)[slots.cuda()]
        ru.check_codes(rows.view(E4M3)[(ok & fine).cuda()], scale[(ok & fine).cuda()], y[ok & fine], slack[ok & fine])
        assert bool(((rows[3] & 0x7F) == 0x7F).all())
    else:
        ru.check_bf16(rows.cpu()[ok & fine], y[ok & fine], slack[ok & fine])
        assert bool(rows[3].isnan().all())
    rest = torch.ones(c.n_pages * 16, dtype=torch.bool, device="cuda")
    rest[slots[ok].cuda()] = False
    for b, x in zip(before, c.caches):
        assert torch.equal(b.flatten(0, 1)[rest], bits(x).flatten(0, 1)[rest])


def test_codes_of_values_that_are_not_finite():
    """Stored as NaN, under the scale of the row's finite values; a row of zeros under the smallest."""
    c = append_case([4], [4], 2, 2, 64, 16, 1, False, False, 4, 3, True)
    c.k[0, 0, 40], c.k[1, 1, 63], c.k[2, 0] = float("inf"), float("nan"), 0
    c.k[3, 1] = 3e38
    bia.bia_append_paged_kv_fp8_rope(c.desc, c.rope, c.table.cuda(), None, c.k, c.v, *c.caches, *c.arrays, None)
    rows = c.caches[0].view(U8).flatten(0, 1)[c.slots.cuda()].view(E4M3).float()
    scale = c.caches[2].view(U8).flatten(0, 1)[c.slots.cuda()]
    for t, h, i in ((0, 0, 40), (1, 1, 63)):
        assert bool(rows[t, h, i].isnan()) and int(rows[t, h].isnan().sum()) == 1
    k = torch.where(c.k.isfinite(), c.k, 0)
    y, slack = ru.reference(k[:3], None, c.rope, c.fa, c.table, c.text[:, :3])
    ru.check_codes(torch.where(rows.isnan(), 0, rows)[:3], scale[:3], y, slack)
    assert int(scale[2, 0]) == 7 and bool((rows[2, 0] == 0).all())
    assert int(scale[3, 1]) == 247 and bool((rows[3, 1, 16:] == 240).all() | (rows[3, 1, 16:] == 224).all())


def test_captured_append_follows_its_arrays():
    """One captured step, replayed while lengths, page table, positions and rows change."""
    keys, page = [40, 7, 100], 8
    c = append_case([k + 30 for k in keys], [1, 1, 1], 8, 2, 128, 128, 1, False, True, page, 11, False)
    table, qo = c.table.cuda(), torch.empty(c.q.shape, dtype=BF16, device="cuda")
    last, status = c.last.cuda(), torch.zeros(1, dtype=I32, device="cuda")
    kvp = c.kvp.clone()
    dev = (c.dev[0], kvp.cuda(), c.dev[2], last)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    call = lambda: bia.bia_append_paged_kv_rope(c.desc, c.rope, table, c.q, c.k, c.v, *c.caches, *dev, c.ap, c.kvp, c.last,
                                                qo, None, c.qw, c.kw, status)
    with torch.cuda.graph(graph, stream=stream):
        call()
    gen = torch.Generator().manual_seed(12)
    for step in range(5):
        now = [k + 5 * step for k in keys]
        count = [-(-k // page) for k in now]
        pages = torch.cat([c.pages[int(c.kvp[b]):int(c.kvp[b]) + n] for b, n in enumerate(count)])
        indptr = torch.tensor([0] + count).cumsum(0).int()
        dev[1].copy_(indptr)
        dev[2][:len(pages)].copy_(pages)
        dev[3].copy_(torch.tensor([k - (n - 1) * page for k, n in zip(now, count)]).int())
        c.fused.copy_(ru.rows(c.fused.shape, gen))
        graph.replay()
        assert bia.bia_read_status(status) == 0
        at = torch.tensor([[k - 1 for k in now]]).int()
        ru.check_bf16(qo, *ru.reference(c.q, c.qw, c.rope, c.fa, c.table, at))
        slots = ru.slots_of(now, [1, 1, 1], page, indptr, pages).cuda()
        ru.check_bf16(c.caches[0].flatten(0, 1)[slots], *ru.reference(c.k, c.kw, c.rope, c.fa, c.table, at))
        assert torch.equal(bits(c.caches[1].flatten(0, 1)[slots]), bits(c.v))


def test_on_another_stream_and_in_any_batch():
    """The call runs on the stream it is given; a request's bits do not depend on its batch."""
    keys, new = [300, 64, 900, 33, 5], [300, 1, 450, 33, 5]
    c = append_case(keys, new, 16, 4, 128, 128, 1, False, True, 16, 21, True)
    s, qo, ko = torch.cuda.Stream(), *(torch.empty(x.shape, dtype=BF16, device="cuda") for x in (c.q, c.k))
    table = c.table.cuda()
    s.wait_stream(torch.cuda.current_stream())
    bia.bia_append_paged_kv_fp8_rope(c.desc, c.rope, table, c.q, c.k, c.v, *c.caches, *c.arrays, qo, ko, None, c.qw, c.kw,
                                     stream=s)
    s.synchronize()
    for b in range(5):
        one = [torch.zeros_like(x.view(U8)).view(x.dtype) for x in c.caches]
        a, n = int(c.ap[b]), new[b]
        host = (torch.tensor([0, n]).int(), torch.tensor([0, int(c.kvp[b + 1] - c.kvp[b])]).int(), c.last[b:b + 1])
        pages = c.pages[int(c.kvp[b]):int(c.kvp[b + 1])].contiguous()
        q1, k1 = torch.empty_like(qo[a:a + n]), torch.empty_like(ko[a:a + n])
        bia.bia_append_paged_kv_fp8_rope(c.desc, c.rope, table, c.q[a:a + n], c.k[a:a + n], c.v[a:a + n], *one,
                                         host[0].cuda(), host[1].cuda(), pages.cuda(), host[2].cuda(), *host, q1, k1, None,
                                         c.qw, c.kw)
        assert torch.equal(bits(q1), bits(qo[a:a + n])) and torch.equal(bits(k1), bits(ko[a:a + n]))
        slots = c.slots[a:a + n].cuda()
        for x, y in zip(one, c.caches):
            assert torch.equal(bits(x).flatten(0, 1)[slots], bits(y).flatten(0, 1)[slots])
