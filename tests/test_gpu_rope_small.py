"""Norms of small heads: with an epsilon of zero or next to it the squares of their elements leave fp32."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import rope_util as ru

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8

# exponents of the heads' magnitudes, bf16's subnormals at one end; the middle ones beside where fp32 squares end
SIZES = [0, -20, -36, -38, -39, -40, -41, -45, -60, -63, -66, -72, -75, -90, -120, -127, -131]


def reference(x, weight, rope, table, at):
    """ru.reference; the products of a head that is not scaled may be fp32 subnormals, two roundings of 2^-150
    each, which the root (2^40 at most there) takes up."""
    y, slack = ru.reference(x, weight, rope, None, table, at)
    r = (x.double().cpu().square().mean(-1, keepdim=True) + rope.norm_eps).rsqrt().clamp(max=2.0 ** 40)
    return y, slack + 2.0 ** -148 * r / ru.NOISE


def heads(shape, gen, spread=0):
    """Every head of another magnitude; with `spread` a head's own columns reach that many binades below it."""
    x = torch.randn(shape, generator=gen, dtype=torch.float64)
    e = torch.tensor(SIZES, dtype=torch.float64)[torch.randint(0, len(SIZES), shape[:2], generator=gen)]
    x *= torch.exp2(e)[..., None] * torch.exp2(-spread * torch.rand(shape, generator=gen, dtype=torch.float64))
    return x.to(BF16).cuda()


@pytest.mark.parametrize("hq,hkv,d,rot,inter", [(8, 4, 128, 128, False), (6, 3, 96, 48, False), (4, 4, 64, 64, True),
                                                (4, 1, 256, 128, True)])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 2.0 ** -81, 2.0 ** -80, 1e-12])
@pytest.mark.parametrize("spread", [0, 30])
def test_small_heads(hq, hkv, d, rot, inter, eps, spread):
    gen = torch.Generator().manual_seed(d)
    total, page = 60, 16
    desc, rope = bia.make_desc(hq, hkv, d, page), bia.make_rope(rot, 100, interleaved=inter, norm_eps=eps)
    table = ru.table_of(100, rot)
    at = torch.arange(total).int()[None]
    q, k = heads((total, hq, d), gen, spread), heads((total, hkv, d), gen, spread)
    v = torch.zeros_like(k)
    qw, kw = ru.weights(d, gen)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    bia.bia_norm_rope(desc, rope, table.cuda(), at.cuda(), q, k, qo, ko, qw, kw)
    y, slack = reference(q, qw, rope, table, at)
    some = (q.cpu() != 0).any(-1)  # 0 / sqrt(0 + 0) has no value
    assert eps > 0 or bool(some.any())
    ok = some if eps == 0 else torch.ones_like(some)
    ru.check_bf16(qo.cpu()[ok], y[ok], slack[ok])
    # into the pages: the same rows, and the codes of the same fp32 rows
    host = torch.tensor([0, total]).int(), torch.tensor([0, 4]).int(), torch.tensor([total - 48]).int()
    pages = torch.arange(4).int().cuda()
    args = (host[0].cuda(), host[1].cuda(), pages, host[2].cuda(), *host)
    caches = [torch.zeros(4, page, hkv, d, dtype=BF16, device="cuda") for _ in range(2)]
    q2 = torch.empty_like(q)
    bia.bia_append_paged_kv_rope(desc, rope, table.cuda(), q, k, v, *caches, *args, q2, None, qw, kw)
    bits = lambda t: t.contiguous().view(torch.int16)
    assert torch.equal(bits(q2), bits(qo)) and torch.equal(bits(caches[0].flatten(0, 1)[:total]), bits(ko))
    codes = [torch.zeros(4, page, hkv, d, dtype=U8, device="cuda").view(bia.E4M3) for _ in range(2)]
    scale = [torch.zeros(4, page, hkv, dtype=U8, device="cuda").view(bia.E8M0) for _ in range(2)]
    k2 = torch.empty_like(k)
    bia.bia_append_paged_kv_fp8_rope(desc, rope, table.cuda(), q, k, v, *codes, *scale, *args, q2, k2, None, qw, kw)
    assert torch.equal(bits(q2), bits(qo)) and torch.equal(bits(k2), bits(ko))
    y, slack = reference(k, kw, rope, table, at)
    ok = (k.cpu() != 0).any(-1) if eps == 0 else torch.ones(total, hkv, dtype=torch.bool)
    ru.check_bf16(ko.cpu()[ok], y[ok], slack[ok])
    rows, byte = codes[0].view(U8).flatten(0, 1)[:total].cpu()[ok], scale[0].view(U8).flatten(0, 1)[:total].cpu()[ok]
    ru.check_codes(rows.view(bia.E4M3), byte, y[ok], slack[ok])


def test_zero_heads():
    """0 / sqrt(0 + eps): zero, and without an epsilon no number, in that head alone."""
    desc = bia.make_desc(4, 2, 128, 16)
    gen = torch.Generator().manual_seed(1)
    q, k = ru.rows((9, 4, 128), gen), ru.rows((9, 2, 128), gen)
    q[3, 1] = 0
    w = [x.cuda() for x in ru.weights(128, gen)]
    at = torch.arange(9).int()[None]
    table = ru.table_of(20, 128)
    for eps in (1e-45, 0.0):
        rope = bia.make_rope(128, 20, norm_eps=eps)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        bia.bia_norm_rope(desc, rope, table.cuda(), at.cuda(), q, k, qo, ko, *w)
        zero = torch.zeros(9, 4, dtype=torch.bool)
        zero[3, 1] = True
        assert bool((qo[3, 1] == 0).all() if eps else qo[3, 1].isnan().all())
        y, slack = ru.reference(q, w[0], rope, None, table, at)
        ru.check_bf16(qo.cpu()[~zero], y[~zero], slack[~zero])
        ru.check_bf16(ko, *ru.reference(k, w[1], rope, None, table, at))
