"""Decode over the 8-bit cache where the value rows' magnitudes lie far apart,
and every other decode at bounds that only the attended values widen."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_bounds as fb
from tests import fp8_util as fu
from tests.gpu_util import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Requests:
    """Requests of their own codes and scales on scattered pages."""

    def __init__(self, lens, hq, hkv, d, page=16, seed=0, size=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.page, self.hq = lens, page, hq
        self.desc = bia.make_desc(hq, hkv, d, page)
        self.indptr, self.idx, self.last, self.pages, total = fu.page_table(lens, page, seed)
        self.q = fu.rows((len(lens), hq, d), g)
        self.codes = [torch.full((total * page, hkv, d), 0x7F, dtype=fu.U8, device=DEV) for _ in "kv"]
        self.scale = [torch.full((total * page, hkv), 255, dtype=fu.U8, device=DEV) for _ in "kv"]
        self.shape = (total, page, hkv)
        for b, n in enumerate(lens):
            for i in range(2):
                rows = fu.rows((n, hkv, d), g)
                if i == 1 and size is not None:
                    rows = (rows.double() * torch.exp2(size(b, n, hkv, g))).bfloat16()
                c, e = fu.quantise(rows)
                self.codes[i][self.slots(b)] = c.float().to(fu.E4M3).view(fu.U8)
                self.scale[i][self.slots(b)] = (e + 127).to(fu.U8)

    def slots(self, b):
        p = torch.arange(self.lens[b])
        return (self.pages[b].long()[p // self.page] * self.page + p % self.page).to(DEV)

    def plant(self, b, key, score, boost):
        """Key `key` of request b scores `score` with every head, and its value
        scale is 2^boost times what it was."""
        slot = self.slots(b)[key]
        d = self.q.shape[-1]
        self.q[b, :, 0] = 8.0
        self.codes[0][slot] = 0
        want = score * d ** 0.5 / 8.0  # = code * scale: a power of two and a code
        code = torch.tensor([want / 2.0 ** 4], dtype=torch.float64).float().to(fu.E4M3)
        self.codes[0][slot, :, 0] = code.view(fu.U8).to(DEV)
        self.scale[0][slot] = 127 + 4
        self.scale[1][slot] += boost

    def decode(self, split=0):
        total, page, hkv = self.shape
        d = self.q.shape[-1]
        caches = [c.view(total, page, hkv, d).view(fu.E4M3) for c in self.codes]
        scales = [s.view(total, page, hkv).view(fu.E8M0) for s in self.scale]
        ws = torch.empty(bia.bia_decode_fp8_workspace_size(self.desc, self.indptr, self.last, split),
                         dtype=torch.uint8, device=DEV)
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device=DEV)
        bia.bia_decode_paged_fp8(self.desc, self.q, *caches, *scales, self.indptr.to(DEV),
                                 self.idx.to(DEV), self.last.to(DEV), self.indptr, self.last, ws, out,
                                 lse, split_size=split)
        assert bia.bia_read_status(ws) == 0
        return out, lse

    def check(self, out, lse, which=None, split=1024):
        for b in range(len(self.lens)) if which is None else which:
            s = self.slots(b)
            (kc, vc), (ks, vs) = [c[s].view(fu.E4M3) for c in self.codes], \
                [e[s].view(fu.E8M0) for e in self.scale]
            fu.check(out[b:b + 1], lse[b:b + 1],
                     *fb.decode_bounds(self.q[b:b + 1], kc, ks, vc, vs, split))


SHAPES = [(64, 8, 8), (64, 16, 2), (96, 8, 2), (128, 4, 4), (128, 32, 8), (128, 16, 2), (256, 16, 8),
          (256, 8, 1), (128, 14, 7)]
LENS = [1, 2, 127, 129, 512, 513, 1024, 1025, 2049, 5000]


@pytest.mark.parametrize("d,hq,hkv", SHAPES)
@pytest.mark.parametrize("many", [False, True])
def test_ordinary_values(d, hq, hkv, many):
    # many: enough tiles that two kv heads share an item
    r = Requests(LENS + [700] * (100 if many else 0), hq, hkv, d, seed=d + hq)
    r.check(*r.decode(), range(len(LENS)))


@pytest.mark.parametrize("split", [128, 384, 640])
def test_ordinary_values_with_other_splits(split):
    r = Requests([1, 384, 385, 3001], 8, 2, 128, seed=split)
    r.check(*r.decode(split), split=split)


@pytest.mark.parametrize("d,hq,hkv", SHAPES)
@pytest.mark.parametrize("boost", [16, 20, 22, 60])
@pytest.mark.parametrize("many", [False, True])
def test_a_large_row_nobody_attends(d, hq, hkv, boost, many):
    # its score is 60 below 0: a weight of 2^-86 before the others' scores
    lens = [300, 1024, 2500] + [700] * (100 if many else 0)
    r = Requests(lens, hq, hkv, d, seed=d + hq)
    plain = r.decode()
    for b, key in enumerate((20, 700, 1024 + 100)):
        r.plant(b, key, -60.0, 0)
    without = r.decode()
    for b, key in enumerate((20, 700, 1024 + 100)):
        r.scale[1][r.slots(b)[key]] += boost
    out, lse = r.decode()
    r.check(out, lse, range(3))
    assert same_bits(lse, without[1])
    for b in range(3, min(len(lens), 6)):  # other requests never see it
        assert same_bits(out[b], plain[0][b])


@pytest.mark.parametrize("d,hq,hkv", SHAPES)
def test_magnitudes_over_eighty_binades(d, hq, hkv):
    size = lambda b, n, h, g: torch.rand((n, h, 1), generator=g, device=DEV, dtype=fu.F64) * 80 - 40
    r = Requests(LENS, hq, hkv, d, seed=d, size=size)
    r.check(*r.decode())


@pytest.mark.parametrize("score,boost", [(-10.0, 14), (-20.0, 30), (-40.0, 55), (20.0, -30)])
def test_a_large_row_that_counts_a_little(score, boost):
    # p * 2^boost about 1 for the first three; the last is attended and small
    r = Requests([512, 1000, 4000], 8, 2, 128, seed=3)
    for b in range(3):
        r.plant(b, 100 + 300 * b, score, boost)
    r.check(*r.decode())


@pytest.mark.parametrize("low,high", [(-100, 0), (0, 100), (-100, 100)])
def test_parts_of_different_magnitude(low, high):
    # alternate 512-key parts, so that a tile's parts and tiles join apart
    def size(b, n, h, g):
        part = (torch.arange(n, device=DEV) // 512) % 2 == 0
        return torch.where(part, float(low), float(high)).double()[:, None, None].expand(n, h, 1)
    r = Requests([513, 1024, 1537, 5000], 16, 4, 128, seed=5, size=size)
    r.check(*r.decode())


def test_one_magnitude_at_either_end_of_the_range():
    for e in (-112.0, 110.0):
        size = lambda b, n, h, g: torch.full((n, h, 1), e, dtype=fu.F64, device=DEV)
        r = Requests([1, 700, 3000], 8, 2, 128, seed=6, size=size)
        r.check(*r.decode())


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("up", [12, 16, 20, 24, 40])
def test_huge_scores(hq, hkv, up):
    # one key a part scores 2^up times the ordinary and takes all the weight:
    # the output is its value row, whatever the spacing of such scores is; the
    # largest value row of the part stands elsewhere
    lens = [300, 513, 1024, 2500]
    r = Requests(lens, hq, hkv, 128, seed=up)
    r.q[:, :, 0] = 8.0
    for b, n in enumerate(lens):
        s = r.slots(b)
        rows = list(range(77, n, 512))
        for i, key in enumerate(rows):
            r.codes[0][s[key]] = 0
            r.codes[0][s[key], :, 0] = 0x38 + i  # 1, 1.125, 1.25, ... in e4m3
            r.scale[0][s[key]] = 127 + up
            r.scale[1][s[key] if i % 2 else s[key - 1]] += 9
        out, lse = r.decode()
        v = fu.cache_values(r.codes[1].view(fu.E4M3), r.scale[1].view(fu.E8M0))
        want = v[s[rows[-1]]].repeat_interleave(hq // hkv, 0)
        # 8 significant bits of the weight, the output's rounding
        assert ((out[b].double() - want).abs() <= 2.02 * 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("byte", [0, 1, 3, 254])
def test_the_ends_of_the_scale_bytes(byte):
    # foreign caches: values down to 2^-136 (bf16 ends at 2^-133) and up to 2^127
    lens = [1, 600]
    r = Requests(lens, 4, 2, 64, seed=byte)
    for b in range(2):
        s = r.slots(b)
        r.scale[1][s] = byte
        if byte == 254:  # 1.75 and less, finite in bf16
            r.codes[1][s] &= 0xBF
    out, lse = r.decode()
    for b in range(2):
        s = r.slots(b)
        want, tol, l, l_tol = fb.decode_bounds(r.q[b:b + 1], r.codes[0][s].view(fu.E4M3),
                                               r.scale[0][s].view(fu.E8M0),
                                               r.codes[1][s].view(fu.E4M3),
                                               r.scale[1][s].view(fu.E8M0))
        # half a step of bf16's smallest values, and fp32's in between
        fu.check(out[b:b + 1], lse[b:b + 1], want, tol + 2.0 ** -134 + 2.0 ** -148, l, l_tol)


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 8), (128, 16, 2), (128, 32, 8), (256, 8, 2)])
@pytest.mark.parametrize("many", [False, True])
def test_non_finite_inputs_stay_with_their_heads(d, hq, hkv, many):
    lens = [700, 1500, 2500] + [600] * (100 if many else 0)
    r = Requests(lens, hq, hkv, d, seed=d + hkv)
    out, lse = r.decode()
    g = hq // hkv
    clean = torch.ones_like(out, dtype=torch.bool)
    # a query element of head 1 of request 0: that head alone
    r.q[0, 1, 5] = float("inf")
    clean[0, 1] = False
    # a NaN value scale, kv head 1 of request 1: its heads' outputs, not their lse
    r.scale[1][r.slots(1)[1200], 1] = 255
    clean[1, g:2 * g] = False
    # a NaN key scale, kv head 0 of request 2: its heads
    r.scale[0][r.slots(2)[40], 0] = 255
    clean[2, :g] = False
    o2, l2 = r.decode()
    assert torch.isnan(o2[~clean]).all()
    assert torch.equal(o2[clean], out[clean])
    dead = torch.zeros_like(lse, dtype=torch.bool)
    dead[0, 1] = True
    dead[2, :g] = True
    assert torch.isnan(l2[dead]).all() and torch.equal(l2[~dead], lse[~dead])


def test_more_requests_than_a_plan_s_chunk():
    lens = [(i * 131) % 300 + 1 for i in range(1300)]
    for b in (0, 511, 512, 1024, 1299):
        lens[b] = 1500 + b
    r = Requests(lens, 8, 2, 64, seed=9)
    out, lse = r.decode()
    r.check(out, lse, (0, 1, 510, 511, 512, 513, 1023, 1024, 1025, 1298, 1299))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
