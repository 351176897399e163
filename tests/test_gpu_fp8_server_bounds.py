"""A server's calls over an 8-bit cache together, the decode at bounds that only
attended values widen: prompts appended, a chunk over the prefix read back,
then single tokens, with value rows of very different size."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_bounds as fb
from tests import fp8_util as fu
from tests.test_gpu_prefill_ragged import run

pytestmark = pytest.mark.gpu
DEV = "cuda"


def underflow(v, hq):
    """What the bounds leave out, as they are relative: a weight below 2^-126 of
    the row's largest is 0 in fp32 (at most 2^-126 |v| a key), and an output
    below half of bf16's smallest number, 2^-133, is 0."""
    return 2.0 ** -126 * v.abs().sum(0).repeat_interleave(hq // v.shape[1], 0) + 2.0 ** -134


def check(out, lse, want, tol, want_lse, tol_lse, v):
    fu.check(out, lse, want, tol + underflow(v, out.shape[1])[None], want_lse, tol_lse)


@pytest.mark.parametrize("d,hq,hkv,page", [(64, 8, 8, 16), (128, 32, 8, 1), (128, 16, 2, 64), (256, 8, 4, 16)])
@pytest.mark.parametrize("spread", [0, 24])
def test_prompts_chunks_and_tokens(d, hq, hkv, page, spread):
    first, total, steps = [300, 1, 1100], [900, 40, 1100], 2
    g = torch.Generator(device=DEV).manual_seed(d + page + spread)
    longest = [n + steps for n in total]
    indptr, idx, _, pages, n_pages = fu.page_table(longest, page, 3)
    proj = [fu.rows((n, hq + 2 * hkv, d), g) for n in longest]
    for p in proj:  # value rows: some 2^spread times the others
        up = torch.randint(0, 8, p.shape[:1], generator=g, device=DEV) == 0
        p[up, hq + hkv:] *= 2.0 ** spread
    desc = bia.make_desc(hq, hkv, d, page)
    codes = [torch.full((n_pages, page, hkv, d), 0x7F, dtype=torch.uint8, device=DEV).view(fu.E4M3)
             for _ in "kv"]
    scale = [torch.full((n_pages, page, hkv), 255, dtype=torch.uint8, device=DEV).view(fu.E8M0)
             for _ in "kv"]

    def put(lo, hi):
        count = [-(-n // page) for n in hi]
        ip, last = fu.indptr_of(count), torch.tensor([n - (c - 1) * page for n, c in zip(hi, count)],
                                                     dtype=torch.int32)
        table = ip.to(DEV), torch.cat([pages[b][:c] for b, c in enumerate(count)]).to(DEV), last.to(DEV)
        rows = torch.cat([p[a:e] for p, a, e in zip(proj, lo, hi)])
        ap = fu.indptr_of([e - a for a, e in zip(lo, hi)])
        bia.bia_append_paged_kv_fp8(desc, rows[:, hq:hq + hkv], rows[:, hq + hkv:], *codes, *scale,
                                    ap.to(DEV), *table, ap, ip, last)
        return rows[:, :hq], table, ip, last

    lo = [0, 0, 0]
    for hi in (first, total):
        q, table, ip, last = put(lo, hi)
        kv = fu.indptr_of(hi)
        k = torch.empty(sum(hi), hkv, d, dtype=torch.bfloat16, device=DEV)
        v = torch.empty_like(k)
        bia.bia_gather_paged_kv_fp8(desc, *codes, *scale, k, v, kv.to(DEV), *table, kv, ip, last)
        new = [e - a for a, e in zip(lo, hi)]
        out, lse = run(q, k, v, new, hi)
        at = 0
        for b, n in enumerate(new):
            if n:
                kb, vb = k[kv[b]:kv[b + 1]].double(), v[kv[b]:kv[b + 1]].double()
                check(out[at:at + n], lse[at:at + n],
                      *fu.attention_bounds(q[at:at + n], kb, vb, lo[b] + 1), vb)
            at += n
        lo = hi
    for _ in range(steps):
        hi = [n + 1 for n in lo]
        q, table, ip, last = put(lo, hi)
        q = q.contiguous()
        ws = torch.empty(bia.bia_decode_fp8_workspace_size(desc, ip, last), dtype=torch.uint8, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        bia.bia_decode_paged_fp8(desc, q, *codes, *scale, *table, ip, last, ws, out, lse)
        assert bia.bia_read_status(ws) == 0
        for b in range(3):
            kc, vc = [fu.quantise(proj[b][:hi[b], s]) for s in (slice(hq, hq + hkv), slice(hq + hkv, None))]
            args = [x for c, e in (kc, vc) for x in (c.float().to(fu.E4M3),
                                                     (e + 127).to(torch.uint8).view(fu.E8M0))]
            check(out[b:b + 1], lse[b:b + 1], *fb.decode_bounds(q[b:b + 1], *args),
                  fu.cache_values(*args[2:]))
        lo = hi
