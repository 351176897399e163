"""Attention with a window and sinks from the definition, in 64 bits, the bounds
its kernels are held to, and requests on scattered pages."""
import math

import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu

F64, I32, BF16 = torch.float64, torch.int32, torch.bfloat16


def seen_of(lq, lk, window, sinks, device="cpu"):
    """bool [lq, lk]: which keys the last lq tokens of a sequence of lk keys see."""
    p = torch.arange(lk - lq, lk, device=device)[:, None]
    j = torch.arange(lk, device=device)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def bounds(q, k, v, seen, sm_scale=None):
    """(out, out_tol, lse, lse_tol) of one request, q [Lq, Hq, D] over k, v [Lk, Hkv, D] where `seen`.
    The bounds are those of fp8_util.attention_bounds (which derives them): half a bf16 step of the
    output and of each weight, fp32 scores and sums."""
    lq, hq, d = q.shape
    hkv = k.shape[1]
    scale = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    out, tol = torch.empty(lq, hq, d, dtype=F64, device=q.device), torch.empty(lq, hq, d, dtype=F64, device=q.device)
    lse, lse_tol = torch.empty(lq, hq, dtype=F64, device=q.device), torch.empty(lq, hq, dtype=F64, device=q.device)
    used = seen.any(0).nonzero()[:, 0]  # a key that no row sees may hold anything
    k, v, seen = k[used].double(), v[used].double(), seen[:, used]
    u = 2.0 ** -8
    for h in range(hq):
        g = h // (hq // hkv)
        x = (q[:, h].double() @ k[:, g].T) * scale
        big = (q[:, h].double().abs() @ k[:, g].abs().T) * scale
        x = x.masked_fill(~seen, -math.inf)
        b = big.masked_fill(~seen, 0.0).amax(-1)
        lse[:, h] = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, h, None])
        out[:, h] = p @ v[:, g]
        ds = d * 2.0 ** -23 * b + 2.0 ** -20 * (b + 1)
        tol[:, h] = u * out[:, h].abs() + (u + 2.0 ** -14 + 2 * ds[:, None]) * 1.01 * (p @ v[:, g].abs())
        lse_tol[:, h] = ds + 2.0 ** -18 * (1 + lse[:, h].abs())
    return out, tol, lse, lse_tol


class Batch:
    """Requests of keys[b] keys whose last new[b] tokens are queried, on scattered pages; slots and page
    entries that no query of the call sees hold NaN and page ids that do not exist."""

    def __init__(self, keys, new, hq, hkv, d, page, window, sinks, seed=0, spread=1.0, spoil=True):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.keys, self.new, self.window, self.sinks = keys, new, window, sinks
        self.desc = bia.make_desc(hq, hkv, d, page)
        self.kvp, self.pages, self.last, ids, self.n_pages = fu.page_table(keys, page, seed)
        self.qo = fu.indptr_of(new)
        self.q = (spread * fu.rows((sum(new), hq, d), gen)).bfloat16()
        self.rows_k = [fu.rows((n, hkv, d), gen) for n in keys]
        self.rows_v = [fu.rows((n, hkv, d), gen) for n in keys]
        caches = [torch.full((self.n_pages * page, hkv, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2)]
        self.pages = self.pages.clone()
        for b, (n, m) in enumerate(zip(keys, new)):
            if n == 0:
                continue
            pos = torch.arange(n)
            slots = (ids[b].long()[pos // page] * page + pos % page)
            used = seen_of(m, n, window, sinks).any(0) if spoil else torch.ones(n, dtype=torch.bool)
            for c, r in zip(caches, (self.rows_k[b], self.rows_v[b])):
                c[slots[used].cuda()] = r[used.cuda()]
            read = torch.zeros(len(ids[b]), dtype=torch.bool)
            read[pos[used] // page] = True
            if spoil:
                at = self.pages[int(self.kvp[b]):int(self.kvp[b + 1])]
                at[~read] = torch.tensor([2**31 - 1, -1, self.n_pages, -2**31], dtype=I32)[torch.arange(len(at)) % 4][~read]
        self.k_cache, self.v_cache = (c.view(self.n_pages, page, hkv, d) for c in caches)
        self.dev = tuple(x.cuda() for x in (self.kvp, self.pages, self.last))
        self.out = torch.full_like(self.q, float("nan"))
        self.lse = torch.full(self.q.shape[:2], float("nan"), device="cuda")

    def decode(self, split=0, ws=None, out=None, lse=True, **kw):
        need = bia.bia_decode_window_workspace_size(self.desc, self.window, self.sinks, self.kvp, self.last, split)
        assert need > 0
        ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda") if ws is None else ws
        if kw.get("stream"):  # the workspace is filled on the current one
            kw["stream"].wait_stream(torch.cuda.current_stream())
        bia.bia_decode_paged_window(self.desc, self.window, self.sinks, self.q, self.k_cache, self.v_cache, *self.dev,
                                    self.kvp, self.last, ws, self.out if out is None else out,
                                    self.lse if lse is True else lse, split, **kw)
        return ws

    def check(self, requests=None, rows=None, sm_scale=None):
        """Every row (or `rows` of each request) within its bound."""
        for b in range(len(self.keys)) if requests is None else requests:
            a, n = int(self.qo[b]), self.new[b]
            if n == 0:
                continue
            t = torch.arange(n) if rows is None else torch.tensor(sorted({r % n for r in rows}))
            seen = seen_of(n, self.keys[b], self.window, self.sinks)[t].cuda()
            t = t.cuda() + a
            fu.check(self.out[t], self.lse[t], *bounds(self.q[t], self.rows_k[b], self.rows_v[b], seen, sm_scale))


def extend(self, split=0, ws=None, out=None, lse=True, **kw):
    need = bia.bia_prefill_window_workspace_size(self.desc, self.window, self.sinks, self.qo, self.kvp, self.last, split)
    assert need > 0
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda") if ws is None else ws
    if kw.get("stream"):
        kw["stream"].wait_stream(torch.cuda.current_stream())
    bia.bia_prefill_paged_window(self.desc, self.window, self.sinks, self.q, self.k_cache, self.v_cache, self.qo.cuda(),
                                 *self.dev, self.qo, self.kvp, self.last, ws, self.out if out is None else out,
                                 self.lse if lse is True else lse, split, **kw)
    return ws


Batch.extend = extend
