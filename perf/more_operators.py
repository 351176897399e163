"""What is measured of the rotary path into the paged caches and of the attention with a window and sinks: the
operators, the calls that use them, and the same mathematics in elementary torch operations.

The operators:

- rotate   norms each query and key head and rotates it by its token's position (one axis, or several), rows to rows
- append   the same on the way into the paged cache: queries to rows, keys and values to their pages, in bf16 or in
           8 bits (e4m3 codes, one power-of-two scale for each key and kv head)
- extend   causal attention of new tokens over a paged cache, each seeing the last ``window`` keys up to its own
           and the first ``sinks`` keys of its sequence
- decode   the same for one new token of each request

A case is a dict of plain values.  ``mix`` seeds the lengths, so that a case's work does not depend on the seed
of its values.  ``run`` computes the plain form, or with ``own`` calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3, E8M0, U8 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8
EPS = 1e-6  # of the norms


# ------------------------------------------------------------------ cases


def listed():
    qwen = dict(q_heads=32, kv_heads=8, head_dim=128)
    text = dict(rot=128, axes=1, interleaved=False, norm=True)
    return [
        # one decode step of a small batch, rows of the fused projection (latency)
        dict(name="rotate step", op="rotate", batch=32, lo=200, hi=1500, new=1, mix=1, **qwen, **text),
        # a batch of whole prompts, for the attention of packed prompts
        dict(name="rotate prompts", op="rotate", batch=6, lo=100, hi=8192, new=0, mix=10, **qwen, **text),
        # prompts with images: time, height and width in turn over the frequencies, half the columns rotate
        dict(name="rotate images", op="rotate", batch=5, lo=700, hi=3001, new=0, mix=3, q_heads=16, kv_heads=2, head_dim=128,
             rot=64, axes=3, interleaved=False, norm=False),
        # one decode step: each request's token into the bf16 cache (latency)
        dict(name="append step", op="append", cache="bf16", batch=64, lo=200, hi=1500, new=1, page=16, mix=4, **qwen, **text),
        # whole prompts into the bf16 cache, one key per page
        dict(name="append prompts", op="append", cache="bf16", batch=8, lo=512, hi=8192, new=0, page=1, mix=2000, **qwen, **text),
        # whole prompts into the 8-bit cache, keys kept as rows too for the prompts' own attention
        dict(name="append 8-bit", op="append", cache="8-bit", batch=8, lo=512, hi=8192, new=0, page=16, mix=2000, **qwen, **text),
        # a few draft tokens of each request to be verified (latency)
        dict(name="extend drafts", op="extend", batch=4, lo=4, hi=7, prefix=9001, window=1024, sinks=4, page=16, mix=7, **qwen),
        # a chunk of each request over a long prefix
        dict(name="extend chunk", op="extend", batch=6, lo=100, hi=600, prefix=16383, window=4096, sinks=64, page=16, mix=8,
             **qwen),
        # a batch of whole prompts, one key per page
        dict(name="extend prompts", op="extend", batch=8, lo=512, hi=8192, prefix=0, window=1024, sinks=4, page=1, mix=2000,
             **qwen),
        # the same with wide heads and a short window without sinks
        dict(name="extend wide", op="extend", batch=8, lo=512, hi=8192, prefix=0, window=1000, sinks=0, page=16, mix=2000,
             q_heads=16, kv_heads=8, head_dim=256),
        # a single request's next token (latency)
        dict(name="decode one", op="decode", batch=1, lo=4097, hi=4097, window=1024, sinks=4, page=16, mix=11, **qwen),
        # a serving batch
        dict(name="decode many", op="decode", batch=64, lo=1024, hi=32768, window=4096, sinks=64, page=16, mix=4000, **qwen),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "extend", "extend", "decode"])
    kv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 96, 128, 128, 128, 256])
    case = dict(op=op, q_heads=kv * g, kv_heads=kv, head_dim=d, mix=rng.randrange(1 << 30))
    if op in ("rotate", "append"):
        total = min(_log(rng, 1, 20000), 60_000_000 // ((kv * g + 2 * kv) * d))
        batch = _log(rng, 1, min(64, total))
        new = rng.choice([0, 0, 1, 5])
        hi = max(1, total // batch) if new == 0 else _log(rng, 5, 4000)
        case |= dict(batch=batch, lo=max(1, hi // 16), hi=hi, new=new, rot=rng.choice([d, d, d // 2 // 16 * 16]),
                     axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.6)
        if op == "append":
            case |= dict(cache=rng.choice(["bf16", "8-bit"]), page=rng.choice([1, 1, 8, 16, 16, 32, 64, 256]))
        return case
    case |= dict(window=_log(rng, 1, 8192), sinks=rng.choice([0, 0, 1, 4, 64, 200]), page=rng.choice([1, 1, 8, 16, 16, 32, 64, 256]))
    if op == "extend":
        n = _log(rng, 1, 4000)
        prefix = 0 if rng.random() < 0.4 else _log(rng, 1, 16000)
        batch = rng.randint(1, max(1, min(16, 8000 // n)))
        while batch * n * min(n + prefix, case["window"] + case["sinks"] + 256) * kv * g > 10**9:
            case["window"] = max(1, case["window"] // 2)
            n, batch = max(1, n * 3 // 4), max(1, batch * 3 // 4)
        return case | dict(batch=batch, lo=max(1, n // 8), hi=n, prefix=prefix)
    hi = _log(rng, 1, 32768)
    batch = _log(rng, 1, max(1, min(64, 1_000_000 * 128 // (hi * kv * d // 8))))
    return case | dict(batch=batch, lo=max(1, hi // 16), hi=hi)


def _lengths(case):
    """New tokens and keys of each of the case's requests."""
    r = random.Random(case["mix"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] == "extend":
        return n, [x + case["prefix"] for x in n]
    if case["op"] == "decode":
        return [1] * len(n), n
    return [min(case["new"], x) if case["new"] else x for x in n], n


def _seen(keys, new, window, sinks):
    """(query, key) pairs of a request's last `new` tokens, and the keys that any of them sees."""
    pairs = sum(min(p + 1, window) + min(max(p + 1 - window, 0), sinks) for p in range(keys - new, keys))
    first = max(0, keys - new - window + 1)
    return pairs, keys - first + min(first, sinks)


def work(case):
    new, keys = _lengths(case)
    hkv, hq, d, n = case["kv_heads"], case["q_heads"], case["head_dim"], sum(new)
    if case["op"] in ("rotate", "append"):
        turned = n * (hq + hkv) * d
        moved = 2 * 2 * turned + 4 * case["rot"] * min(n, max(keys)) + (4 * case["axes"] * n if case["axes"] > 1 or case["op"] == "rotate" else 0)
        if case["op"] == "append":
            moved += n * hkv * (4 * d if case["cache"] == "bf16" else 2 * d + 2 * (d + 1))
        return {"bytes": moved, "flops": turned * (7 if case["norm"] else 3)}
    both = [_seen(k, x, case["window"], case["sinks"]) for x, k in zip(new, keys)]
    return {"bytes": 4 * d * (n * hq + hkv * sum(b for _, b in both)) + 4 * n * hq, "flops": 4 * d * hq * sum(a for a, _ in both)}


# ------------------------------------------------------------------ inputs


def _rows(shape, gen):
    """bf16 rows [..., D]: normal values, with a magnitude of its own for each row."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=BF16)
    size = torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    return x.mul_(size.to(BF16))


def _table(n, page, gen):
    """A page table for requests of n[b] keys, on scattered pages, and the number of pages."""
    count = [-(-x // page) for x in n]
    indptr = torch.tensor([0] + count).cumsum(0).to(I32)
    last = torch.tensor([x - (c - 1) * page for x, c in zip(n, count)], dtype=I32)
    pages = torch.randperm(int(indptr[-1]), generator=gen, device="cuda").to(I32)
    return {"kv_indptr_host": indptr, "last_host": last, "kv_indptr": indptr.cuda(), "last": last.cuda(),
            "kv_indices": pages, "pages": int(indptr[-1])}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    (new, keys), hq, hkv, d = _lengths(case), case["q_heads"], case["kv_heads"], case["head_dim"]
    s = {"case": case, "new": new, "keys": keys}
    s["qo_indptr_host"] = torch.tensor([0] + new).cumsum(0).to(I32)
    s["qo_indptr"] = s["qo_indptr_host"].cuda()
    if case["op"] != "rotate":
        s |= _table(keys, case["page"], gen)
        shape = (s["pages"], case["page"], hkv, d)
    if case["op"] in ("extend", "decode"):
        s["k_cache"], s["v_cache"] = _rows(shape, gen), _rows(shape, gen)
        s["q"] = _rows((sum(new), hq, d), gen)
        return s
    # the rows of a fused projection
    rows = _rows((sum(new), hq + 2 * hkv, d), gen)
    s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    s["q_weight"], s["k_weight"] = ((torch.exp(0.3 * torch.randn(d, generator=gen, device="cuda")) for _ in range(2))
                                    if case["norm"] else (None, None))
    half = case["rot"] // 2
    angle = torch.arange(max(keys), device="cuda", dtype=F64)[:, None] * 1e6 ** (-torch.arange(half, device="cuda", dtype=F64) / half)
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(F32)
    s["freq_axis"] = [i % case["axes"] for i in range(half)]
    at = torch.cat([torch.arange(k - x, k) for x, k in zip(new, keys)]).to(I32).cuda()
    s["positions"] = at[None].contiguous()
    if case["axes"] > 1:  # tokens of an image stand at a time, a row and a column behind the text before it
        s["positions"] = torch.stack([at - at % 256, at - at % 256 + at % 256 // 16, at - at % 16]).contiguous()
    if case["op"] == "append":
        wide = case["cache"] == "bf16"
        for c in ("k", "v"):
            old = torch.randint(0, 120, shape, generator=gen, device="cuda", dtype=U8)  # what was there
            s[c + "_cache"] = old.to(BF16) if wide else old.view(E4M3)
            s[c + "_scale"] = None if wide else torch.full(shape[:3], 127, device="cuda", dtype=U8).view(E8M0)
    return s


# ------------------------------------------------------------------ plain forms


def _turn(s, x, weight):
    """Rows x[n, heads, D] in fp32, normed and rotated."""
    case, half = s["case"], s["case"]["rot"] // 2
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    f = torch.arange(half, device="cuda")
    at = s["positions"].long()[f % case["axes"]]  # [half, n]
    cos, sin = s["table"][at, f[:, None]].T[:, None], s["table"][at, half + f[:, None]].T[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_quantise(x):
    """e4m3 codes and e8m0 scale bytes of the rows x[..., D]: the scale is 2^e with the smallest e >= -120 for which
    the row's largest magnitude is at most 448 * 2^e."""
    x = x.float()
    big = x.abs().amax(-1)
    m, e = torch.frexp(big)  # big = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(big > 0, e, -120).clamp(-120, 120).to(I32)
    codes = (x * ((127 - e) << 23).view(F32)[..., None]).to(E4M3)
    return codes, (e + 127).to(U8).view(E8M0)


def _slots(s, request, pos):
    """Flat cache slots of the positions `pos` of the requests `request` (integer tensors of one shape)."""
    page = s["case"]["page"]
    at = s["kv_indptr"].long()[request] + torch.div(pos, page, rounding_mode="floor")
    return s["kv_indices"].long()[at] * page + pos % page


def _key_counts(s):
    return (s["kv_indptr"][1:] - s["kv_indptr"][:-1] - 1).long() * s["case"]["page"] + s["last"].long()


def _rotate(s):
    return {"q": _turn(s, s["q"], s["q_weight"]).to(BF16), "k": _turn(s, s["k"], s["k_weight"]).to(BF16)}


def _append(s):
    hkv, d = s["k_cache"].shape[2:]
    at = s["qo_indptr"].long()
    rows = torch.arange(s["k"].shape[0], device="cuda")
    request = torch.searchsorted(at, rows, right=True) - 1
    slots = _slots(s, request, _key_counts(s)[request] - at[request + 1] + rows)
    q, k = _turn(s, s["q"], s["q_weight"]).to(BF16), _turn(s, s["k"], s["k_weight"])
    if s["case"]["cache"] == "bf16":
        s["k_cache"].view(-1, hkv, d)[slots] = k.to(BF16)
        s["v_cache"].view(-1, hkv, d)[slots] = s["v"]
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    kc, ke = _plain_quantise(k)
    vc, ve = _plain_quantise(s["v"])
    s["k_cache"].view(U8).view(-1, hkv, d)[slots] = kc.view(U8)
    s["v_cache"].view(U8).view(-1, hkv, d)[slots] = vc.view(U8)
    s["k_scale"].view(U8).view(-1, hkv)[slots] = ke.view(U8)
    s["v_scale"].view(U8).view(-1, hkv)[slots] = ve.view(U8)
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "k_rows": k.to(BF16)}


def _attend(s):
    """Blocks of up to 256 queries of one request, each over the sinks and its own band of keys."""
    case, hq, (hkv, d) = s["case"], s["case"]["q_heads"], s["k_cache"].shape[2:]
    window, sinks, most, longest = case["window"], case["sinks"], min(256, max(s["new"])), max(s["keys"])
    qo, keys = s["qo_indptr"].long(), _key_counts(s)
    blocks = (qo[1:] - qo[:-1] + most - 1) // most
    request = torch.repeat_interleave(blocks)  # of each block
    start = (torch.arange(request.shape[0], device="cuda") - (blocks.cumsum(0) - blocks)[request]) * most
    t = start[:, None] + torch.arange(most, device="cuda")  # in-call token [block, query]
    real = t < (qo[1:] - qo[:-1])[request][:, None]
    at_q = torch.where(real, qo[request][:, None] + t, 0)
    first = keys[request] - (qo[1:] - qo[:-1])[request]  # position of the request's first new token
    p = first[:, None] + t
    # key positions of each block: the sinks, then the band
    lowest = (p[:, :1] - window + 1).clamp(min=0)
    band = lowest + torch.arange(min(window + most - 1, longest), device="cuda")
    pos = torch.cat([torch.arange(min(sinks, longest), device="cuda").expand(band.shape[0], -1), band], 1)
    sink = torch.arange(pos.shape[1], device="cuda") < min(sinks, longest)
    there = (pos < keys[request][:, None]) & (sink | (pos >= sinks))
    seen = there[:, None] & (pos[:, None] <= p[..., None]) & (sink | (pos[:, None] > p[..., None] - window))
    slots = _slots(s, request[:, None].expand_as(pos), torch.where(there, pos, 0))
    k = torch.where(there[..., None, None], s["k_cache"].view(-1, hkv, d)[slots], 0).float()
    v = torch.where(there[..., None, None], s["v_cache"].view(-1, hkv, d)[slots], 0).float()
    n, g = request.shape[0], hq // hkv
    q = (s["q"][at_q].float() * d ** -0.5).view(n, most, hkv, g, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(n, hkv, -1, d), k.permute(0, 2, 3, 1)).view(n, hkv, g, most, -1)
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, hkv, -1, pos.shape[1]), v.permute(0, 2, 1, 3)).view(n, hkv, g, most, d) / l
    lse = (m + l.log()).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)[real].to(BF16),
            "lse": lse.permute(0, 3, 1, 2).reshape(n, most, hq)[real]}


# ------------------------------------------------------------------ the library's calls


def _own(s):
    import invariant_paged_attention_gb300 as bia

    case = s["case"]
    if "desc" not in s:  # a server keeps its descriptors and its workspace
        s["desc"] = bia.make_desc(case["q_heads"], case["kv_heads"], case["head_dim"], case.get("page", 1))
        need = 0
        if case["op"] == "extend":
            need = bia.bia_prefill_window_workspace_size(s["desc"], case["window"], case["sinks"], s["qo_indptr_host"],
                                                         s["kv_indptr_host"], s["last_host"])
        elif case["op"] == "decode":
            need = bia.bia_decode_window_workspace_size(s["desc"], case["window"], case["sinks"], s["kv_indptr_host"],
                                                        s["last_host"])
        else:
            s["rope"] = bia.make_rope(case["rot"], s["table"].shape[0], case["axes"], s["freq_axis"], case["interleaved"], EPS)
        s["ws"] = torch.empty(need, dtype=U8, device="cuda")
    desc = s["desc"]
    if case["op"] == "rotate":
        q = torch.empty(s["q"].shape, dtype=BF16, device="cuda")
        k = torch.empty(s["k"].shape, dtype=BF16, device="cuda")
        bia.bia_norm_rope(desc, s["rope"], s["table"], s["positions"], s["q"], s["k"], q, k, s["q_weight"], s["k_weight"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        q = torch.empty(s["q"].shape, dtype=BF16, device="cuda")
        arrays = (s["qo_indptr"], s["kv_indptr"], s["kv_indices"], s["last"], s["qo_indptr_host"], s["kv_indptr_host"],
                  s["last_host"])
        positions = s["positions"] if case["axes"] > 1 else None  # text: a token's position is its key's
        if case["cache"] == "bf16":
            bia.bia_append_paged_kv_rope(desc, s["rope"], s["table"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                         *arrays, q, positions, s["q_weight"], s["k_weight"])
            return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
        k = torch.empty(s["k"].shape, dtype=BF16, device="cuda")
        bia.bia_append_paged_kv_fp8_rope(desc, s["rope"], s["table"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                         s["k_scale"], s["v_scale"], *arrays, q, k, positions, s["q_weight"], s["k_weight"])
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "k_rows": k}
    out = torch.empty(s["q"].shape, dtype=BF16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=F32, device="cuda")
    if case["op"] == "extend":
        bia.bia_prefill_paged_window(desc, case["window"], case["sinks"], s["q"], s["k_cache"], s["v_cache"], s["qo_indptr"],
                                     s["kv_indptr"], s["kv_indices"], s["last"], s["qo_indptr_host"], s["kv_indptr_host"],
                                     s["last_host"], s["ws"], out, lse)
    else:
        bia.bia_decode_paged_window(desc, case["window"], case["sinks"], s["q"], s["k_cache"], s["v_cache"], s["kv_indptr"],
                                    s["kv_indices"], s["last"], s["kv_indptr_host"], s["last_host"], s["ws"], out, lse)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _rotate, "append": _append, "extend": _attend, "decode": _attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------ from the definition, in 64 bits


def _exact_turn(s, x, weight):
    case, x = s["case"], x.double()
    half = case["rot"] // 2
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    out = x.clone()
    for f in range(half):  # each pair of columns as one complex number
        one, two = (2 * f, 2 * f + 1) if case["interleaved"] else (f, f + half)
        at = s["positions"][s["freq_axis"][f]].long()
        turn = torch.complex(s["table"][at, f].double(), s["table"][at, half + f].double())[:, None]
        z = torch.complex(x[..., one], x[..., two]) * turn
        out[..., one], out[..., two] = z.real, z.imag
    return out


def _exact_codes(y):
    """Codes (as the values they stand for) and scales of rows in 64 bits."""
    big = y.abs().amax(-1).clamp(min=2.0 ** -200)
    e = torch.ceil(torch.log2(big / 448.0) - 1e-12).clamp(-120, 120)
    e = torch.where(big > 448.0 * torch.exp2(e), e + 1, e)
    y = y / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -40)) + 1e-12).clamp(min=-6) - 3)
    return torch.round(y / step) * step, torch.exp2(e)  # half to even


def _exact_attention(q, k, v, window, sinks):
    """One request: q [Lq, Hq, D], the last of the keys' tokens, over k, v [Lk, Hkv, D], all fp64."""
    lq, hq, d = q.shape
    lk, hkv, _ = k.shape
    out, lse = torch.empty_like(q), q.new_empty(lq, hq)
    for a in range(0, lq, 1024):
        p = torch.arange(lk - lq + a, lk - lq + min(a + 1024, lq), device=q.device)[:, None]
        lo, hi = max(0, int(p[0]) - window + 1), int(p[-1]) + 1
        j = torch.arange(hi, device=q.device)
        j = torch.cat([j[:min(sinks, lo)], j[lo:]])
        hide = (j > p) | ((j <= p - window) & (j >= sinks))
        for h in range(hq):
            x = (q[a:a + 1024, h] @ k[j, h * hkv // hq].T) / math.sqrt(d)
            x.masked_fill_(hide, -math.inf)
            lse[a:a + 1024, h] = torch.logsumexp(x, 1)
            out[a:a + 1024, h] = torch.softmax(x, 1) @ v[j, h * hkv // hq]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    new, keys = s["new"], s["keys"]
    if case["op"] in ("rotate", "append"):
        q, k = _exact_turn(s, s["q"], s["q_weight"]), _exact_turn(s, s["k"], s["k_weight"])
        if case["op"] == "rotate":
            return {"q": q, "k": k}
    page, indptr, at = case["page"], s["kv_indptr_host"].tolist(), 0
    slots = []
    for b, x in enumerate(keys):
        p = torch.arange(x, device="cuda")
        slots.append(s["kv_indices"][indptr[b]:indptr[b + 1]].long()[p // page] * page + p % page)
    if case["op"] == "append":
        to = torch.cat([x[len(x) - n:] for x, n in zip(slots, new)])
        cache = {c: s[c + "_cache"].double() for c in ("k", "v")}
        rows = {"k": k, "v": s["v"].double()}
        if case["cache"] == "bf16":
            for c in ("k", "v"):
                cache[c].flatten(0, 1)[to] = rows[c]
            return {"q": q} | cache
        scale = {c + "_scale": torch.exp2(s[c + "_scale"].view(U8).double() - 127) for c in ("k", "v")}
        for c in ("k", "v"):
            cache[c].flatten(0, 1)[to], scale[c + "_scale"].flatten(0, 1)[to] = _exact_codes(rows[c])
        return {"q": q, "k_rows": k} | cache | scale
    got = []
    for x, n in zip(slots, new):
        got.append(_exact_attention(s["q"][at:at + n].double(), s["k_cache"].flatten(0, 1)[x].double(),
                                    s["v_cache"].flatten(0, 1)[x].double(), case["window"], case["sinks"]))
        at += n
    return {"out": torch.cat([o for o, _ in got]), "lse": torch.cat([e for _, e in got])}
