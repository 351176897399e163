"""What is measured of the 8-bit paged cache and of the packed-prompt attention: the operators, the calls that
use them, and the same mathematics in elementary torch operations.

The operators:

- write    quantises the key and value rows of new tokens into their pages (e4m3 codes, one power-of-two scale
           for each key and kv head)
- read     reads rows back from the pages as bf16, packed one request after the other
- decode   attention of one new token of each request over its 8-bit pages
- prompt   attention of packed sequences over contiguous keys and values, causal from the bottom right

A case is a dict of plain values.  ``mix`` seeds the lengths, so that a case's work does not depend on the seed
of its values.  ``run`` computes the plain form, or with ``own`` calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
E4M3, E8M0, U8 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8


# ------------------------------------------------------------------ cases


def listed():
    qwen = dict(q_heads=32, kv_heads=8, head_dim=128)
    return [
        # one decode step of a small batch: each request appends one token (latency)
        dict(name="write step", op="write", batch=32, lo=200, hi=1500, new=1, page=16, fused=True, mix=1, **qwen),
        # a batch of whole prompts into the cache, one key per page
        dict(name="write prompts", op="write", batch=8, lo=512, hi=8192, new=0, page=1, fused=True, mix=2000, **qwen),
        # one request's cached prefix, for its next chunk
        dict(name="read prefix", op="read", batch=1, lo=4097, hi=4097, page=16, mix=3, **qwen),
        # the prefixes of a batch
        dict(name="read batch", op="read", batch=8, lo=512, hi=8192, page=1, mix=2000, **qwen),
        # a single request's next token (latency)
        dict(name="decode one", op="decode", batch=1, lo=4097, hi=4097, page=16, mix=5, **qwen),
        # a small batch, one key per page
        dict(name="decode few", op="decode", batch=8, lo=1024, hi=32768, page=1, mix=4000, **qwen),
        # a serving batch
        dict(name="decode many", op="decode", batch=64, lo=1024, hi=32768, page=16, mix=4000, **qwen),
        # a serving batch with wide heads
        dict(name="decode wide", op="decode", batch=32, lo=1024, hi=16384, page=1, mix=7500, q_heads=16, kv_heads=8,
             head_dim=256),
        # one short prompt (latency)
        dict(name="prompt short", op="prompt", batch=1, lo=256, hi=256, prefix=0, causal=True, fused=False, mix=9,
             q_heads=4, kv_heads=1, head_dim=64),
        # prompts of a chat batch, rows of one fused projection
        dict(name="prompt batch", op="prompt", batch=6, lo=100, hi=2048, prefix=0, causal=True, fused=True, mix=10, **qwen),
        # long prompts
        dict(name="prompt long", op="prompt", batch=3, lo=4096, hi=8192, prefix=0, causal=True, fused=False, mix=2002, **qwen),
        # a chunk of each request over a long prefix
        dict(name="prompt chunk", op="prompt", batch=4, lo=100, hi=600, prefix=16383, causal=True, fused=False, mix=12,
             q_heads=16, kv_heads=2, head_dim=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prompt", "prompt"])
    kv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 96, 128, 128, 128, 256])
    case = dict(op=op, q_heads=kv * g, kv_heads=kv, head_dim=d, mix=rng.randrange(1 << 30))
    if op == "prompt":
        n = _log(rng, 40, 6000)
        most = max(1, min(16, 6000 * 6000 // (n * n)))
        prefix = 0 if rng.random() < 0.6 else _log(rng, 1, 12000)
        while n * (n + prefix) * most * kv * g > 2 * 10**9:
            prefix //= 2
            most = max(1, most // 2)
            n = n if prefix or most > 1 else n * 3 // 4
        return dict(case, batch=rng.randint(1, most), lo=max(1, n // 8), hi=n, prefix=prefix, causal=rng.random() < 0.85,
                    fused=rng.random() < 0.5)
    case["page"] = rng.choice([1, 1, 8, 16, 16, 32, 64, 256])
    hi = _log(rng, 60, 32768)
    most = max(1, min(64, 1_000_000 * 128 // (hi * kv * d // 8)))
    batch = _log(rng, 1, most)
    lo = max(1, hi // 16)
    if op == "write":
        return dict(case, batch=batch, lo=lo, hi=min(hi, 16384), new=rng.choice([0, 1, 1, 5]), fused=rng.random() < 0.5)
    return dict(case, batch=batch, lo=lo, hi=hi)


def _lengths(case):
    """Key counts of the case's requests."""
    r = random.Random(case["mix"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def work(case):
    n, hkv, hq, d = _lengths(case), case["kv_heads"], case["q_heads"], case["head_dim"]
    if case["op"] == "write":  # bf16 rows in; codes and scales out
        new = sum(min(case["new"], x) if case["new"] else x for x in n)
        return {"bytes": new * hkv * 2 * (2 * d + d + 1), "flops": new * hkv * 2 * 3 * d}
    if case["op"] == "read":  # codes and scales in; bf16 rows out
        return {"bytes": sum(n) * hkv * 2 * (2 * d + d + 1), "flops": sum(n) * hkv * 2 * d}
    if case["op"] == "decode":
        return {"bytes": sum(n) * hkv * 2 * (d + 1) + len(n) * hq * (4 * d + 4), "flops": 4 * d * hq * sum(n)}
    p = case["prefix"]
    pairs = sum(x * p + x * (x + 1) // 2 if case["causal"] else x * (x + p) for x in n)
    rows, keys = sum(n), sum(n) + len(n) * p
    return {"bytes": 2 * d * (2 * rows * hq + 2 * keys * hkv) + 4 * rows * hq, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs


def _rows(shape, gen):
    """bf16 rows [..., D]: normal values, with a magnitude of its own for each row."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=BF16)
    size = torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    return x.mul_(size.to(BF16))


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
    n, hq, hkv, d = _lengths(case), case["q_heads"], case["kv_heads"], case["head_dim"]
    s = {"case": case, "n": n}
    if case["op"] == "prompt":
        keys = [x + case["prefix"] for x in n]
        for name, v in (("qo_indptr", n), ("kv_indptr", keys)):
            s[name + "_host"] = torch.tensor([0] + v).cumsum(0).to(I32)
            s[name] = s[name + "_host"].cuda()
        rows = _rows((sum(n), hq + 2 * hkv, d), gen)
        s["q"] = rows[:, :hq] if case["fused"] else rows[:, :hq].contiguous()
        if case["prefix"] == 0:
            s["k"], s["v"] = rows[:, hq:hq + hkv], rows[:, hq + hkv:]
            if not case["fused"]:
                s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        else:
            s["k"], s["v"] = _rows((sum(keys), hkv, d), gen), _rows((sum(keys), hkv, d), gen)
        return s
    s |= _table(n, case["page"], gen)
    for name in ("k", "v"):
        codes = torch.empty((s["pages"], case["page"], hkv, d), dtype=U8, device="cuda")
        scale = torch.empty((s["pages"], case["page"], hkv), dtype=U8, device="cuda")
        step = max(1, (1 << 27) // (case["page"] * hkv * d))
        for a in range(0, s["pages"], step):
            c, e = _plain_quantise(_rows(tuple(codes[a:a + step].shape), gen))
            codes[a:a + step], scale[a:a + step] = c.view(U8), e.view(U8)
        s[name + "_cache"], s[name + "_scale"] = codes.view(E4M3), scale.view(E8M0)
    if case["op"] == "decode":
        s["q"] = _rows((len(n), hq, d), gen)
        return s
    if case["op"] == "write":
        new = [min(case["new"], x) if case["new"] else x for x in n]
        rows = _rows((sum(new), hq + 2 * hkv if case["fused"] else 2 * hkv, d), gen)
        s["k_new"], s["v_new"] = rows[:, -2 * hkv:-hkv], rows[:, -hkv:]
        if not case["fused"]:
            s["k_new"], s["v_new"] = s["k_new"].contiguous(), s["v_new"].contiguous()
    else:
        new = n
    s["row_indptr_host"] = torch.tensor([0] + new).cumsum(0).to(I32)
    s["row_indptr"] = s["row_indptr_host"].cuda()
    return s


# ------------------------------------------------------------------ plain forms


def _slots(s, request, pos):
    """Flat cache slots of the positions `pos` of the requests `request` (integer tensors of one shape)."""
    page = s["case"]["page"]
    at = s["kv_indptr"].long()[request] + torch.div(pos, page, rounding_mode="floor")
    return s["kv_indices"].long()[at] * page + pos % page


def _values(cache, scale, slots):
    """fp32 values of the cache rows at `slots`."""
    hkv, d = cache.shape[2:]
    codes = cache.view(U8).view(-1, hkv, d)[slots].view(E4M3).float()
    return codes.mul_((scale.view(U8).view(-1, hkv)[slots].to(I32) << 23).view(F32)[..., None])


def _write(s):
    hkv, d = s["k_cache"].shape[2:]
    at = s["row_indptr"].long()
    rows = torch.arange(s["k_new"].shape[0], device="cuda")
    request = torch.searchsorted(at, rows, right=True) - 1
    keys = (s["kv_indptr"][1:] - s["kv_indptr"][:-1] - 1).long() * s["case"]["page"] + s["last"].long()
    pos = keys[request] - at[request + 1] + rows
    slots = _slots(s, request, pos)
    kc, ke = _plain_quantise(s["k_new"])
    vc, ve = _plain_quantise(s["v_new"])
    s["k_cache"].view(U8).view(-1, hkv, d)[slots] = kc.view(U8)
    s["v_cache"].view(U8).view(-1, hkv, d)[slots] = vc.view(U8)
    s["k_scale"].view(U8).view(-1, hkv)[slots] = ke.view(U8)
    s["v_scale"].view(U8).view(-1, hkv)[slots] = ve.view(U8)
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _read(s):
    at = s["row_indptr"].long()
    rows = torch.arange(sum(s["n"]), device="cuda")
    request = torch.searchsorted(at, rows, right=True) - 1
    slots = _slots(s, request, rows - at[request])
    return {"k": _values(s["k_cache"], s["k_scale"], slots).to(BF16),
            "v": _values(s["v_cache"], s["v_scale"], slots).to(BF16)}


def _attend(q, k, v, seen):
    """o and lse of q [B, Lq, Hq, D] over k, v [B, Lk, Hkv, D] (fp32) where `seen` [B, 1, 1, Lq, Lk]."""
    b, lq, hq, d = q.shape
    hkv = k.shape[2]
    q = (q * d ** -0.5).view(b, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, Lq, D]
    p = torch.matmul(q.reshape(b, hkv, -1, d), k.permute(0, 2, 3, 1)).view(b, hkv, hq // hkv, lq, -1)
    p = p.masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, -1, k.shape[1]), v.permute(0, 2, 1, 3)).view(b, hkv, hq // hkv, lq, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + l.log()).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d), lse.permute(0, 3, 1, 2).reshape(b, lq, hq)


def _decode(s):
    keys = (s["kv_indptr"][1:] - s["kv_indptr"][:-1] - 1).long() * s["case"]["page"] + s["last"].long()
    pos = torch.arange(max(s["n"]), device="cuda")[None]
    seen = pos < keys[:, None]
    request = torch.arange(len(s["n"]), device="cuda")[:, None].expand_as(seen)
    slots = _slots(s, request, torch.where(seen, pos, torch.zeros_like(pos)))
    k = _values(s["k_cache"], s["k_scale"], slots)
    v = _values(s["v_cache"], s["v_scale"], slots)
    o, lse = _attend(s["q"][:, None].float(), k, v, seen[:, None, None, None])
    return {"out": o[:, 0].to(BF16), "lse": lse[:, 0]}


def _prompt(s):
    qo, kv = s["qo_indptr"].long(), s["kv_indptr"].long()
    lq, lk = (qo[1:] - qo[:-1])[:, None], (kv[1:] - kv[:-1])[:, None]
    tq = torch.arange(max(s["n"]), device="cuda")[None]
    tk = torch.arange(max(s["n"]) + s["case"]["prefix"], device="cuda")[None]
    at_q = torch.where(tq < lq, qo[:-1, None] + tq, 0)
    at_k = torch.where(tk < lk, kv[:-1, None] + tk, 0)
    seen = (tk < lk)[:, None, :]
    if s["case"]["causal"]:
        seen = seen & (tk[:, None, :] <= (lk - lq + tq)[:, :, None])
    k = torch.where((tk < lk)[:, :, None, None], s["k"][at_k], 0).float()
    v = torch.where((tk < lk)[:, :, None, None], s["v"][at_k], 0).float()
    o, lse = _attend(s["q"][at_q].float(), k, v, seen[:, None, None])
    return {"out": o[tq < lq].to(BF16), "lse": lse[tq < lq]}


# ------------------------------------------------------------------ the library's calls


def _own(s):
    import invariant_paged_attention_gb300 as bia

    case = s["case"]
    if "desc" not in s:  # a server keeps its descriptor and its workspace
        s["desc"] = bia.make_desc(case["q_heads"], case["kv_heads"], case["head_dim"], case.get("page", 1))
        need = 0
        if case["op"] == "decode":
            need = bia.bia_decode_fp8_workspace_size(s["desc"], s["kv_indptr_host"], s["last_host"])
        elif case["op"] == "prompt":
            need = bia.bia_prefill_ragged_workspace_size(s["desc"], s["qo_indptr_host"], s["kv_indptr_host"],
                                                         causal=case["causal"])
        s["ws"] = torch.empty(need, dtype=U8, device="cuda")
    desc = s["desc"]
    if case["op"] == "write":
        bia.bia_append_paged_kv_fp8(desc, s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                    s["row_indptr"], s["kv_indptr"], s["kv_indices"], s["last"], s["row_indptr_host"],
                                    s["kv_indptr_host"], s["last_host"])
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if case["op"] == "read":
        hkv, d = s["k_cache"].shape[2:]
        k = torch.empty((sum(s["n"]), hkv, d), dtype=BF16, device="cuda")
        v = torch.empty_like(k)
        bia.bia_gather_paged_kv_fp8(desc, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], k, v, s["row_indptr"],
                                    s["kv_indptr"], s["kv_indices"], s["last"], s["row_indptr_host"],
                                    s["kv_indptr_host"], s["last_host"])
        return {"k": k, "v": v}
    out = torch.empty(s["q"].shape, dtype=BF16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=F32, device="cuda")
    if case["op"] == "decode":
        bia.bia_decode_paged_fp8(desc, s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["kv_indptr"],
                                 s["kv_indices"], s["last"], s["kv_indptr_host"], s["last_host"], s["ws"], out, lse)
    else:
        bia.bia_prefill_ragged(desc, s["q"], s["k"], s["v"], s["qo_indptr"], s["kv_indptr"], s["qo_indptr_host"],
                               s["kv_indptr_host"], s["ws"], out, lse, causal=case["causal"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"write": _write, "read": _read, "decode": _decode, "prompt": _prompt}[state["case"]["op"]](state)


# ------------------------------------------------------------------ from the definition, in 64 bits


def _exact_attention(q, k, v, first):
    """One request: q [Lq, Hq, D] over k, v [Lk, Hkv, D], all fp64; row t sees the first first + t keys at most."""
    lq, hq, d = q.shape
    lk, hkv, _ = k.shape
    out, lse = torch.empty_like(q), q.new_empty(lq, hq)
    for h in range(hq):
        kh, vh = k[:, h * hkv // hq], v[:, h * hkv // hq]
        for a in range(0, lq, 4096):
            x = (q[a:a + 4096, h] @ kh.T) / math.sqrt(d)
            if first is not None:
                t = torch.arange(a, a + x.shape[0], device=x.device)[:, None]
                x.masked_fill_(torch.arange(lk, device=x.device)[None] >= first + t, -math.inf)
            lse[a:a + 4096, h] = torch.logsumexp(x, 1)
            out[a:a + 4096, h] = torch.softmax(x, 1) @ vh
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    n, at = s["n"], 0
    if case["op"] == "prompt":
        outs, qa, ka = [], 0, 0
        for x in n:
            keys = x + case["prefix"]
            outs.append(_exact_attention(s["q"][qa:qa + x].double(), s["k"][ka:ka + keys].double(),
                                         s["v"][ka:ka + keys].double(), case["prefix"] + 1 if case["causal"] else None))
            qa, ka = qa + x, ka + keys
        return {"out": torch.cat([o for o, _ in outs]), "lse": torch.cat([e for _, e in outs])}
    page, indptr = case["page"], s["kv_indptr_host"].tolist()
    cache = {c: s[c + "_cache"].double().flatten(0, 1) if case["op"] == "write" else s[c + "_cache"].flatten(0, 1)
             for c in ("k", "v")}
    scale = {c: torch.exp2(s[c + "_scale"].view(U8).flatten(0, 1).double() - 127) for c in ("k", "v")}
    got = []
    for b, x in enumerate(n):
        p = torch.arange(x, device="cuda")
        slots = s["kv_indices"][indptr[b]:indptr[b + 1]].long()[p // page] * page + p % page
        if case["op"] == "write":
            new = min(case["new"], x) if case["new"] else x
            for c in ("k", "v"):
                y = s[c + "_new"][at:at + new].double()
                big = y.abs().amax(-1).clamp(min=2.0 ** -200)
                e = torch.ceil(torch.log2(big / 448.0) - 1e-12).clamp(-120, 120)
                e = torch.where(big > 448.0 * torch.exp2(e), e + 1, e)
                y = y / torch.exp2(e)[..., None]
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -40)) + 1e-12).clamp(min=-6) - 3)
                cache[c][slots[x - new:]] = torch.round(y / step) * step  # half to even
                scale[c][slots[x - new:]] = torch.exp2(e)
            at += new
        else:
            rows = {c: cache[c].view(U8)[slots].view(E4M3).double() * scale[c][slots][..., None] for c in ("k", "v")}
            got.append(rows if case["op"] == "read" else
                       _exact_attention(s["q"][b:b + 1].double(), rows["k"], rows["v"], None))
    if case["op"] == "write":
        shape = s["k_cache"].shape
        return {"k": cache["k"].view(shape), "v": cache["v"].view(shape), "k_scale": scale["k"].view(shape[:3]),
                "v_scale": scale["v"].view(shape[:3])}
    if case["op"] == "read":
        return {c: torch.cat([r[c] for r in got]) for c in ("k", "v")}
    return {"out": torch.cat([o for o, _ in got]), "lse": torch.cat([e for _, e in got])}
