"""Plain 64-bit forms of the 8-bit cache and of packed attention, and the
bounds their kernels are held to.  Written from the definitions in
include/bia.h; no code of the library."""
from __future__ import annotations

import math

import torch

E4M3, E8M0, U8, F64, I32 = (torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8, torch.float64,
                            torch.int32)


def row_exponent(x: torch.Tensor) -> torch.Tensor:
    """Smallest integer e >= -120 with amax(finite |x|) <= 448 * 2^e, per row."""
    big = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1).double()
    m, ex = torch.frexp(big)  # big = m * 2^ex
    e = torch.where(m <= 0.875, ex - 9, ex - 8)  # 448 = 0.875 * 2^9
    return torch.where(big > 0, e, -120).clamp(min=-120)


def round_e4m3(y: torch.Tensor) -> torch.Tensor:
    """fp64 values |y| <= 448 to the nearest e4m3 value (ties to even)."""
    _, ex = torch.frexp(y)
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def quantise(x: torch.Tensor):
    """(code values fp64, exponents) of bf16 rows; non-finite elements NaN."""
    e = row_exponent(x)
    y = x.double() * torch.exp2(-e.double())[..., None]
    codes = torch.where(torch.isfinite(y), round_e4m3(torch.where(torch.isfinite(y), y, 0.0)),
                        float("nan"))
    return codes, e


def cache_values(codes, scale):
    """fp64 values of a cache (or of rows of it)."""
    return codes.double() * torch.exp2(scale.view(U8).double() - 127)[..., None]


def make_cache(rows_k, rows_v, pages, page_size, n_pages, device="cuda", fill=0x7F):
    """An 8-bit cache holding the given per-request bf16 rows [len, Hkv, D] at
    the page ids `pages[b]`; every other slot holds `fill` (a NaN code).
    Quantised by the plain form."""
    hkv, d = rows_k[0].shape[1:]
    out = []
    for rows in (rows_k, rows_v):
        codes = torch.full((n_pages * page_size, hkv, d), fill, dtype=U8, device=device)
        scale = torch.full((n_pages * page_size, hkv), 255, dtype=U8, device=device)
        for r, ids in zip(rows, pages):
            if r.shape[0] == 0:
                continue
            p = torch.arange(r.shape[0], device=device)
            slots = ids.to(device).long()[p // page_size] * page_size + p % page_size
            c, e = quantise(r)
            codes[slots] = c.float().to(E4M3).view(U8)
            scale[slots] = (e + 127).to(U8)
        out += [codes.view(n_pages, page_size, hkv, d).view(E4M3),
                scale.view(n_pages, page_size, hkv).view(E8M0)]
    return out[0], out[2], out[1], out[3]  # k, v, k_scale, v_scale


def attention_bounds(q, k, v, first=None, sm_scale=None, floor=0.0):
    """One request in 64 bits: q [Lq, Hq, D], k, v [Lk, Hkv, D]; row t sees the
    first `first + t` keys (None: all).  Returns (out, out_tol, lse, lse_tol).

    Where the bounds come from, with u = 2^-8 the half step of bf16:
    - out is rounded once: u * |out|
    - the softmax weights are rounded to 8 significant bits: each is off by at
      most u relative, so an output is off by u * A, A = sum p |v|
    - scores: sums of D products in fp32 are off by at most ds = D * 2^-23 *
      B, B = scale * sum |q k| (the largest over the keys), plus 2^-20 * (B +
      1) for the roundings of scale, log2 e and the exponent: weights are
      then off by 2 * ds relative (numerator and sum), lse by ds
    - sums over keys, rescaling and the merge in fp32: 2^-14 * A (2^10 keys'
      steps of 2^-24)
    - floor: weights below the grid of the 8-bit terms are off by at most
      `floor` of the largest weight (absolute), times sum |v| over the keys
    """
    lq, hq, d = q.shape
    lk, hkv = k.shape[:2]
    scale = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    kh = k.double().repeat_interleave(hq // hkv, 1)
    vh = v.double().repeat_interleave(hq // hkv, 1)
    x = torch.einsum("qhd,khd->hqk", q.double(), kh) * scale
    big = torch.einsum("qhd,khd->hqk", q.double().abs(), kh.abs()) * scale
    if first is not None:
        t = torch.arange(lq, device=q.device)[:, None]
        hide = torch.arange(lk, device=q.device)[None] >= first + t
        x = x.masked_fill(hide, -math.inf)
        big = big.masked_fill(hide, 0.0)
    if lk == 0:
        z = torch.zeros(lq, hq, d, dtype=F64, device=q.device)
        return z, z, torch.full((lq, hq), -math.inf, dtype=F64, device=q.device), z[..., 0]
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    p = torch.where(torch.isnan(p), 0.0, p)  # a row without keys
    out = torch.einsum("hqk,khd->qhd", p, vh)
    area = torch.einsum("hqk,khd->qhd", p, vh.abs())
    b = big.amax(-1)
    ds = d * 2.0 ** -23 * b + 2.0 ** -20 * (b + 1)
    u = 2.0 ** -8
    tol = u * out.abs() + (u + 2.0 ** -14 + 2 * ds.T[..., None]) * 1.01 * area
    if floor:
        tol = tol + floor * p.amax(-1).T[..., None] * vh.abs().sum(0)[None]
    return out, tol, lse.T, ds.T + 2.0 ** -18 * (1 + lse.T.abs().nan_to_num(0.0, 0.0, 0.0))


def check(got, lse, want, tol, want_lse, tol_lse):
    """Every element within its bound; -inf where the row sees nothing."""
    got = got.double()
    assert torch.isfinite(got).all()
    over = ((got - want).abs() - tol).max().item()
    assert over <= 0, f"out is {over:.3g} over its bound"
    dead = want_lse == -math.inf
    assert torch.equal(dead, lse == -math.inf)
    d = torch.where(dead, 0.0, (lse.double() - want_lse).abs() - tol_lse)
    assert d.max().item() <= 0, f"lse is {d.max().item():.3g} over its bound"


def rows(shape, gen, device="cuda"):
    """bf16 rows with a magnitude of their own for each row."""
    x = torch.randn(shape, generator=gen, device=device)
    return (x * torch.exp(torch.randn(shape[:-1] + (1,), generator=gen, device=device))).bfloat16()


def page_table(lens, page_size, seed=0, spare=3):
    """(kv_indptr, kv_indices, last, pages per request, number of pages), CPU,
    on scattered pages."""
    g = torch.Generator().manual_seed(seed)
    count = [-(-n // page_size) for n in lens]
    total = sum(count) + spare
    ids = torch.randperm(total, generator=g).to(I32)
    indptr = torch.tensor([0] + count).cumsum(0).to(I32)
    pages = [ids[indptr[b]:indptr[b + 1]] for b in range(len(lens))]
    last = torch.tensor([n - (c - 1) * page_size if c else 0 for n, c in zip(lens, count)],
                        dtype=I32)
    return indptr, torch.cat(pages) if pages else ids[:0], last, pages, total


def indptr_of(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(I32)
