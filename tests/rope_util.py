"""Norm and rotation from the definition, in 64 bits, and inputs for its tests."""
import torch

import invariant_paged_attention_gb300 as bia

EPS = 1e-5


def table_of(num_positions, rot, theta=1e4, device="cpu"):
    i = torch.arange(rot // 2, dtype=torch.float64)
    angle = torch.arange(num_positions, dtype=torch.float64)[:, None] * theta ** (-2 * i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def reference(x, weight, rope, freq_axis, table, positions):
    """x [total, heads, D] -> (y, slack): y in fp64, and per element |a| + |b| of its pair after the
    norm (|y| where nothing turns), which the fp32 arithmetic's error is relative to."""
    x = x.double().cpu()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + rope.norm_eps).sqrt() * weight.double().cpu()
    half = rope.rot_dim // 2
    y, slack = x.clone(), x.abs()
    table, positions = table.double().cpu(), positions.cpu().long().view(rope.num_axes, -1)
    for f in range(half):
        i, j = (2 * f, 2 * f + 1) if rope.interleaved else (f, f + half)
        p = positions[freq_axis[f] if rope.num_axes > 1 else 0]
        c, s = table[p, f][:, None], table[p, half + f][:, None]
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        slack[..., i] = slack[..., j] = a.abs() + b.abs()
    return y, slack


# fp32 from the loaded values on: the sum of D <= 256 squares (16 in a lane, 4 shuffle steps: at most
# 20 roundings, half of that behind the root), the mean's fma, rsqrt (2 ulp), two products and the two
# roundings of a turn: below 2^-19 relative to |a| + |b| of the pair.
NOISE = 2.0 ** -19


def check_bf16(got, y, slack):
    err = (got.double().cpu() - y).abs()
    tol = y.abs() * 2.0 ** -8 + slack * NOISE * (1 + 2.0 ** -8) + 2.0 ** -134
    assert bool((err <= tol).all()), float((err / tol).max())


def check_codes(codes, scale, y, slack):
    """codes e4m3 [.., D], scale bytes [..]: each value within half a step, each scale the smallest."""
    e = scale.view(torch.uint8).double().cpu() - 127
    step = torch.exp2(e)[..., None]
    err = (codes.double().cpu() * step - y).abs()
    tol = y.abs() * 2.0 ** -4 + step * 2.0 ** -10 + slack * NOISE * 1.1
    assert bool((err <= tol).all()), float((err / tol).max())
    big, near = y.abs().amax(-1), slack.amax(-1) * NOISE
    assert bool((big - near <= 448 * torch.exp2(e)).all())
    assert bool(((e == -120) | (big + near > 448 * torch.exp2(e - 1))).all())


def axes_of(axes, rot, how="turns"):
    half = rot // 2
    if how == "turns":
        return [i % axes for i in range(half)]
    return [min(axes - 1, i * axes // half) for i in range(half)]


def rows(shape, gen):
    x = torch.randn(shape, generator=gen) * torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen))
    return x.bfloat16().cuda()


def weights(d, gen, some=True):
    return tuple(torch.exp(0.3 * torch.randn(d, generator=gen)).cuda() if some else None for _ in range(2))


def page_table(n, page, gen, spare=3):
    """Scattered pages for requests of n[b] keys: host and device arrays, and the number of pages."""
    count = [-(-x // page) for x in n]
    indptr = torch.tensor([0] + count).cumsum(0).int()
    last = torch.tensor([x - (c - 1) * page if c else 0 for x, c in zip(n, count)]).int()
    pages = torch.randperm(int(indptr[-1]) + spare, generator=gen)[:int(indptr[-1])].int()
    return indptr, last, pages, int(indptr[-1]) + spare


def slots_of(keys, new, page, indptr, pages):
    """Flat cache slots of the last new[b] of keys[b] positions, all requests in turn."""
    out = []
    for b, (k, n) in enumerate(zip(keys, new)):
        p = torch.arange(k - n, k)
        out.append(pages[int(indptr[b]):int(indptr[b + 1])].long()[p // page] * page + p % page)
    return torch.cat(out) if out else torch.zeros(0).long()


def make(rot, num_positions, axes=1, interleaved=False, how="turns"):
    fa = axes_of(axes, rot, how)
    return bia.make_rope(rot, num_positions, axes, fa, interleaved, EPS), fa
