"""What the rotation and windowed calls of the binding refuse by shape and by range: the host code alone,
over a library that takes every call (so a call that is let through is seen)."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia


class Taken(Exception):
    """The call reached the library."""


class Library:
    def __getattr__(self, name):
        def call(*args):
            raise Taken(name)
        return call


@pytest.fixture(autouse=True)
def host_alone(monkeypatch):
    monkeypatch.setattr(bia, "load", Library)
    monkeypatch.setattr(bia, "_check_cuda", lambda tensors, stream: None)
    monkeypatch.setattr(bia, "_handle", lambda stream: None)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


N, ROT = 6, 64
DESC = bia.make_desc(4, 2, 64, 16)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def rotate(rope, at):
    bia.bia_norm_rope(DESC, rope, torch.zeros(10, ROT), at, bf16(N, 4, 64), bf16(N, 2, 64), bf16(N, 4, 64), bf16(N, 2, 64))


def append(rope, at):
    caches = bf16(1, 16, 2, 64), bf16(1, 16, 2, 64)
    host = i32(0, N), i32(0, 1), i32(8)
    bia.bia_append_paged_kv_rope(DESC, rope, torch.zeros(10, ROT), bf16(N, 4, 64), bf16(N, 2, 64), bf16(N, 2, 64), *caches,
                                 host[0], host[1], i32(0), host[2], *host, bf16(N, 4, 64), at)


def append_fp8(rope, at):
    codes, scale = torch.zeros(1, 16, 2, 64, dtype=torch.uint8), torch.zeros(1, 16, 2, dtype=torch.uint8)
    host = i32(0, N), i32(0, 1), i32(8)
    bia.bia_append_paged_kv_fp8_rope(DESC, rope, torch.zeros(10, ROT), bf16(N, 4, 64), bf16(N, 2, 64), bf16(N, 2, 64),
                                     codes.view(bia.E4M3), codes.view(bia.E4M3), scale.view(bia.E8M0), scale.view(bia.E8M0),
                                     host[0], host[1], i32(0), host[2], *host, bf16(N, 4, 64), positions=at)


@pytest.mark.parametrize("call", [rotate, append, append_fp8])
def test_positions_lie_an_axis_a_row(call):
    """[num_axes, total]; a transposed tensor has as many entries, each of another token's or axis'."""
    for axes in (2, 3, 4):
        rope = bia.make_rope(ROT, 10, axes, [f % axes for f in range(ROT // 2)])
        at = torch.zeros(axes, N, dtype=torch.int32)
        for bad in (at.T.contiguous(), at.view(1, axes * N), at.view(axes, N // 2, 2), at[:, :N - 1].contiguous()):
            with pytest.raises(ValueError, match="positions"):
                call(rope, bad)
        for good in (at, at.view(-1)):
            with pytest.raises(Taken):
                call(rope, good)
    rope = bia.make_rope(ROT, 10)
    at = torch.zeros(1, N, dtype=torch.int32)
    for good in (at, at.view(-1), at.view(N, 1)):  # one axis: the same entries in the same order
        with pytest.raises(Taken):
            call(rope, good)
    with pytest.raises(ValueError, match="positions"):
        call(rope, torch.zeros(2, N, dtype=torch.int32))


WIDE = [2**31, 2**32, 2**32 + 5, 2**32 + 128, 2**63 - 1, 2**80, -2**31 - 1, -2**32 + 128]


def windowed(window=100, sinks=4, split=0):
    """Each windowed call, of one request of 24 keys."""
    q, c, ws = bf16(1, 4, 64), bf16(2, 16, 2, 64), torch.zeros(4096, dtype=torch.uint8)
    qo, kvp, pages, last = i32(0, 1), i32(0, 2), i32(0, 1), i32(8)
    b = bia.make_bounds(max_kv_len=64)
    tail = (ws, torch.zeros_like(q), None, split)
    return {
        "decode": lambda: bia.bia_decode_paged_window(DESC, window, sinks, q, c, c, kvp, pages, last, kvp, last, *tail),
        "bounded": lambda: bia.bia_decode_paged_window_bounded(DESC, b, window, sinks, q, c, c, kvp, pages, last, *tail),
        "extend": lambda: bia.bia_prefill_paged_window(DESC, window, sinks, q, c, c, qo, kvp, pages, last, qo, kvp, last, *tail),
        "decode size": lambda: bia.bia_decode_window_workspace_size(DESC, window, sinks, kvp, last, split),
        "bounded size": lambda: bia.bia_decode_window_bounded_workspace_size(DESC, b, window, sinks, 1, split),
        "extend size": lambda: bia.bia_prefill_window_workspace_size(DESC, window, sinks, qo, kvp, last, split),
    }


@pytest.mark.parametrize("name", list(windowed()))
def test_window_sinks_and_split_of_32_bits(name):
    """A number past 32 bits is refused, not cut to its low bits (2^32 sinks would be none)."""
    for wide in WIDE:
        for what in ("window", "sinks", "split"):
            with pytest.raises(ValueError, match=what):
                windowed(**{what: wide})[name]()
    for good in (dict(), dict(window=2**31 - 1), dict(sinks=2**31 - 1), dict(split=128), dict(window=-2**31)):
        with pytest.raises(Taken):  # the library refuses what it does not take
            windowed(**good)[name]()


def test_rotation_of_32_bits():
    for wide in WIDE:
        for args in ((wide, 10), (64, wide), (64, 10, wide, [0] * 32)):
            with pytest.raises(ValueError):
                bia.make_rope(*args)
    assert bia.make_rope(64, 2**31 - 1).num_positions == 2**31 - 1
