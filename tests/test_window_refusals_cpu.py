"""What the windowed attention refuses, on the host: bad arguments come back
before anything is enqueued, so these run without a GPU (device addresses are
made up and never dereferenced)."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
FAKE = 1 << 20
BIG = 1 << 40
p = ctypes.c_void_p


@pytest.fixture(scope="module")
def bia():
    from invariant_paged_attention_gb300 import build
    build.build()
    import invariant_paged_attention_gb300 as m
    m.load()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def decode(bia, desc, kvp, last, *, window=64, sinks=4, split=0, q=FAKE, cache=FAKE, ws=FAKE, ws_bytes=BIG,
           pages=1 << 20, lse=0):
    kvp, last = i32(kvp), i32(last)
    return bia.load().bia_decode_paged_window(
        ctypes.byref(desc) if desc else None, window, sinks, p(q), p(cache), p(FAKE), pages, p(FAKE), p(FAKE),
        p(FAKE), p(kvp.data_ptr()), p(last.data_ptr()), len(kvp) - 1, split, p(ws), ws_bytes, p(FAKE), p(lse), None)


def bounded(bia, desc, kvp, last, *, window=64, sinks=4, split=0, q=FAKE, cache=FAKE, ws=FAKE, ws_bytes=BIG,
            pages=1 << 20, lse=0, most=4096):
    b = bia.make_bounds(max_kv_len=most)
    return bia.load().bia_decode_paged_window_bounded(
        ctypes.byref(desc) if desc else None, ctypes.byref(b), window, sinks, p(q), p(cache), p(FAKE), pages,
        p(FAKE), p(FAKE), p(FAKE), len(kvp) - 1, split, p(ws), ws_bytes, p(FAKE), p(lse), None)


@pytest.mark.parametrize("call", [decode, bounded])
def test_decode(bia, call):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d = bia.make_desc(32, 8, 128, 16)
    one = ([0, 4], [7])
    for bad in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(q=0), dict(cache=0), dict(ws=0),
                dict(q=FAKE + 8), dict(cache=FAKE + 8), dict(ws=FAKE + 128), dict(lse=FAKE + 2), dict(pages=0)):
        assert call(bia, d, *one, **bad) == inv, bad
    assert call(bia, None, *one) == inv
    assert call(bia, d, [0], []) == inv  # no request
    for split in (-128, 64, 200):
        assert call(bia, d, *one, split=split) == uns
    assert call(bia, bia.make_desc(32, 8, 80, 16), *one) == uns
    assert call(bia, bia.make_desc(24, 8, 128, 16), *one) == uns
    assert call(bia, bia.make_desc(32, 8, 128, 24), *one) == uns
    assert call(bia, d, *one, ws_bytes=511) == bia.BIA_ERR_WORKSPACE_TOO_SMALL  # 256 of status, 8 words of CTAs
    if call is decode:
        assert call(bia, d, [0, 0], [0]) == inv  # a request without a key
        assert call(bia, d, [0, 4], [17]) == inv
        assert call(bia, d, [0, 4], [0]) == inv
        assert call(bia, d, [3, 2], [1]) == inv
        assert call(bia, d, [0, 1 << 27], [1]) == uns
    else:
        assert call(bia, d, *one, most=0) == inv
        assert call(bia, d, *one, most=2**31 - 1) == uns


def test_workspace_follows_the_window(bia):
    """Not the lengths: a longer request needs no more once the window is full."""
    d = bia.make_desc(32, 8, 128, 16)
    size = lambda n, w, s: bia.bia_decode_window_workspace_size(d, w, s, i32([0, n]), i32([16]))
    assert size(100, 1024, 4) == size(1 << 20, 1024, 4) > 0
    assert size(2, 1024, 4) < size(100, 1024, 4)
    assert size(1 << 20, 2**31 - 1, 2**31 - 1) > size(1 << 20, 1024, 4)
    assert bia.bia_decode_window_workspace_size(d, 0, 4, i32([0, 4]), i32([16])) == 0
    b = bia.make_bounds(max_kv_len=1600)
    assert bia.bia_decode_window_bounded_workspace_size(d, b, 1024, 4, 1) == size(100, 1024, 4)
    assert bia.bia_decode_window_bounded_workspace_size(d, b, 1024, -1, 1) == 0


def test_binding(bia):
    d = bia.make_desc(4, 2, 64, 16)
    q, c = torch.zeros(1, 4, 64).bfloat16(), torch.zeros(3, 16, 2, 64).bfloat16()
    kvp, pages, last, ws = i32([0, 2]), i32([0, 1]), i32([5]), torch.zeros(4096, dtype=torch.uint8)
    call = lambda **k: bia.bia_decode_paged_window(
        d, 100, 4, k.get("q", q), k.get("k", c), c, k.get("kvp", kvp), k.get("pages", pages), last,
        k.get("kvp", kvp), last, ws, k.get("out", q.clone()), k.get("lse"))
    for bad in (dict(q=q.float()), dict(k=c.float()), dict(pages=pages.long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(), dict(k=c[:, :8].contiguous()), dict(out=q[:, :2].contiguous()), dict(lse=torch.zeros(3)),
                dict(kvp=i32([0, 3])), dict(kvp=i32([0, 1, 2])), dict(q=torch.zeros(1, 2, 64).bfloat16())):
        with pytest.raises(ValueError):  # the first: host tensors
            call(**bad)


def extend(bia, desc, qo, kvp, last, *, window=64, sinks=4, split=0, q=FAKE, cache=FAKE, ws=FAKE, ws_bytes=BIG,
           pages=1 << 20, lse=0, dev=FAKE):
    qo, kvp, last = i32(qo), i32(kvp), i32(last)
    return bia.load().bia_prefill_paged_window(
        ctypes.byref(desc) if desc else None, window, sinks, p(q), p(cache), p(FAKE), pages, p(dev), p(FAKE), p(FAKE),
        p(FAKE), p(qo.data_ptr()), p(kvp.data_ptr()), p(last.data_ptr()), len(qo) - 1, split, p(ws), ws_bytes, p(FAKE),
        p(lse), None)


def test_extend(bia):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d = bia.make_desc(32, 8, 128, 16)
    one = ([0, 20], [0, 4], [7])
    for bad in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(q=0), dict(cache=0), dict(ws=0), dict(dev=0),
                dict(q=FAKE + 8), dict(cache=FAKE + 8), dict(ws=FAKE + 128), dict(lse=FAKE + 2), dict(pages=0),
                dict(dev=FAKE + 2)):
        assert extend(bia, d, *one, **bad) == inv, bad
    assert extend(bia, None, *one) == inv
    assert extend(bia, d, [0], [0], []) == inv  # no request
    for split in (-128, 64, 200, (1 << 24) + 128):
        assert extend(bia, d, *one, split=split) == uns
    for desc in (bia.make_desc(32, 8, 80, 16), bia.make_desc(24, 8, 128, 16), bia.make_desc(32, 8, 128, 24)):
        assert extend(bia, desc, *one) == uns
    assert extend(bia, d, *one, pages=1 << 40) == uns
    assert extend(bia, d, *one, pages=(1 << 31) // 128) == uns  # rows past the tensor maps'
    assert extend(bia, d, *one, ws_bytes=511) == bia.BIA_ERR_WORKSPACE_TOO_SMALL
    assert extend(bia, d, [0, 60], [0, 4], [7]) == inv  # more tokens than keys
    assert extend(bia, d, [0, 5, 3], [0, 4, 8], [7, 7]) == inv
    assert extend(bia, d, [1, 5], [0, 4], [7]) == inv
    assert extend(bia, d, [0, 5], [0, 4], [17]) == inv
    assert extend(bia, d, [0, 5], [3, 2], [7]) == inv
    assert extend(bia, d, [0, 5], [0, 1 << 27], [1]) == uns
    long = ([0, 5], [0, 1 << 19], [16])  # 2^23 keys
    assert extend(bia, d, *long, sinks=bia.BIA_WINDOW_MAX_SINKS + 1) == uns
    assert extend(bia, d, *one, sinks=2**31 - 1, ws_bytes=511) == bia.BIA_ERR_WORKSPACE_TOO_SMALL
    assert extend(bia, d, [0, 0], [0, 0], [0]) == bia.BIA_OK  # no token


def splits_of(q_len, kv_len, tile, t, window, sinks, split, block):
    """Split tiles that hold a key block that a row of the q tile sees, from the definition."""
    first, last = kv_len - q_len + tile * t, kv_len - q_len + min(q_len, tile * t + t) - 1
    blocks = {j // block for j in range(last + 1)
              if any(j <= p and (j > p - window or j < sinks) for p in {first, last, min(max(j, first), last)})}
    seen = sorted(blocks)
    lo = max(0, first - window + 1) // block
    if any(b < lo and b not in range(-(-min(sinks, last + 1) // block)) for b in seen):
        raise AssertionError("a block between the sinks and the window")
    return seen


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 1), (64, 4, 4), (256, 8, 4)])
def test_states_hold_every_split(bia, d, hq, hkv):
    """The workspace of few q tiles has a state for each row and each split tile that a pair of q tiles touches."""
    block, nt, t = (64, 1, 128 * hkv // hq) if d == 256 else (128, 2, 128 * hkv // hq)
    desc = bia.make_desc(hq, hkv, d, 1)
    for n, keys in ((1, 700), (130, 900), (257, 257), (40, 1500)):
        for window in (1, 100, 300, 5000):
            for sinks in (0, 1, 130, 600):
                for split in (128, 256, 1024):
                    need = bia.bia_prefill_window_workspace_size(desc, window, sinks, i32([0, n]), i32([0, keys]), i32([1]), split)
                    parts = 1
                    for pair in range(-(-n // (nt * t))):
                        seen = [splits_of(n, keys, tile, t, window, sinks, split, block)
                                for tile in range(nt * pair, min(nt * pair + nt, -(-n // t)))]
                        ends = [b * block // split for s in seen for b in s]
                        whole = [s for s in seen if len(s) == s[-1] + 1]
                        low = 0 if whole else min((b * block // split for s in seen for b in s if b > -(-sinks // block) - 1),
                                                  default=0)
                        parts = max(parts, max(ends) - low + 1)
                    if parts > 1:
                        assert need >= n * parts * hq * (d + 1) * 4, (n, keys, window, sinks, split)
