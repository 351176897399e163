"""What the 8-bit cache's calls and the packed prefill refuse, on the host:
bad arguments come back before anything is enqueued, so these run without a
GPU (device addresses are made up and never dereferenced)."""
import ctypes
import shutil
import os

import pytest
import torch

from tests import fp8_util as fu

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
FAKE = 1 << 20
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


def ptr(t):
    return p(t.data_ptr())


def append(bia, desc, rows, kvp, last, *, k=FAKE, scale=FAKE, stride=0, pages=1 << 20, cache=FAKE,
           status=None):
    rows, kvp, last = i32(rows), i32(kvp), i32(last)
    return bia.load().bia_append_paged_kv_fp8(
        ctypes.byref(desc), p(k), p(FAKE), stride, 0, p(cache), p(FAKE), p(scale), p(FAKE), pages,
        p(FAKE), p(FAKE), p(FAKE), p(FAKE), ptr(rows), ptr(kvp), ptr(last), len(rows) - 1,
        status and p(status), None)


def gather(bia, desc, rows, kvp, last, *, out=FAKE, scale=FAKE, pages=1 << 20):
    rows, kvp, last = i32(rows), i32(kvp), i32(last)
    return bia.load().bia_gather_paged_kv_fp8(
        ctypes.byref(desc), p(FAKE), p(FAKE), p(scale), p(FAKE), pages, p(FAKE), p(FAKE), p(FAKE),
        p(FAKE), ptr(rows), ptr(kvp), ptr(last), len(rows) - 1, p(out), p(FAKE), None, None)


@pytest.mark.parametrize("call", [append, gather])
def test_append_and_gather_refuse(bia, call):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d = bia.make_desc(32, 8, 128, 16)
    assert call(bia, d, [0, 17], [0, 1], [16]) == inv  # more rows than keys
    assert call(bia, d, [0, 5, 3], [0, 1, 2], [16, 16]) == inv  # indptr falls
    assert call(bia, d, [1, 5], [0, 1], [16]) == inv
    assert call(bia, d, [0, 5], [0, 1], [17]) == inv  # past the page
    assert call(bia, d, [0, 5], [0, 1], [0]) == inv
    assert call(bia, d, [0, 5], [1, 0], [5]) == inv
    assert call(bia, d, [0, 5], [0, 1], [5], scale=0) == inv
    assert call(bia, d, [0, 5], [0, 1], [5], pages=0) == inv
    assert call(bia, bia.make_desc(32, 8, 80, 16), [0, 5], [0, 1], [5]) == uns
    assert call(bia, bia.make_desc(32, 8, 128, 3), [0, 5], [0, 1], [3]) == uns
    assert call(bia, bia.make_desc(8, 8, 128, 256), [0, 1 << 27], [0, 1 << 19], [256]) == uns
    assert call(bia, d, [0, 0], [0, 0], [0]) == bia.BIA_OK  # nothing to do


def test_append_refuses_rows_off_their_grid(bia):
    inv = bia.BIA_ERR_INVALID_ARG
    d = bia.make_desc(32, 8, 128, 16)
    assert append(bia, d, [0, 5], [0, 1], [5], k=FAKE + 8) == inv
    assert append(bia, d, [0, 5], [0, 1], [5], cache=FAKE + 8) == inv
    assert append(bia, d, [0, 5], [0, 1], [5], scale=FAKE + 1) == inv
    assert append(bia, d, [0, 5], [0, 1], [5], status=FAKE + 2) == inv
    assert gather(bia, d, [0, 5], [0, 1], [5], out=FAKE + 8) == inv


def decode(bia, desc, kvp, last, *, split=0, ws=FAKE, ws_bytes=1 << 40, scale=FAKE, q=FAKE):
    kvp, last = i32(kvp), i32(last)
    return bia.load().bia_decode_paged_fp8(
        ctypes.byref(desc), p(q), p(FAKE), p(FAKE), p(scale), p(FAKE), 1 << 20, p(FAKE), p(FAKE),
        p(FAKE), ptr(kvp), ptr(last), len(kvp) - 1, split, p(ws), ws_bytes, p(FAKE), None, None)


def test_decode_refuses(bia):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d = bia.make_desc(32, 8, 128, 16)
    assert decode(bia, d, [0, 0], [1]) == inv  # a request without a key
    assert decode(bia, d, [0, 2, 1], [1, 1]) == inv
    assert decode(bia, d, [0, 2], [17]) == inv
    assert decode(bia, d, [0, 2], [4], scale=0) == inv
    assert decode(bia, d, [0, 2], [4], scale=FAKE + 1) == inv
    assert decode(bia, d, [0, 2], [4], q=FAKE + 8) == inv
    assert decode(bia, d, [0, 2], [4], ws=FAKE + 16) == inv
    assert decode(bia, d, [0, 2], [4], split=100) == uns
    assert decode(bia, d, [0, 2], [4], split=bia.BIA_DECODE_FP8_SPLIT + 128) == uns
    assert decode(bia, bia.make_desc(48, 3, 128, 16), [0, 2], [4]) == uns
    assert decode(bia, d, [0, 2], [4], ws_bytes=256) == bia.BIA_ERR_WORKSPACE_TOO_SMALL
    assert bia.load().bia_decode_paged_fp8_bounded(
        ctypes.byref(d), None, *[p(FAKE)] * 5, 1 << 20, p(FAKE), p(FAKE), p(FAKE), 1, 0, p(FAKE),
        1 << 40, p(FAKE), None, None) == inv
    assert bia.bia_decode_fp8_workspace_size(d, i32([0, 2]), i32([4])) > 0
    assert bia.bia_decode_fp8_workspace_size(d, i32([0, 0]), i32([4])) == 0
    assert bia.bia_decode_fp8_bounded_workspace_size(d, bia.make_bounds(max_kv_len=0), 4) == 0
    exact = bia.bia_decode_fp8_workspace_size(d, i32([0, 400]), i32([16]))
    assert bia.bia_decode_fp8_bounded_workspace_size(d, bia.make_bounds(max_kv_len=6400), 1) >= exact


def prompt(bia, desc, qo, kv, *, causal=1, split=0, q_stride=0, k_stride=0, ws=FAKE,
           ws_bytes=1 << 40, k=FAKE, out=FAKE):
    qo, kv = i32(qo), i32(kv)
    return bia.load().bia_prefill_ragged(
        ctypes.byref(desc), p(FAKE), p(k), p(FAKE), q_stride, k_stride, 0, p(FAKE), p(FAKE), ptr(qo),
        ptr(kv), len(qo) - 1, causal, split, p(ws), ws_bytes, p(out), None, None)


def test_packed_prefill_refuses(bia):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d = bia.make_desc(32, 8, 128, 1)
    assert prompt(bia, d, [0, 10], [0, 9]) == inv  # q_len > kv_len, causal
    assert prompt(bia, d, [0, 10, 4], [0, 10, 20]) == inv
    assert prompt(bia, d, [0, 10], [3, 13]) == inv  # starts past 0
    assert prompt(bia, d, [1, 10], [0, 10]) == inv
    assert prompt(bia, d, [0, 10], [0, 10], k=0) == inv
    assert prompt(bia, d, [0, 10], [0, 10], k=FAKE + 8) == inv
    assert prompt(bia, d, [0, 10], [0, 10], out=FAKE + 8) == inv
    assert prompt(bia, d, [0, 10], [0, 10], q_stride=4092) == inv  # below a token's row
    assert prompt(bia, d, [0, 10], [0, 10], k_stride=1028) == inv  # off the 16-byte grid
    assert prompt(bia, d, [0, 10], [0, 10], split=64) == uns
    most = bia.BIA_RAGGED_MAX_SPLIT
    assert prompt(bia, d, [0, 10], [0, 10], split=most + 128) == uns
    assert prompt(bia, d, [0, 10], [0, 10], split=most, ws_bytes=64) == bia.BIA_ERR_WORKSPACE_TOO_SMALL
    header = os.path.join(os.path.dirname(__file__), "..", "include", "bia.h")
    assert f"#define BIA_RAGGED_MAX_SPLIT {most}\n" in open(header).read()
    assert prompt(bia, bia.make_desc(32, 8, 112, 1), [0, 10], [0, 10]) == uns
    assert prompt(bia, bia.make_desc(36, 12, 128, 1), [0, 10], [0, 10]) == uns
    assert prompt(bia, d, [0, 10], [0, 10], ws_bytes=64) == bia.BIA_ERR_WORKSPACE_TOO_SMALL
    assert prompt(bia, d, [0, 0], [0, 10]) == bia.BIA_OK  # nothing to do
    assert bia.bia_prefill_ragged_workspace_size(d, i32([0, 10]), i32([0, 9])) == 0
    assert bia.bia_prefill_ragged_workspace_size(d, i32([0, 10]), i32([0, 9]), causal=False) > 0


def test_the_binding_checks_its_tensors(bia):
    d = bia.make_desc(4, 2, 64, 4)
    codes = torch.zeros(3, 4, 2, 64, dtype=torch.uint8)
    kc, ks = codes.view(fu.E4M3), torch.zeros(3, 4, 2, dtype=torch.uint8).view(fu.E8M0)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    ip, kvp, idx, last = i32([0, 5]), i32([0, 2]), i32([0, 1]), i32([1])
    tail = (ip, kvp, idx, last, ip, kvp, last)

    def put(k=x, v=x, cache=kc, scale=ks, tail=tail):
        bia.bia_append_paged_kv_fp8(d, k, v, cache, kc, scale, ks, *tail)

    with pytest.raises(ValueError, match="CUDA"):
        put()  # host tensors pass every other check
    with pytest.raises(TypeError, match="k_cache"):
        put(cache=codes)
    with pytest.raises(TypeError, match="k_scale"):
        put(scale=ks.view(torch.uint8))
    with pytest.raises(ValueError, match="k_scale"):
        put(scale=ks[:2])
    with pytest.raises(TypeError, match="k_new"):
        put(k=x.float())
    with pytest.raises(ValueError, match="k_new"):
        put(k=torch.zeros(5, 2, 128, dtype=torch.bfloat16)[:, :, ::2])
    with pytest.raises(ValueError, match="k_new"):
        put(k=torch.zeros(5, 132, dtype=torch.bfloat16)[:, :128].unflatten(1, (2, 64)))
    with pytest.raises(ValueError, match="tokens"):
        put(v=x[:4])
    with pytest.raises(ValueError, match="kv_indices"):
        put(tail=(ip, kvp, idx[:1], last, ip, kvp, last))
    with pytest.raises(ValueError, match="kv_last_page_len"):
        put(tail=(ip, kvp, idx, i32([1, 1]), ip, kvp, last))
    with pytest.raises(ValueError, match="k_out"):
        bia.bia_gather_paged_kv_fp8(d, kc, kc, ks, ks, x[:4], x[:4], *tail)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="q and out must be"):
        bia.bia_decode_paged_fp8(d, q[:, :2].contiguous(), kc, kc, ks, ks, kvp, idx, last, kvp, last,
                                 ws, q[:, :2].contiguous())
    with pytest.raises(ValueError, match="CUDA"):
        bia.bia_decode_paged_fp8(d, q, kc, kc, ks, ks, kvp, idx, last, kvp, last, ws, q)
    with pytest.raises(ValueError, match="q must be"):
        bia.bia_prefill_ragged(d, q, x, x, ip, ip, ip, ip, ws, q)
    qq = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k must be"):
        bia.bia_prefill_ragged(d, qq, qq, x, ip, ip, ip, ip, ws, qq)
    with pytest.raises(ValueError, match="CUDA"):
        bia.bia_prefill_ragged(d, qq, x, x, ip, ip, ip, ip, ws, qq)


def test_the_plain_rounding_is_e4m3(bia):
    # the 64-bit rounding the GPU tests rely on, against torch's cast of values
    # on and between the grid's points
    grid = torch.arange(127, dtype=torch.uint8).view(fu.E4M3).double()
    y = torch.cat([grid, (grid[1:] + grid[:-1]) / 2, grid[1:] * 0.99, grid[:-1] * 1.01])
    y = torch.cat([y, -y])
    assert torch.equal(fu.round_e4m3(y), y.float().to(fu.E4M3).double())
