"""A paged call without its host mirrors is refused, whatever the page size
(device addresses are made up and never dereferenced)."""
import ctypes
import os
import shutil

import pytest
import torch

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


def arrays(pages):
    return (torch.tensor([0, 2], dtype=torch.int32), torch.tensor([0, pages], dtype=torch.int32),
            torch.tensor([1], dtype=torch.int32))


def at(t):
    return p(t.data_ptr())


@pytest.mark.parametrize("page", [1, 16])
def test_workspace_sizes_without_last_page_lengths(bia, page):
    lib = bia.load()
    desc, mla = bia.make_desc(8, 2, 128, page), bia.make_mla_desc(16, page)
    d, m = ctypes.byref(desc), ctypes.byref(mla)
    qo, kv, last = arrays(5)
    for l, want in ((at(last), True), (None, False)):
        sizes = (lib.bia_prefill_workspace_size(d, at(qo), at(kv), l, 1, 1, 0),
                 lib.bia_decode_workspace_size(d, at(kv), l, 1, 0),
                 lib.bia_decode_fp8_workspace_size(d, at(kv), l, 1, 0),
                 lib.bia_mla_decode_workspace_size(m, at(kv), l, 1, 0),
                 lib.bia_mla_prefill_workspace_size(m, at(qo), at(kv), l, 1, 0))
        assert [s > 0 for s in sizes] == [want] * 5


@pytest.mark.parametrize("page", [1, 16])
def test_calls_without_last_page_lengths(bia, page):
    lib, inv = bia.load(), bia.BIA_ERR_INVALID_ARG
    desc = bia.make_desc(8, 2, 128, page)
    d = ctypes.byref(desc)
    qo, kv, _ = arrays(5)
    f, big = p(FAKE), 1 << 30
    mask_at = torch.tensor([0], dtype=torch.int64)
    assert lib.bia_prefill_paged(d, f, f, f, 64, f, f, f, f, at(qo), at(kv), None, 1, 1, 0, f, big,
                                 f, None, None) == inv
    assert lib.bia_decode_paged(d, f, f, f, 64, f, f, f, at(kv), None, 1, 0, f, big, f, None,
                                None) == inv
    assert lib.bia_decode_paged_noalloc(d, f, f, f, 64, f, f, f, at(kv), None, 1, 0, f, None,
                                        None) == inv
    assert lib.bia_decode_paged_fp8(d, f, f, f, f, f, 64, f, f, f, at(kv), None, 1, 0, f, big, f,
                                    None, None) == inv
    assert lib.bia_prefill_paged_mask(d, f, f, f, 64, f, f, f, f, at(qo), at(kv), None, 1, 1, 0, f,
                                      64, f, at(mask_at), f, big, f, None, None) == inv


def test_packed_calls_have_no_last_page_lengths(bia):
    desc = bia.make_desc(8, 2, 128, 16)
    qo, kv, _ = arrays(5)
    assert bia.bia_prefill_ragged_workspace_size(desc, qo, kv) > 0
