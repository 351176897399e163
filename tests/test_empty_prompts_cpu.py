"""A packed prefill without a token has nothing to do, whether its empty
tensors have addresses or none; with tokens, missing rows are refused."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
FAKE = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def bia():
    from invariant_paged_attention_gb300 import build
    build.build()
    import invariant_paged_attention_gb300 as m
    m.load()
    return m


def prompt(bia, qo, kv, q=FAKE, k=FAKE, v=FAKE, out=FAKE):
    qo, kv = (torch.tensor(x, dtype=torch.int32) for x in (qo, kv))
    at = lambda t: ctypes.c_void_p(t.data_ptr())
    return bia.load().bia_prefill_ragged(
        ctypes.byref(bia.make_desc(8, 2, 128, 1)), q, k, v, 0, 0, 0, FAKE, FAKE, at(qo), at(kv),
        len(qo) - 1, 1, 0, FAKE, 1 << 40, out, None, None)


def test_no_tokens(bia):
    assert prompt(bia, [0, 0], [0, 10]) == bia.BIA_OK
    assert prompt(bia, [0, 0], [0, 10], q=None, out=None) == bia.BIA_OK
    assert prompt(bia, [0, 0, 0], [0, 0, 0], q=None, k=None, v=None, out=None) == bia.BIA_OK


def test_missing_rows(bia):
    inv = bia.BIA_ERR_INVALID_ARG
    for name in ("q", "k", "v", "out"):
        assert prompt(bia, [0, 5], [0, 10], **{name: None}) == inv
    assert prompt(bia, [0, 0, 4], [0, 9, 10], q=None, out=None) == inv  # 4 tokens over 1 key
