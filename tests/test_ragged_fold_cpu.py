"""Which packed prefills fold a row's splits in the CTA that computes it: those
whose longest row of keys is no longer than a CTA's share of the whole call.
The workspace tells: a folded call holds a state per CTA, any other one per row
and split."""
import os
import shutil

import pytest
import torch

from tests import fp8_util as fu

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
CTAS, ROWS = 152, 128  # of the chip; rows of a q tile


@pytest.fixture(scope="module")
def bia():
    from invariant_paged_attention_gb300 import build
    build.build()
    import invariant_paged_attention_gb300 as m
    m.load()
    return m


def folds(bia, q_lens, kv_lens, hq=32, hkv=8, d=128, causal=True, split=0):
    need = bia.bia_prefill_ragged_workspace_size(bia.make_desc(hq, hkv, d, 1), fu.indptr_of(q_lens),
                                                 fu.indptr_of(kv_lens), causal, split)
    states = CTAS * 2 * ROWS * max(64, 1 << (d - 1).bit_length()) * 4
    merged = sum(q * -(-k // (split or 4096)) * hq * d * 4
                 for q, k in zip(q_lens, kv_lens) if k > (split or 4096))
    assert abs(states - merged) > 2 ** 21  # the two can be told apart
    assert min(abs(need - states), abs(need - merged)) < 2 ** 20
    return abs(need - states) < abs(need - merged)


def test_one_long_row_among_short_prompts_keeps_its_splits(bia):
    # 40 short prompts and a token over 500000 keys: 320 items of a block and
    # 8 of 3907, 26 times a CTA's share
    assert not folds(bia, [64] * 40 + [1], [64] * 40 + [500_000])
    assert not folds(bia, [64] * 40 + [1], [64] * 40 + [500_000], causal=False)
    assert not folds(bia, [200] * 100 + [64], [200] * 100 + [100_000])


def test_even_batches_and_long_prompts_fold(bia):
    assert folds(bia, [16384], [16384])
    assert folds(bia, [16384], [16384], hq=8, hkv=2)
    assert folds(bia, [8192, 4096, 6000], [8192, 4096, 6000])
    assert folds(bia, [2048] * 4, [2048 + 16383] * 4, hq=16, hkv=4)
    assert folds(bia, [1500, 700, 1, 64, 0, 1100], [1500, 2900, 1300, 64, 7, 1101], split=256)
    assert folds(bia, [100] * 64, [9000] * 64, d=64, causal=False)
    # the long row is one of many like it
    assert folds(bia, [64] * 60, [100_000] * 60)


def test_few_items_merge(bia):
    assert not folds(bia, [128] * 4, [16383 + 128] * 4)
    assert not folds(bia, [1], [200_000])
