"""One long row among many short prompts: its splits are items of their own,
with the bits of the row alone."""
import pytest

import invariant_paged_attention_gb300 as bia
from tests.gpu_util import same_bits
from tests.test_gpu_prefill_ragged import check, draw, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_a_long_row_among_short_prompts(d, causal):
    hq, hkv = 16, 4
    q_lens, kv_lens = [64] * 50 + [3] + [100] * 40, [64] * 50 + [60_001] + [100] * 40
    q, k, v = draw(hq, hkv, d, q_lens, kv_lens, d)
    before = bia.bia_launch_count()
    out, lse = run(q, k, v, q_lens, kv_lens, causal)
    assert bia.bia_launch_count() - before == 3  # plan, attention, merge
    qa, ka = 64 * 50, 64 * 50
    one, l = run(q[qa:qa + 3], k[ka:ka + 60_001], v[ka:ka + 60_001], [3], [60_001], causal)
    assert same_bits(one, out[qa:qa + 3]) and same_bits(l, lse[qa:qa + 3])
    check(q, k, v, q_lens, kv_lens, out, lse, causal)


def test_many_equal_rows_fold_with_the_same_bits():
    hq, hkv, d = 16, 4, 128
    q_lens, kv_lens = [64] * 90, [9000] * 90
    q, k, v = draw(hq, hkv, d, q_lens, kv_lens, 3)
    before = bia.bia_launch_count()
    out, lse = run(q, k, v, q_lens, kv_lens)
    assert bia.bia_launch_count() - before == 2  # no merge
    for i in (0, 41, 89):
        a, b = 64 * i, 9000 * i
        one, l = run(q[a:a + 64], k[b:b + 9000], v[b:b + 9000], [64], [9000])
        assert same_bits(one, out[a:a + 64]) and same_bits(l, lse[a:a + 64])
