"""Device index arrays of a packed prefill that hold anything at all: nothing
is computed, out and lse read NaN, and the plan ends at once."""
import time

import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def refused(qo, kv, d, split=128):
    """A call of len(qo) - 1 requests of 5 tokens and keys whose device arrays
    hold `qo` and `kv` instead; seconds until it is done."""
    n = len(qo) - 1
    desc = bia.make_desc(16, 2, d, 1)
    host = fu.indptr_of([5] * n)
    q = torch.zeros(5 * n, 16, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(5 * n, 2, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, host, host, False, split),
                     dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    dev = [torch.tensor(x, dtype=torch.int64).to(torch.int32).to(DEV) for x in (qo, kv)]
    torch.cuda.synchronize()
    t = time.perf_counter()
    bia.bia_prefill_ragged(desc, q, k, k, *dev, host, host, ws, out, lse, causal=False,
                           split_size=split)
    status = bia.bia_read_status(ws)
    t = time.perf_counter() - t
    assert status == 2 and torch.isnan(out).all() and torch.isnan(lse).all()
    return t


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n", [3, 40, 1100])
def test_arrays_of_anything(d, n):
    end = 5 * n
    g = torch.Generator().manual_seed(n)
    honest = list(range(0, end + 1, 5))
    far = [0] + [1 << 30] * (n - 1) + [end]     # up to 2^30 and back
    wild = [0] + torch.randint(-2 ** 31, 2 ** 31, (n - 1,), generator=g).tolist() + [end]
    below = [0] + [-7] * (n - 1) + [end]
    for bad in (far, wild, below):
        assert refused(bad, honest, d) < 1
        assert refused(honest, bad, d) < 1
        assert refused(bad, bad, d) < 1
    assert refused(honest[:-1] + [end + 1], honest, d) < 1
    # lengths shared out otherwise: a plan of another size
    assert refused([0] + [0] * (n - 1) + [end], honest, d) < 1
