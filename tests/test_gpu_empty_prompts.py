"""Empty tensors through the binding: nothing is launched."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("keys", [0, 10])
@pytest.mark.parametrize("d", [128, 256])
def test_a_packed_prefill_without_tokens(keys, d):
    desc = bia.make_desc(8, 2, d, 1)
    qo, kv = fu.indptr_of([0, 0]), fu.indptr_of([0, keys])
    rows = lambda n, h: torch.zeros(n, h, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(bia.bia_prefill_ragged_workspace_size(desc, qo, kv), dtype=torch.uint8, device=DEV)
    before = bia.bia_launch_count()
    bia.bia_prefill_ragged(desc, rows(0, 8), rows(keys, 2), rows(keys, 2), qo.to(DEV), kv.to(DEV), qo,
                           kv, ws, rows(0, 8), torch.zeros(0, 8, device=DEV))
    assert bia.bia_launch_count() == before


def test_an_append_and_a_gather_without_tokens():
    desc = bia.make_desc(8, 2, 64, 16)
    codes = torch.zeros(3, 16, 2, 64, dtype=torch.uint8, device=DEV).view(fu.E4M3)
    scale = torch.zeros(3, 16, 2, dtype=torch.uint8, device=DEV).view(fu.E8M0)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    ip, kv, idx, last = fu.indptr_of([0, 0]), fu.indptr_of([1, 2]), torch.arange(3, dtype=torch.int32), \
        torch.tensor([4, 5], dtype=torch.int32)
    tail = [x.to(DEV) for x in (ip, kv, idx, last)] + [ip, kv, last]
    status = torch.ones(1, dtype=torch.int32, device=DEV)
    before = bia.bia_launch_count()
    bia.bia_append_paged_kv_fp8(desc, none, none, codes, codes, scale, scale, *tail, status=status)
    assert bia.bia_read_status(status) == 0
    bia.bia_gather_paged_kv_fp8(desc, codes, codes, scale, scale, none, none, *tail)
    assert bia.bia_launch_count() == before
