"""Scale bytes that the append never writes, read back: 0 to 6, down to the
subnormal 2^-127."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import fp8_util as fu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_small_scales_round_to_bf16_once():
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(1, 1, 1, 256)
    n = 7
    kc = codes.repeat(n, 1, 1, 1).view(fu.E4M3)
    ks = torch.arange(n, dtype=torch.uint8, device=DEV).view(-1, 1, 1).view(fu.E8M0)
    ip, last = fu.indptr_of([n]), torch.tensor([1], dtype=torch.int32)
    idx = torch.arange(n, dtype=torch.int32, device=DEV)
    ko = torch.empty(n, 1, 256, dtype=torch.bfloat16, device=DEV)
    vo = torch.empty_like(ko)
    bia.bia_gather_paged_kv_fp8(bia.make_desc(1, 1, 256, 1), kc, kc, ks, ks, ko, vo, ip.to(DEV),
                                ip.to(DEV), idx, last.to(DEV), ip, ip, last)
    want = fu.cache_values(kc, ks).view(n, 1, 256)
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(ko))
    # bf16's subnormals are multiples of 2^-133: ties to even, on the host in 64 bits
    step = torch.exp2(torch.frexp(want.nan_to_num(0.0))[1].clamp(min=-125).double() - 8)
    want = torch.round(want.nan_to_num(0.0) / step) * step
    assert torch.equal(ko.double().nan_to_num(0.0), want)
    assert torch.equal(ko.view(torch.int16), vo.view(torch.int16))
