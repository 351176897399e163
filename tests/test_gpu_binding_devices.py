"""Tensors that are not on the GPU, one at a time, in the rotation and windowed calls of the binding: refused by
name, with nothing launched."""
import pytest
import torch

import invariant_paged_attention_gb300 as bia
from tests import rope_util as ru
from tests import window_util as wu

pytestmark = pytest.mark.gpu


def refused(call, args, names):
    for name in names:
        bad = dict(args)
        bad[name] = args[name].cpu().pin_memory() if name != "q" else args[name].cpu()
        before = bia.bia_launch_count()
        with pytest.raises(ValueError, match="cpu"):
            call(**bad)
        assert bia.bia_launch_count() == before, name
    before = bia.bia_launch_count()
    call(**args)
    assert bia.bia_launch_count() > before


def test_windowed_calls():
    c = wu.Batch([300, 40], [1, 1], 8, 4, 128, 16, 100, 4, spoil=False)
    args = dict(q=c.q, k_cache=c.k_cache, v_cache=c.v_cache, kv_indptr=c.dev[0], kv_indices=c.dev[1], kv_last_page_len=c.dev[2],
                kv_indptr_host=c.kvp, kv_last_page_len_host=c.last, out=c.out, lse=c.lse,
                workspace=torch.empty(bia.bia_decode_window_workspace_size(c.desc, 100, 4, c.kvp, c.last), dtype=torch.uint8,
                                      device="cuda"))
    device = ["q", "k_cache", "v_cache", "kv_indptr", "kv_indices", "kv_last_page_len", "out", "lse", "workspace"]
    refused(lambda **kw: bia.bia_decode_paged_window(c.desc, 100, 4, **kw), args, device)
    e = wu.Batch([300, 40], [30, 40], 8, 4, 128, 16, 100, 4, spoil=False)
    args |= dict(q=e.q, k_cache=e.k_cache, v_cache=e.v_cache, qo_indptr=e.qo.cuda(), qo_indptr_host=e.qo, out=e.out, lse=e.lse,
                 kv_indices=e.dev[1],
                 workspace=torch.empty(bia.bia_prefill_window_workspace_size(e.desc, 100, 4, e.qo, e.kvp, e.last),
                                       dtype=torch.uint8, device="cuda"))
    refused(lambda **kw: bia.bia_prefill_paged_window(e.desc, 100, 4, **kw), args, device + ["qo_indptr"])


def test_rotation_calls():
    gen = torch.Generator().manual_seed(1)
    desc, (rope, _) = bia.make_desc(8, 4, 128, 16), ru.make(128, 400)
    rows = ru.rows((30, 16, 128), gen).cuda()
    w = [x.cuda() for x in ru.weights(128, gen)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    new = lambda h: torch.empty(30, h, 128, dtype=torch.bfloat16, device="cuda")
    args = dict(table=ru.table_of(400, 128).cuda(), positions=torch.arange(30).int().cuda()[None], q=rows[:, :8], k=rows[:, 8:12],
                q_out=new(8), k_out=new(4), q_weight=w[0], k_weight=w[1], status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    refused(lambda **kw: bia.bia_norm_rope(desc, rope, **kw), args, list(args))
    caches = [torch.zeros(3, 16, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    host = i32(0, 30), i32(0, 2), i32(14)
    args = {k: v for k, v in args.items() if k not in ("k", "k_out")} | dict(
        k_new=rows[:, 8:12], v_new=rows[:, 12:], k_cache=caches[0], v_cache=caches[1], append_indptr=host[0].cuda(),
        kv_indptr=host[1].cuda(), kv_indices=i32(2, 0).cuda(), kv_last_page_len=host[2].cuda())
    refused(lambda **kw: bia.bia_append_paged_kv_rope(desc, rope, append_indptr_host=host[0], kv_indptr_host=host[1],
                                                      kv_last_page_len_host=host[2], **kw), args, list(args))
