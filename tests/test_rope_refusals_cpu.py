"""What the rotation calls refuse, on the host: bad arguments come back before
anything is enqueued, so these run without a GPU (device addresses are made up
and never dereferenced)."""
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


def rows_call(bia, desc, rope, *, table=FAKE, positions=FAKE, q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE,
              qs=0, total=5, weight=FAKE, status=None):
    return bia.load().bia_norm_rope(
        ctypes.byref(desc) if desc else None, ctypes.byref(rope) if rope else None, p(table),
        p(positions), p(q), p(k), qs, 0, p(weight), p(FAKE), total, p(q_out), p(k_out), 0, 0,
        status and p(status), None)


def append_call(bia, fp8, desc, rope, rows, kvp, last, *, table=FAKE, q=FAKE, q_out=FAKE, k=FAKE,
                cache=FAKE, scale=FAKE, pages=1 << 20, vs=0, k_out=FAKE, status=None):
    t = [torch.tensor(x, dtype=torch.int32) for x in (rows, kvp, last)]
    head = [ctypes.byref(desc), ctypes.byref(rope), p(table), None, p(q), p(k), p(FAKE), 0, 0, vs,
            p(FAKE), p(FAKE), p(cache), p(FAKE)]
    mid = [pages] + [p(FAKE)] * 4 + [p(x.data_ptr()) for x in t] + [len(rows) - 1]
    if fp8:
        return bia.load().bia_append_paged_kv_fp8_rope(*head, p(scale), p(FAKE), *mid, p(q_out),
                                                       p(k_out), 0, 0, status and p(status), None)
    return bia.load().bia_append_paged_kv_rope(*head, *mid, p(q_out), 0, status and p(status), None)


def test_rotation_itself(bia):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d = bia.make_desc(32, 8, 128, 16)
    ok = dict(total=0)
    assert rows_call(bia, d, bia.make_rope(128, 10), **ok) == bia.BIA_OK
    assert rows_call(bia, None, bia.make_rope(128, 10), **ok) == inv
    assert rows_call(bia, d, None, **ok) == inv
    for rot in (0, 8, 24, 144, -16):
        r = bia.make_rope(16, 10)
        r.rot_dim = rot
        assert rows_call(bia, d, r, **ok) == uns
    assert rows_call(bia, d, bia.make_rope(64, 0), **ok) == inv
    assert rows_call(bia, d, bia.make_rope(64, 10, norm_eps=-1), **ok) == inv
    assert rows_call(bia, d, bia.make_rope(64, 10, norm_eps=float("nan")), **ok) == inv
    assert rows_call(bia, d, bia.make_rope(64, 10, norm_eps=float("inf")), **ok) == inv
    r = bia.make_rope(64, 10)
    r.num_axes = 5
    assert rows_call(bia, d, r, **ok) == uns
    r = bia.make_rope(64, 10, 3, [0] * 32)
    r.freq_axis[31] = 3
    assert rows_call(bia, d, r, **ok) == inv
    assert rows_call(bia, bia.make_desc(32, 8, 80, 16), bia.make_rope(64, 10), **ok) == uns
    with pytest.raises(ValueError):
        bia.make_rope(64, 10, 3, [0] * 31)
    with pytest.raises(ValueError):
        bia.make_rope(64, 10, 3, [0] * 31 + [3])
    with pytest.raises(ValueError):
        bia.make_rope(64, 10, 2)


def test_rows(bia):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d, r = bia.make_desc(32, 8, 128, 3), bia.make_rope(128, 10)  # the page size is not used
    for bad in (dict(table=0), dict(table=FAKE + 8), dict(positions=0), dict(positions=FAKE + 2),
                dict(q=0), dict(q_out=0), dict(k_out=0), dict(k=0), dict(q=FAKE + 8),
                dict(q=0, q_out=0, k=0, k_out=0), dict(weight=FAKE + 4), dict(qs=4095),
                dict(qs=4100), dict(total=-1), dict(status=FAKE + 2)):
        assert rows_call(bia, d, r, **bad) == inv, bad
    assert rows_call(bia, d, r, total=1 << 26) == uns
    assert rows_call(bia, d, r, total=0, table=0, positions=0, q=0, q_out=0, k=0, k_out=0) == bia.BIA_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_appends(bia, fp8):
    inv, uns = bia.BIA_ERR_INVALID_ARG, bia.BIA_ERR_UNSUPPORTED
    d, r = bia.make_desc(32, 8, 128, 16), bia.make_rope(128, 10)
    call = lambda *a, desc=d, **k: append_call(bia, fp8, desc, r, *a, **k)
    assert call([0, 17], [0, 1], [16]) == inv  # more rows than keys
    assert call([0, 5, 3], [0, 1, 2], [16, 16]) == inv  # indptr falls
    assert call([1, 5], [0, 1], [16]) == inv
    assert call([0, 5], [0, 1], [17]) == inv  # past the page
    assert call([0, 5], [0, 1], [0]) == inv
    assert call([0, 5], [1, 0], [5]) == inv
    assert call([0, 5], [0, 1], [5], pages=0) == inv
    for bad in (dict(table=0), dict(q=0), dict(q_out=0), dict(k=0), dict(cache=0), dict(cache=FAKE + 8),
                dict(vs=1020), dict(vs=1028), dict(q_out=FAKE + 8), dict(status=FAKE + 1)):
        assert call([0, 5], [0, 1], [5], **bad) == inv, bad
    if fp8:
        for bad in (dict(scale=0), dict(scale=FAKE + 1), dict(k_out=FAKE + 8)):
            assert call([0, 5], [0, 1], [5], **bad) == inv, bad
    assert call([0, 5], [0, 1], [3], desc=bia.make_desc(32, 8, 128, 3)) == uns
    assert call([0, 1 << 27], [0, 1 << 23], [16]) == uns
    assert call([0, 0], [0, 0], [0]) == bia.BIA_OK  # nothing to do


def test_binding(bia):
    d, r = bia.make_desc(4, 2, 64, 16), bia.make_rope(64, 10)
    table = torch.zeros(10, 64)
    at = torch.zeros(1, 3, dtype=torch.int32)
    q, k = torch.zeros(3, 4, 64).bfloat16(), torch.zeros(3, 2, 64).bfloat16()
    qo, ko = q.clone(), k.clone()
    with pytest.raises(TypeError):
        bia.bia_norm_rope(d, r, table, at, None, None, None, None)
    with pytest.raises(TypeError):
        bia.bia_norm_rope(d, r, table, None, q, k, qo, ko)
    with pytest.raises(TypeError):
        bia.bia_norm_rope(d, r, table, at, q, k, None, ko)
    with pytest.raises(TypeError):
        bia.bia_norm_rope(d, r, table.double(), at, q, k, qo, ko)
    with pytest.raises(TypeError):
        bia.bia_norm_rope(d, r, table, at.long(), q, k, qo, ko)
    with pytest.raises(TypeError):
        bia.bia_norm_rope(d, r, table, at, q.float(), k, qo, ko)
    for bad in (dict(table=table[:9]), dict(at=at[:, :2].contiguous()), dict(qo=qo[:2]), dict(ko=qo),
                dict(w=torch.zeros(32))):
        with pytest.raises(ValueError):
            bia.bia_norm_rope(d, r, bad.get("table", table), bad.get("at", at), q, k,
                              bad.get("qo", qo), bad.get("ko", ko), bad.get("w"))
