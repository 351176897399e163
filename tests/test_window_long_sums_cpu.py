"""How a windowed call's plan cuts ranges of very many keys, by the workspace that it asks for (without a GPU)."""
import pytest
import torch

from tests.test_window_refusals_cpu import bia, i32, pytestmark  # noqa: F401

MOST = 2**31 - 1


def extend(bia, desc, n, keys, window, sinks, split=0):  # noqa: F811
    return bia.bia_prefill_window_workspace_size(desc, window, sinks, i32([0, n]), i32([0, -(-keys // 16)]),
                                                 i32([keys - (-(-keys // 16) - 1) * 16]), split)


@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 64), (32, 8, 128), (16, 8, 256)])
def test_extend(bia, hq, hkv, d):  # noqa: F811
    desc = bia.make_desc(hq, hkv, d, 16)
    states = lambda n, parts: n * parts * hq * (d + 1) * 4
    keys = 1 << 20
    # few sinks and a short window are one state, whatever the length
    assert extend(bia, desc, 4, keys, 1024, 4096) == extend(bia, desc, 4, keys, 1024, 4) < 4096
    # a state has 65536 keys at most, whatever split size is asked for
    for window, sinks in ((MOST, 0), (1024, MOST), (100000, 4), (1024, 70000)):
        want = extend(bia, desc, 4, keys, window, sinks, 65536)
        assert extend(bia, desc, 4, keys, window, sinks, 1 << 24) == want
    assert extend(bia, desc, 4, keys, MOST, 0, 1 << 24) >= states(4, 16)
    # many sinks behind the window: every split up to the window
    assert extend(bia, desc, 4, keys, 1024, 70000, 1 << 24) >= states(4, 16)
    # windows of one state keep theirs at any split size
    assert extend(bia, desc, 4, keys, 65536, 4, 1 << 24) == extend(bia, desc, 4, 70000, 65536, 4, 1 << 24) < 4096


@pytest.mark.parametrize("d", [64, 128])
def test_decode(bia, d):  # noqa: F811
    desc = bia.make_desc(8, 4, d, 16)
    size = lambda keys, split: bia.bia_decode_window_workspace_size(desc, MOST, 0, i32([0, keys // 16]), i32([16]), split)
    for split in (1 << 17, 1 << 20, 1 << 30, MOST // 128 * 128):
        assert size(1 << 20, split) == size(1 << 20, 65536) >= 16 * 8 * (d + 1) * 4
        assert size(65536, split) == size(65536, 65536) < 4096
        b = bia.make_bounds(max_kv_len=1 << 20)
        assert bia.bia_decode_window_bounded_workspace_size(desc, b, MOST, 0, 1, split) == size(1 << 20, 65536)


@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 64), (32, 8, 128), (16, 8, 256)])
def test_default_split_with_sinks(bia, hq, hkv, d):  # noqa: F811
    """A short window is one state by default, but not with all the sinks that it may meet."""
    desc = bia.make_desc(hq, hkv, d, 16)
    states = lambda n, parts: n * parts * hq * (d + 1) * 4
    keys = 1 << 20
    assert extend(bia, desc, 4, keys, 1024, MOST) >= states(4, keys // 4096)
    assert extend(bia, desc, 4, keys, 1024, MOST) == extend(bia, desc, 4, keys, MOST, 0)
    assert extend(bia, desc, 4, keys, 1024, 5000) >= states(4, 2)
