"""The rotation and windowed calls set their kernels up on the device that they
run on: the host code over the made-up runtime with two devices."""
import ctypes

import torch

from tests.test_two_devices_cpu import BIG, FAKE, at, lib, pytestmark  # noqa: F401


def calls(bia, lib):
    keep = []

    def arr(x):
        t, p = at(x)
        keep.append(t)
        return p

    f = FAKE
    qo, kv, last = arr([0, 200, 30000]), arr([0, 60000, 120000]), arr([1, 1])
    for d in (64, 96, 128, 256):
        for g in (1, 2, 4, 8):
            for page in (1, 16):
                desc = bia.make_desc(4 * g, 4, d, page)
                bounds = bia.make_bounds(max_kv_len=1 << 20)
                r, b = ctypes.byref(desc), ctypes.byref(bounds)
                keep += [desc, bounds]
                yield f"extend {d} {g} {page}", lambda r=r: lib.bia_prefill_paged_window(
                    r, 1024, 4, f, f, f, 1 << 20, f, f, f, f, qo, kv, last, 2, 0, f, BIG, f, None, None)
                yield f"decode {d} {g} {page}", lambda r=r: lib.bia_decode_paged_window(
                    r, 40960, 4, f, f, f, 1 << 20, f, f, f, kv, last, 2, 0, f, BIG, f, None, None)
                yield f"bounded decode {d} {g} {page}", lambda r=r, b=b: lib.bia_decode_paged_window_bounded(
                    r, b, 40960, 4, f, f, f, 1 << 20, f, f, f, 2, 0, f, BIG, f, None, None)
        for inter in (False, True):
            desc, rope = bia.make_desc(8, 4, d, 16), bia.make_rope(32, 10, interleaved=inter)
            r, p = ctypes.byref(desc), ctypes.byref(rope)
            keep += [desc, rope]
            yield f"rotate {d}", lambda r=r, p=p: lib.bia_norm_rope(
                r, p, f, f, f, f, 0, 0, f, f, 9000, f, f, 0, 0, None, None)
            kv16 = arr([0, 4000, 8000])
            yield f"append {d}", lambda r=r, p=p, kv=kv16: lib.bia_append_paged_kv_rope(
                r, p, f, None, f, f, f, 0, 0, 0, f, f, f, f, 1 << 20, f, f, f, f, qo, kv, last, 2, f, 0, None, None)
            yield f"8-bit append {d}", lambda r=r, p=p, kv=kv16: lib.bia_append_paged_kv_fp8_rope(
                r, p, f, None, f, f, f, 0, 0, 0, f, f, f, f, f, f, 1 << 20, f, f, f, f, qo, kv, last, 2, f, f, 0, 0,
                None, None)


def test_every_call_runs_on_the_second_device(lib):  # noqa: F811
    bia, lib = lib
    failed = []
    for dev in (0, 1):
        lib.fake_set_device(dev)
        for name, call in calls(bia, lib):
            before = lib.fake_launches()
            rc = call()
            if rc != 0 or lib.fake_launches() == before:
                failed.append((dev, name, rc))
    assert not failed


def test_persistent_grids_follow_the_device_s_size(lib):  # noqa: F811
    bia, lib = lib
    for dev, sms in ((0, 152), (1, 100), (0, 152)):
        lib.fake_set_device(dev)
        for name, call in calls(bia, lib):
            if name.startswith(("extend", "decode 128", "bounded decode 128")):
                before = lib.fake_launches()
                assert call() == 0
                at_kernel = before + (1 if name.startswith("extend") else 0)  # behind the plan
                assert lib.fake_grid(at_kernel) == sms, (dev, name)


def test_a_call_of_fewer_items_than_ctas(lib):  # noqa: F811
    """The status words of a decode's CTAs fit its workspace on any device."""
    bia, lib = lib
    kvp, kv = at([0, 3])
    last, lp = at([1])
    for dev in (0, 1):
        lib.fake_set_device(dev)
        for d in (64, 128):
            desc = bia.make_desc(8, 2, d, 1)
            need = lib.bia_decode_window_workspace_size(ctypes.byref(desc), 5, 0, kv, lp, 1, 0)
            assert lib.bia_decode_paged_window(ctypes.byref(desc), 5, 0, FAKE, FAKE, FAKE, 8, FAKE, FAKE, FAKE, kv, lp, 1, 0,
                                               FAKE, need, FAKE, None, None) == 0
            assert lib.bia_decode_paged_window(ctypes.byref(desc), 5, 0, FAKE, FAKE, FAKE, 8, FAKE, FAKE, FAKE, kv, lp, 1, 0,
                                               FAKE, need - 1, FAKE, None, None) == bia.BIA_ERR_WORKSPACE_TOO_SMALL
    assert isinstance(kvp, torch.Tensor) and isinstance(last, torch.Tensor)
