"""Every kernel's launch set-up is made on the device that the call runs on:
the library's host code over a made-up runtime with two devices of different
size, the same calls on each."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
pytestmark = pytest.mark.skipif(not os.path.exists(NVCC) or shutil.which("gcc") is None,
                                reason="nvcc not available")
FAKE = ctypes.c_void_p(1 << 20)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from invariant_paged_attention_gb300 import build
    import invariant_paged_attention_gb300 as bia
    build.build()
    objects = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    if not all(os.path.exists(o) for o in objects):
        build.build(force=True)
    out = tmp_path_factory.mktemp("fake")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(NVCC))), "include")
    run = lambda *cmd: subprocess.run(cmd, check=True, capture_output=True, text=True)
    run("gcc", "-c", "-fPIC", "-O1", "-I", include, os.path.join(HERE, "fake_cuda_runtime.c"), "-o",
        str(out / "fake.o"))
    so = str(out / "libfake.so")
    run("g++", "-shared", "-Wl,-Bsymbolic", *objects, str(out / "fake.o"), "-o", so)
    real, bia._lib = bia._lib, None
    try:
        made = bia.load(so)
    finally:
        bia._lib = real
    made.fake_grid.restype = ctypes.c_uint
    return bia, made


def at(x, dtype=torch.int32):
    t = torch.tensor(x, dtype=dtype)
    return t, ctypes.c_void_p(t.data_ptr())


def calls(bia, lib):
    """(name, call) of every attention entry point and shape of kernel."""
    keep = []

    def arr(x, dtype=torch.int32):
        t, p = at(x, dtype)
        keep.append(t)
        return p

    f = FAKE
    qo, kv, last = arr([0, 200, 9000]), arr([0, 60000, 120000]), arr([1, 1])
    mask_at = arr([0, 200 * 60000], torch.int64)
    for d in (64, 96, 128, 256):
        for g in (1, 2, 4, 8):
            desc = bia.make_desc(4 * g, 4, d, 1)
            r = ctypes.byref(desc)
            keep.append(desc)
            yield f"prefill {d} {g}", lambda r=r: lib.bia_prefill_paged(
                r, f, f, f, 1 << 20, f, f, f, f, qo, kv, last, 2, 1, 0, f, BIG, f, None, None)
            yield f"masked prefill {d} {g}", lambda r=r: lib.bia_prefill_paged_mask(
                r, f, f, f, 1 << 20, f, f, f, f, qo, kv, last, 2, 0, 0, f, 1 << 30, f, mask_at, f, BIG,
                f, None, None)
            yield f"decode {d} {g}", lambda r=r: lib.bia_decode_paged(
                r, f, f, f, 1 << 20, f, f, f, kv, last, 2, 0, f, BIG, f, None, None)
            yield f"8-bit decode {d} {g}", lambda r=r: lib.bia_decode_paged_fp8(
                r, f, f, f, f, f, 1 << 20, f, f, f, kv, last, 2, 0, f, BIG, f, None, None)
            yield f"packed prefill {d} {g}", lambda r=r: lib.bia_prefill_ragged(
                r, f, f, f, 0, 0, 0, f, f, qo, kv, 2, 1, 0, f, BIG, f, None, None)
    for heads in (8, 16, 32):
        mla = bia.make_mla_desc(heads, 1)
        r = ctypes.byref(mla)
        keep.append(mla)
        yield f"mla decode {heads}", lambda r=r: lib.bia_mla_decode_paged(
            r, f, f, f, f, 1 << 20, f, f, f, kv, last, 2, 0, f, BIG, f, None, None)
        yield f"mla prefill {heads}", lambda r=r: lib.bia_mla_prefill_paged(
            r, f, f, f, f, 1 << 20, f, f, f, f, qo, kv, last, 2, 0, f, BIG, f, None, None)


def test_every_call_runs_on_the_second_device(lib):
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


def test_persistent_grids_follow_the_device_s_size(lib):
    bia, lib = lib
    for dev, sms in ((0, 152), (1, 100), (0, 152)):
        lib.fake_set_device(dev)
        for name, call in calls(bia, lib):
            if name.startswith(("decode 128", "8-bit decode", "packed prefill 128")):
                before = lib.fake_launches()
                assert call() == 0
                assert lib.fake_grid(before + 1) == sms, (dev, name)  # behind the plan
            if name.startswith("prefill 128"):  # its merge: two CTAs an SM
                assert call() == 0
                assert lib.fake_grid(lib.fake_launches() - 1) == 2 * sms, (dev, name)
