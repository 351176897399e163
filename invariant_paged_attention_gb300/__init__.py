"""Python binding of libbia.so: batch-invariant paged-KV GQA attention on
GB300 (sm_103a).

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of libbia.so; PyTorch supplies device memory and streams.  There is
no fallback: if the library is missing or fails to load, every call raises.

The functions carry the C names of ``include/bia.h`` and take torch tensors:
device tensors for the data and the device copies of the index arrays, CPU
int32 tensors for the host mirrors.  Before a call reaches the library, its
device tensors are checked for dtype, contiguity, the shapes the passed sizes
come from and the CUDA device the call enqueues on (TypeError / ValueError);
everything else (descriptor, index arrays, workspace size) is checked by the
library itself, which raises BiaError with its status code.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbia.so")

BIA_OK = 0
BIA_ERR_INVALID_ARG = -1
BIA_ERR_UNSUPPORTED = -2
BIA_ERR_WORKSPACE_TOO_SMALL = -3
BIA_ERR_CUDA = -4
BIA_Q_TILE_ROWS = 128
BIA_PREFILL_SPLIT = 4096
BIA_RAGGED_MAX_SPLIT = 1 << 24
BIA_DECODE_SPLIT = 2048
BIA_DECODE_FP8_SPLIT = 1024
BIA_WINDOW_DECODE_SPLIT = 512
BIA_WINDOW_MAX_SINKS = 1 << 22

# every symbol include/bia.h exports
EXPORTS = ("bia_prefill_paged", "bia_prefill_workspace_size", "bia_decode_paged",
           "bia_decode_workspace_size", "bia_merge_states", "bia_q_tile_tokens",
           "bia_status_string", "bia_read_status", "bia_set_profile_events",
           "bia_launch_count", "bia_last_error", "bia_decode_paged_noalloc",
           "bia_append_paged_kv", "bia_prefill_paged_mask", "bia_mla_decode_paged",
           "bia_mla_decode_workspace_size", "bia_mla_prefill_paged",
           "bia_mla_prefill_workspace_size", "bia_prefill_paged_bounded",
           "bia_prefill_bounded_workspace_size", "bia_decode_paged_bounded",
           "bia_decode_bounded_workspace_size", "bia_append_paged_kv_fp8",
           "bia_gather_paged_kv_fp8", "bia_decode_paged_fp8", "bia_decode_fp8_workspace_size",
           "bia_decode_paged_fp8_bounded", "bia_decode_fp8_bounded_workspace_size",
           "bia_prefill_ragged", "bia_prefill_ragged_workspace_size", "bia_norm_rope",
           "bia_append_paged_kv_rope", "bia_append_paged_kv_fp8_rope", "bia_decode_paged_window",
           "bia_decode_window_workspace_size", "bia_decode_paged_window_bounded",
           "bia_decode_window_bounded_workspace_size", "bia_prefill_paged_window",
           "bia_prefill_window_workspace_size")


class BiaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status == BIA_ERR_CUDA:
            detail = ": " + load().bia_last_error().decode()
        super().__init__(f"{where} failed: {status_string(status)} ({status}){detail}")


class AttnDesc(ctypes.Structure):
    _fields_ = [("num_qo_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("sm_scale", ctypes.c_float)]


_lib = None


class MlaDesc(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("sm_scale", ctypes.c_float)]


MLA_CKV_DIM, MLA_KPE_DIM = 512, 64


class Bounds(ctypes.Structure):
    _fields_ = [("max_q_len", ctypes.c_int32), ("max_kv_len", ctypes.c_int32),
                ("max_total_q", ctypes.c_int64)]


class Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("num_positions", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("freq_axis", ctypes.c_uint8 * 128)]


def load(path: str = LIB_PATH):
    """Loads libbia.so (built by ``build.build()``); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libbia.so not built at {path}: run "
                           "`python -m invariant_paged_attention_gb300.build`")
    lib = ctypes.CDLL(path)
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    dp = ctypes.POINTER(AttnDesc)
    lib.bia_prefill_paged.argtypes = [dp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32,
                                      i32, vp, sz, vp, vp, vp]
    lib.bia_prefill_paged.restype = ctypes.c_int
    lib.bia_prefill_workspace_size.argtypes = [dp, vp, vp, vp, i32, i32, i32]
    lib.bia_prefill_workspace_size.restype = sz
    lib.bia_decode_paged.argtypes = [dp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, i32, vp, sz,
                                     vp, vp, vp]
    lib.bia_decode_paged.restype = ctypes.c_int
    lib.bia_decode_workspace_size.argtypes = [dp, vp, vp, i32, i32]
    lib.bia_decode_workspace_size.restype = sz
    lib.bia_merge_states.argtypes = [vp, vp, vp, i64, i32, i32, i32, vp, vp, vp]
    lib.bia_merge_states.restype = ctypes.c_int
    lib.bia_q_tile_tokens.argtypes = [i32]
    lib.bia_q_tile_tokens.restype = i32
    lib.bia_status_string.argtypes = [ctypes.c_int]
    lib.bia_status_string.restype = ctypes.c_char_p
    lib.bia_read_status.argtypes = [vp, ctypes.POINTER(i32), vp]
    lib.bia_read_status.restype = ctypes.c_int
    lib.bia_set_profile_events.argtypes = [vp, vp]
    lib.bia_set_profile_events.restype = None
    lib.bia_launch_count.argtypes = []
    lib.bia_launch_count.restype = ctypes.c_uint64
    lib.bia_last_error.argtypes = []
    lib.bia_last_error.restype = ctypes.c_char_p
    lib.bia_decode_paged_noalloc.argtypes = [dp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, i32,
                                             vp, vp, vp]
    lib.bia_decode_paged_noalloc.restype = ctypes.c_int
    lib.bia_append_paged_kv.argtypes = [dp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32,
                                        vp, vp]
    lib.bia_append_paged_kv.restype = ctypes.c_int
    lib.bia_prefill_paged_mask.argtypes = [dp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32,
                                           i32, i32, vp, sz, vp, vp, vp, sz, vp, vp, vp]
    lib.bia_prefill_paged_mask.restype = ctypes.c_int
    mp = ctypes.POINTER(MlaDesc)
    lib.bia_mla_decode_paged.argtypes = [mp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, i32,
                                         vp, sz, vp, vp, vp]
    lib.bia_mla_decode_paged.restype = ctypes.c_int
    lib.bia_mla_decode_workspace_size.argtypes = [mp, vp, vp, i32, i32]
    lib.bia_mla_decode_workspace_size.restype = sz
    lib.bia_mla_prefill_paged.argtypes = [mp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp,
                                          i32, i32, vp, sz, vp, vp, vp]
    lib.bia_mla_prefill_paged.restype = ctypes.c_int
    lib.bia_mla_prefill_workspace_size.argtypes = [mp, vp, vp, vp, i32, i32]
    lib.bia_mla_prefill_workspace_size.restype = sz
    bp = ctypes.POINTER(Bounds)
    lib.bia_prefill_paged_bounded.argtypes = [dp, bp, vp, vp, vp, i64, vp, vp, vp, vp, i32, i32,
                                              i32, vp, sz, vp, vp, vp]
    lib.bia_prefill_paged_bounded.restype = ctypes.c_int
    lib.bia_prefill_bounded_workspace_size.argtypes = [dp, bp, i32, i32, i32]
    lib.bia_prefill_bounded_workspace_size.restype = sz
    lib.bia_decode_paged_bounded.argtypes = [dp, bp, vp, vp, vp, i64, vp, vp, vp, i32, i32, vp,
                                             sz, vp, vp, vp]
    lib.bia_decode_paged_bounded.restype = ctypes.c_int
    lib.bia_decode_bounded_workspace_size.argtypes = [dp, bp, i32, i32]
    lib.bia_decode_bounded_workspace_size.restype = sz
    lib.bia_append_paged_kv_fp8.argtypes = [dp, vp, vp, i64, i64, vp, vp, vp, vp, i64, vp, vp, vp,
                                            vp, vp, vp, vp, i32, vp, vp]
    lib.bia_append_paged_kv_fp8.restype = ctypes.c_int
    lib.bia_gather_paged_kv_fp8.argtypes = [dp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp,
                                            i32, vp, vp, vp, vp]
    lib.bia_gather_paged_kv_fp8.restype = ctypes.c_int
    lib.bia_decode_paged_fp8.argtypes = [dp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32,
                                         i32, vp, sz, vp, vp, vp]
    lib.bia_decode_paged_fp8.restype = ctypes.c_int
    lib.bia_decode_fp8_workspace_size.argtypes = [dp, vp, vp, i32, i32]
    lib.bia_decode_fp8_workspace_size.restype = sz
    lib.bia_decode_paged_fp8_bounded.argtypes = [dp, bp, vp, vp, vp, vp, vp, i64, vp, vp, vp, i32,
                                                 i32, vp, sz, vp, vp, vp]
    lib.bia_decode_paged_fp8_bounded.restype = ctypes.c_int
    lib.bia_decode_fp8_bounded_workspace_size.argtypes = [dp, bp, i32, i32]
    lib.bia_decode_fp8_bounded_workspace_size.restype = sz
    lib.bia_prefill_ragged.argtypes = [dp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, i32, i32,
                                       i32, vp, sz, vp, vp, vp]
    lib.bia_prefill_ragged.restype = ctypes.c_int
    lib.bia_prefill_ragged_workspace_size.argtypes = [dp, vp, vp, i32, i32, i32]
    lib.bia_prefill_ragged_workspace_size.restype = sz
    lib.bia_decode_paged_window.argtypes = [dp, i32, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32,
                                            i32, vp, sz, vp, vp, vp]
    lib.bia_decode_paged_window.restype = ctypes.c_int
    lib.bia_decode_window_workspace_size.argtypes = [dp, i32, i32, vp, vp, i32, i32]
    lib.bia_decode_window_workspace_size.restype = sz
    lib.bia_decode_paged_window_bounded.argtypes = [dp, bp, i32, i32, vp, vp, vp, i64, vp, vp, vp,
                                                    i32, i32, vp, sz, vp, vp, vp]
    lib.bia_decode_paged_window_bounded.restype = ctypes.c_int
    lib.bia_decode_window_bounded_workspace_size.argtypes = [dp, bp, i32, i32, i32, i32]
    lib.bia_decode_window_bounded_workspace_size.restype = sz
    lib.bia_prefill_paged_window.argtypes = [dp, i32, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp,
                                             vp, i32, i32, vp, sz, vp, vp, vp]
    lib.bia_prefill_paged_window.restype = ctypes.c_int
    lib.bia_prefill_window_workspace_size.argtypes = [dp, i32, i32, vp, vp, vp, i32, i32]
    lib.bia_prefill_window_workspace_size.restype = sz
    rp = ctypes.POINTER(Rope)
    lib.bia_norm_rope.argtypes = [dp, rp, vp, vp, vp, vp, i64, i64, vp, vp, i64, vp, vp, i64, i64,
                                  vp, vp]
    lib.bia_norm_rope.restype = ctypes.c_int
    rows = [dp, rp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    table = [i64, vp, vp, vp, vp, vp, vp, vp, i32]
    lib.bia_append_paged_kv_rope.argtypes = rows + [vp, vp] + table + [vp, i64, vp, vp]
    lib.bia_append_paged_kv_rope.restype = ctypes.c_int
    lib.bia_append_paged_kv_fp8_rope.argtypes = (rows + [vp, vp, vp, vp] + table +
                                                 [vp, vp, i64, i64, vp, vp])
    lib.bia_append_paged_kv_fp8_rope.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu  # the 8-bit cache's codes and scales


# The library sees only the addresses of the device tensors: a host tensor, a
# strided view or a tensor of another dtype would be read as a dense device
# array of the stated type.  So every call checks its tensors first: dtype and
# layout (_check_types), the shapes the sizes it passes are taken from, and
# last that all of them live on one CUDA device (_check_cuda).


def _check_types(*specs):
    """Each spec is (name, tensor, dtype[, optional]): dtype None takes any
    dtype (a byte buffer); an optional argument may be None.  Returns the
    (name, tensor) pairs that were given."""
    given = []
    for spec in specs:
        name, t, dtype = spec[:3]
        if t is None:
            if len(spec) > 3 and spec[3]:
                continue
            raise TypeError(f"{name} is required")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        given.append((name, t))
    return given


def _launch_device(stream) -> torch.device:
    """The device the library enqueues on: a torch stream's own device, else
    the current one (a raw cudaStream_t handle is taken to belong to it)."""
    dev = getattr(stream, "device", None)
    if isinstance(dev, torch.device) and dev.type == "cuda":
        return torch.device("cuda", dev.index if dev.index is not None else
                            torch.cuda.current_device())
    return torch.device("cuda", torch.cuda.current_device())


def _check_cuda(given, stream=None):
    device = None
    for name, t in given:
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")
    if device is not None:
        want = _launch_device(stream)
        have = torch.device("cuda", device.index if device.index is not None else want.index)
        if have != want:
            raise ValueError(f"the tensors are on {have} but the work would run on {want}")


def _check_rows(q, out, lse, qname="q"):
    """out has q's shape; lse, when given, one float per (token, head) of q."""
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out has shape {tuple(out.shape)}, {qname} {tuple(q.shape)}")
    if lse is not None and (q.dim() < 2 or lse.numel() != q.shape[0] * q.shape[1]):
        raise ValueError(f"lse must hold {qname}.shape[0] x {qname}.shape[1] floats")


def _check_caches(k_cache, v_cache):
    if tuple(v_cache.shape) != tuple(k_cache.shape) or k_cache.dim() != 4:
        raise ValueError(f"k_cache and v_cache must both be [num_pages, page_size, "
                         f"num_kv_heads, head_dim], got {tuple(k_cache.shape)} and "
                         f"{tuple(v_cache.shape)}")


def _host_i32(t) -> torch.Tensor:
    t = torch.as_tensor(t, dtype=torch.int32)
    if t.device.type != "cpu":
        raise ValueError("host mirrors must be CPU tensors")
    return t.contiguous()


def _int32(name, x) -> int:
    """x as a 32-bit argument; ctypes would cut a wider one to its low bits."""
    x = int(x)
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_desc(num_qo_heads, num_kv_heads, head_dim, page_size, sm_scale=0.0) -> AttnDesc:
    return AttnDesc(num_qo_heads, num_kv_heads, head_dim, page_size, float(sm_scale))


def status_string(status: int) -> str:
    return load().bia_status_string(int(status)).decode()


def bia_q_tile_tokens(gqa_group: int) -> int:
    return int(load().bia_q_tile_tokens(int(gqa_group)))


def bia_prefill_workspace_size(desc, qo_indptr_host, kv_indptr_host, kv_last_page_len_host,
                               causal=True, split_size=0) -> int:
    qo, kvp, last = (_host_i32(qo_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    return int(load().bia_prefill_workspace_size(ctypes.byref(desc), _ptr(qo), _ptr(kvp),
                                                 _ptr(last), len(qo) - 1, int(bool(causal)),
                                                 int(split_size)))


def bia_decode_workspace_size(desc, kv_indptr_host, kv_last_page_len_host, split_size=0) -> int:
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    return int(load().bia_decode_workspace_size(ctypes.byref(desc), _ptr(kvp), _ptr(last),
                                                len(kvp) - 1, int(split_size)))


def bia_prefill_paged(desc, q, k_cache, v_cache, qo_indptr, kv_indptr, kv_indices,
                      kv_last_page_len, qo_indptr_host, kv_indptr_host, kv_last_page_len_host,
                      workspace, out, lse=None, causal=True, split_size=0, stream=None):
    ts = _check_types(("q", q, BF16), ("k_cache", k_cache, BF16), ("v_cache", v_cache, BF16),
                      ("qo_indptr", qo_indptr, I32), ("kv_indptr", kv_indptr, I32),
                      ("kv_indices", kv_indices, I32), ("kv_last_page_len", kv_last_page_len, I32),
                      ("workspace", workspace, None), ("out", out, BF16), ("lse", lse, F32, True))
    _check_caches(k_cache, v_cache)
    _check_rows(q, out, lse)
    _check_cuda(ts, stream)
    qo, kvp, last = (_host_i32(qo_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    rc = load().bia_prefill_paged(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(qo_indptr), _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len), _ptr(qo),
        _ptr(kvp), _ptr(last), len(qo) - 1, int(bool(causal)), int(split_size), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_prefill_paged")


def bia_prefill_paged_mask(desc, q, k_cache, v_cache, qo_indptr, kv_indptr, kv_indices,
                           kv_last_page_len, qo_indptr_host, kv_indptr_host,
                           kv_last_page_len_host, mask, mask_indptr, mask_indptr_host,
                           workspace, out, lse=None, causal=True, split_size=0, stream=None):
    """bia_prefill_paged with a custom mask: ``mask`` a device uint8 tensor of
    little-endian bits, ``mask_indptr`` its device int64 [batch+1] bit
    offsets (include/bia.h states the rule)."""
    ts = _check_types(("q", q, BF16), ("k_cache", k_cache, BF16), ("v_cache", v_cache, BF16),
                      ("qo_indptr", qo_indptr, I32), ("kv_indptr", kv_indptr, I32),
                      ("kv_indices", kv_indices, I32), ("kv_last_page_len", kv_last_page_len, I32),
                      ("mask", mask, U8), ("mask_indptr", mask_indptr, I64),
                      ("workspace", workspace, None), ("out", out, BF16), ("lse", lse, F32, True))
    _check_caches(k_cache, v_cache)
    _check_rows(q, out, lse)
    _check_cuda(ts, stream)
    qo, kvp, last = (_host_i32(qo_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    mih = torch.as_tensor(mask_indptr_host, dtype=torch.int64).contiguous()
    if mih.device.type != "cpu":
        raise ValueError("host mirrors must be CPU tensors")
    rc = load().bia_prefill_paged_mask(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(qo_indptr), _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len), _ptr(qo),
        _ptr(kvp), _ptr(last), len(qo) - 1, int(bool(causal)), int(split_size), _ptr(mask),
        mask.numel() * mask.element_size(), _ptr(mask_indptr), _ptr(mih), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_prefill_paged_mask")


def bia_decode_paged(desc, q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len,
                     kv_indptr_host, kv_last_page_len_host, workspace, out, lse=None,
                     split_size=0, stream=None):
    ts = _check_types(("q", q, BF16), ("k_cache", k_cache, BF16), ("v_cache", v_cache, BF16),
                      ("kv_indptr", kv_indptr, I32), ("kv_indices", kv_indices, I32),
                      ("kv_last_page_len", kv_last_page_len, I32), ("workspace", workspace, None),
                      ("out", out, BF16), ("lse", lse, F32, True))
    _check_caches(k_cache, v_cache)
    _check_rows(q, out, lse)
    _check_cuda(ts, stream)
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    rc = load().bia_decode_paged(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len), _ptr(kvp), _ptr(last),
        len(kvp) - 1, int(split_size), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_decode_paged")


def make_bounds(max_q_len=1, max_kv_len=1, max_total_q=0) -> Bounds:
    return Bounds(int(max_q_len), int(max_kv_len), int(max_total_q))


def bia_prefill_bounded_workspace_size(desc, bounds, batch, causal=True, split_size=0) -> int:
    return int(load().bia_prefill_bounded_workspace_size(ctypes.byref(desc), ctypes.byref(bounds),
                                                         int(batch), int(bool(causal)),
                                                         int(split_size)))


def bia_decode_bounded_workspace_size(desc, bounds, batch, split_size=0) -> int:
    return int(load().bia_decode_bounded_workspace_size(ctypes.byref(desc), ctypes.byref(bounds),
                                                        int(batch), int(split_size)))


def bia_prefill_paged_bounded(desc, bounds, q, k_cache, v_cache, qo_indptr, kv_indptr,
                              kv_indices, kv_last_page_len, workspace, out, lse=None,
                              causal=True, split_size=0, stream=None):
    """bia_prefill_paged sized from `bounds` (a Bounds): the index arrays are
    read on the device only, so a captured call replays while they change.
    q / out / lse hold bounds.max_total_q token rows."""
    ts = _check_types(("q", q, BF16), ("k_cache", k_cache, BF16), ("v_cache", v_cache, BF16),
                      ("qo_indptr", qo_indptr, I32), ("kv_indptr", kv_indptr, I32),
                      ("kv_indices", kv_indices, I32), ("kv_last_page_len", kv_last_page_len, I32),
                      ("workspace", workspace, None), ("out", out, BF16), ("lse", lse, F32, True))
    _check_caches(k_cache, v_cache)
    _check_rows(q, out, lse)
    if q.shape[0] < bounds.max_total_q:
        raise ValueError(f"q holds {q.shape[0]} token rows, bounds.max_total_q is "
                         f"{bounds.max_total_q}")
    _check_cuda(ts, stream)
    rc = load().bia_prefill_paged_bounded(
        ctypes.byref(desc), ctypes.byref(bounds), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], _ptr(qo_indptr), _ptr(kv_indptr), _ptr(kv_indices),
        _ptr(kv_last_page_len), qo_indptr.numel() - 1, int(bool(causal)), int(split_size),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
        _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_prefill_paged_bounded")


def bia_decode_paged_bounded(desc, bounds, q, k_cache, v_cache, kv_indptr, kv_indices,
                             kv_last_page_len, workspace, out, lse=None, split_size=0,
                             stream=None):
    """bia_decode_paged sized from `bounds` (max_kv_len): the index arrays are
    read on the device only, so a captured decode replays step after step."""
    ts = _check_types(("q", q, BF16), ("k_cache", k_cache, BF16), ("v_cache", v_cache, BF16),
                      ("kv_indptr", kv_indptr, I32), ("kv_indices", kv_indices, I32),
                      ("kv_last_page_len", kv_last_page_len, I32), ("workspace", workspace, None),
                      ("out", out, BF16), ("lse", lse, F32, True))
    _check_caches(k_cache, v_cache)
    _check_rows(q, out, lse)
    if q.shape[0] != kv_indptr.numel() - 1:
        raise ValueError(f"q holds {q.shape[0]} rows for {kv_indptr.numel() - 1} requests")
    _check_cuda(ts, stream)
    rc = load().bia_decode_paged_bounded(
        ctypes.byref(desc), ctypes.byref(bounds), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len),
        kv_indptr.numel() - 1, int(split_size), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_decode_paged_bounded")


BIA_DECODE_NOALLOC_SCRATCH_BYTES = 64 << 20


def bia_decode_paged_noalloc(desc, q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len,
                             kv_indptr_host, kv_last_page_len_host, out, lse=None, split_size=0,
                             stream=None):
    """bia_decode_paged for callers that cannot allocate device memory: no
    workspace argument; the library's static scratch array is used instead
    (see include/bia.h for its size, first-call and concurrency rules)."""
    ts = _check_types(("q", q, BF16), ("k_cache", k_cache, BF16), ("v_cache", v_cache, BF16),
                      ("kv_indptr", kv_indptr, I32), ("kv_indices", kv_indices, I32),
                      ("kv_last_page_len", kv_last_page_len, I32), ("out", out, BF16),
                      ("lse", lse, F32, True))
    _check_caches(k_cache, v_cache)
    _check_rows(q, out, lse)
    _check_cuda(ts, stream)
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    rc = load().bia_decode_paged_noalloc(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len), _ptr(kvp), _ptr(last),
        len(kvp) - 1, int(split_size), _ptr(out), _ptr(lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_decode_paged_noalloc")


def bia_append_paged_kv(desc, k_new, v_new, k_cache, v_cache, append_indptr, kv_indptr,
                        kv_indices, kv_last_page_len, append_indptr_host, kv_indptr_host,
                        kv_last_page_len_host, status=None, stream=None):
    """Write the new tokens' K/V rows [total_new, Hkv, D] into the last
    n_new positions of each request's pages (include/bia.h states the rule);
    `status` is an optional 1-element device int32 tensor."""
    ts = _check_types(("k_new", k_new, BF16), ("v_new", v_new, BF16), ("k_cache", k_cache, BF16),
                      ("v_cache", v_cache, BF16), ("append_indptr", append_indptr, I32),
                      ("kv_indptr", kv_indptr, I32), ("kv_indices", kv_indices, I32),
                      ("kv_last_page_len", kv_last_page_len, I32), ("status", status, I32, True))
    _check_caches(k_cache, v_cache)
    if tuple(v_new.shape) != tuple(k_new.shape):
        raise ValueError(f"v_new has shape {tuple(v_new.shape)}, k_new {tuple(k_new.shape)}")
    _check_cuda(ts, stream)
    ap, kvp, last = (_host_i32(append_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    rc = load().bia_append_paged_kv(
        ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], _ptr(append_indptr), _ptr(kv_indptr), _ptr(kv_indices),
        _ptr(kv_last_page_len), _ptr(ap), _ptr(kvp), _ptr(last), len(ap) - 1, _ptr(status),
        _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_append_paged_kv")


def bia_merge_states(v, s, out, out_lse=None, num_states=None, stream=None):
    """v [n, S, H, D] fp32, s [n, S, H] fp32 -> out [n, H, D] bf16, out_lse [n, H]."""
    ts = _check_types(("v", v, F32), ("s", s, F32), ("out", out, BF16),
                      ("out_lse", out_lse, F32, True), ("num_states", num_states, I32, True))
    if v.dim() != 4:
        raise ValueError(f"v must be [n, S, H, D], got shape {tuple(v.shape)}")
    n, S, H, D = v.shape
    if tuple(s.shape) != (n, S, H) or tuple(out.shape) != (n, H, D):
        raise ValueError(f"s must be {(n, S, H)} and out {(n, H, D)}, got "
                         f"{tuple(s.shape)} and {tuple(out.shape)}")
    if out_lse is not None and tuple(out_lse.shape) != (n, H):
        raise ValueError(f"out_lse must be {(n, H)}, got {tuple(out_lse.shape)}")
    if num_states is not None and num_states.numel() != n:
        raise ValueError(f"num_states must hold {n} counts, got {num_states.numel()}")
    _check_cuda(ts, stream)
    rc = load().bia_merge_states(_ptr(v), _ptr(s), _ptr(num_states), n, S, H, D, _ptr(out),
                                 _ptr(out_lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_merge_states")


def bia_read_status(workspace, stream=None) -> int:
    ts = _check_types(("workspace", workspace, None))
    _check_cuda(ts, stream)
    st = ctypes.c_int32(0)
    rc = load().bia_read_status(_ptr(workspace), ctypes.byref(st), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_read_status")
    return int(st.value)


def bia_set_profile_events(begin=None, end=None):
    """Record torch.cuda.Event `begin` / `end` (created with enable_timing)
    around the attention kernel of every later prefill / decode call
    (None, None: off)."""
    def handle(e):
        if e is None:
            return None
        if not e.cuda_event:  # torch creates the CUDA event on first record
            e.record()
        return ctypes.c_void_p(e.cuda_event)
    load().bia_set_profile_events(handle(begin), handle(end))


def bia_launch_count() -> int:
    return int(load().bia_launch_count())


def make_mla_desc(num_heads, page_size, sm_scale=0.0) -> MlaDesc:
    return MlaDesc(num_heads, page_size, float(sm_scale))


def bia_mla_decode_workspace_size(desc, kv_indptr_host, kv_last_page_len_host,
                                  split_size=0) -> int:
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    return int(load().bia_mla_decode_workspace_size(ctypes.byref(desc), _ptr(kvp), _ptr(last),
                                                    len(kvp) - 1, int(split_size)))


def bia_mla_decode_paged(desc, q_nope, q_pe, ckv_cache, kpe_cache, kv_indptr, kv_indices,
                         kv_last_page_len, kv_indptr_host, kv_last_page_len_host, workspace,
                         out, lse=None, split_size=0, stream=None):
    """Multi-head latent attention decode (include/bia.h states the layouts)."""
    ts = _check_types(("q_nope", q_nope, BF16), ("q_pe", q_pe, BF16), ("ckv_cache", ckv_cache, BF16),
                      ("kpe_cache", kpe_cache, BF16), ("kv_indptr", kv_indptr, I32),
                      ("kv_indices", kv_indices, I32), ("kv_last_page_len", kv_last_page_len, I32),
                      ("workspace", workspace, None), ("out", out, BF16), ("lse", lse, F32, True))
    if kpe_cache.dim() < 1 or ckv_cache.dim() < 1 or kpe_cache.shape[0] != ckv_cache.shape[0]:
        raise ValueError("ckv_cache and kpe_cache must have the same number of pages")
    _check_rows(q_nope, out, lse, "q_nope")
    _check_cuda(ts, stream)
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    rc = load().bia_mla_decode_paged(
        ctypes.byref(desc), _ptr(q_nope), _ptr(q_pe), _ptr(ckv_cache), _ptr(kpe_cache),
        ckv_cache.shape[0], _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len),
        _ptr(kvp), _ptr(last), len(kvp) - 1, int(split_size), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_mla_decode_paged")


def bia_mla_prefill_workspace_size(desc, qo_indptr_host, kv_indptr_host, kv_last_page_len_host,
                                   split_size=0) -> int:
    qo, kvp, last = (_host_i32(qo_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    return int(load().bia_mla_prefill_workspace_size(ctypes.byref(desc), _ptr(qo), _ptr(kvp),
                                                     _ptr(last), len(qo) - 1, int(split_size)))


def bia_mla_prefill_paged(desc, q_nope, q_pe, ckv_cache, kpe_cache, qo_indptr, kv_indptr,
                          kv_indices, kv_last_page_len, qo_indptr_host, kv_indptr_host,
                          kv_last_page_len_host, workspace, out, lse=None, split_size=0,
                          stream=None):
    """Causal multi-head latent attention extend: q_nope / q_pe / out hold
    total_q token rows (include/bia.h states the layouts and the rule)."""
    ts = _check_types(("q_nope", q_nope, BF16), ("q_pe", q_pe, BF16),
                      ("ckv_cache", ckv_cache, BF16), ("kpe_cache", kpe_cache, BF16),
                      ("qo_indptr", qo_indptr, I32), ("kv_indptr", kv_indptr, I32),
                      ("kv_indices", kv_indices, I32), ("kv_last_page_len", kv_last_page_len, I32),
                      ("workspace", workspace, None), ("out", out, BF16), ("lse", lse, F32, True))
    if kpe_cache.dim() < 1 or ckv_cache.dim() < 1 or kpe_cache.shape[0] != ckv_cache.shape[0]:
        raise ValueError("ckv_cache and kpe_cache must have the same number of pages")
    _check_rows(q_nope, out, lse, "q_nope")
    _check_cuda(ts, stream)
    qo, kvp, last = (_host_i32(qo_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    rc = load().bia_mla_prefill_paged(
        ctypes.byref(desc), _ptr(q_nope), _ptr(q_pe), _ptr(ckv_cache), _ptr(kpe_cache),
        ckv_cache.shape[0], _ptr(qo_indptr), _ptr(kv_indptr), _ptr(kv_indices),
        _ptr(kv_last_page_len), _ptr(qo), _ptr(kvp), _ptr(last), len(qo) - 1, int(split_size),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
        _stream(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_mla_prefill_paged")


# ---------------------------------------------------------------- 8-bit cache
#
# These calls are made once per layer and decode step, so what a well-formed
# call pays on the host counts (a 32-token append's kernel takes about 5 us):
# _dense looks the tensors over, and only a call that fails it goes through
# the checks that find the reason.

_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _index(t) -> int:
    """CUDA device index of a tensor, -1 of anything else."""
    return t.get_device() if type(t) is torch.Tensor else -1


def _dense(device, dtype, *tensors) -> bool:
    """Whether all are contiguous tensors of `dtype` on CUDA device `device`."""
    for t in tensors:
        if (type(t) is not torch.Tensor or t.dtype is not dtype or t.get_device() != device or
                not t.is_contiguous()):
            return False
    return True


def _handle(stream):
    """The raw handle of `stream`, or of the current device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _at(t):
    """Address of a tensor (ctypes takes it as a void pointer), None of none."""
    return None if t is None else t.data_ptr()


def _last(t) -> int:
    """Last entry of a host mirror."""
    return ctypes.c_int32.from_address(t.data_ptr() + 4 * (t.numel() - 1)).value


def _host(t) -> torch.Tensor:
    """_host_i32 with at least one entry."""
    if not (isinstance(t, torch.Tensor) and t.dtype is I32 and t.is_contiguous() and
            t.get_device() < 0):
        t = _host_i32(t)
    if t.numel() == 0:
        raise ValueError("host mirrors hold at least one entry")
    return t


def _check_caches_fp8(desc, k_cache, v_cache, k_scale, v_scale):
    rows = (k_cache.shape[0], desc.page_size, desc.num_kv_heads)
    want = rows + (desc.head_dim,)
    if k_cache.shape != want or v_cache.shape != want:
        raise ValueError(f"k_cache and v_cache must be {want} (num_pages, page_size, "
                         f"num_kv_heads, head_dim) for this descriptor, got "
                         f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    if k_scale.shape != rows or v_scale.shape != rows:
        raise ValueError(f"k_scale and v_scale must be {rows}, got {tuple(k_scale.shape)} and "
                         f"{tuple(v_scale.shape)}")


def _check_table(batch, kv_indptr, kv_indices, kv_last_page_len, kvp=None, last=None):
    """The page table's arrays hold what a call of `batch` requests reads."""
    if (kv_indptr.numel() == batch + 1 and kv_last_page_len.numel() == batch and
            (kvp is None or (kvp.numel() == batch + 1 and last.numel() == batch and
                             kv_indices.numel() >= _last(kvp)))):
        return
    for name, t, want in (("kv_indptr", kv_indptr, batch + 1),
                          ("kv_last_page_len", kv_last_page_len, batch),
                          ("kv_indptr_host", kvp, batch + 1),
                          ("kv_last_page_len_host", last, batch)):
        if t is not None and t.numel() != want:
            raise ValueError(f"{name} must hold {want} entries for {batch} requests, got "
                             f"{t.numel()}")
    if kvp is not None and kv_indices.numel() < _last(kvp):
        raise ValueError(f"kv_indices holds {kv_indices.numel()} pages, kv_indptr ends at "
                         f"{_last(kvp)}")


def _packed(name, t, heads, head_dim, tokens):
    """Token stride of packed bf16 rows [tokens, heads, head_dim]: a token's
    heads and columns dense, any multiple of 8 elements from one token to the
    next, on the device of the contiguous tensors (checked by the caller)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not BF16:
        raise TypeError(f"{name} must be {BF16}, got {t.dtype}")
    if t.shape != (tokens, heads, head_dim):
        raise ValueError(f"{name} must be [{tokens} tokens, {heads}, {head_dim}], got "
                         f"{tuple(t.shape)}")
    row = heads * head_dim
    if tokens == 0:
        return row
    step, head, col = t.stride()
    if (head_dim > 1 and col != 1) or (heads > 1 and head != head_dim):
        raise ValueError(f"{name} must hold each token's heads one after the other, got strides "
                         f"{t.stride()}")
    if tokens == 1:
        return row
    if step < row or step % 8 != 0:
        raise ValueError(f"{name} must step a multiple of 8 elements, at least {row}, from token "
                         f"to token, got {step}")
    return step


def bia_append_paged_kv_fp8(desc, k_new, v_new, k_cache, v_cache, k_scale, v_scale, append_indptr,
                            kv_indptr, kv_indices, kv_last_page_len, append_indptr_host,
                            kv_indptr_host, kv_last_page_len_host, status=None, stream=None):
    """bia_append_paged_kv into the 8-bit cache: codes torch.float8_e4m3fn
    [num_pages, page_size, Hkv, D], scales torch.float8_e8m0fnu [num_pages,
    page_size, Hkv] (include/bia.h states the format).  k_new and v_new
    [total_new, Hkv, D] may be slices of a fused projection's rows."""
    ap, kvp, last = (_host(append_indptr_host), _host(kv_indptr_host),
                     _host(kv_last_page_len_host))
    batch = ap.numel() - 1
    total, hkv, d = _last(ap), desc.num_kv_heads, desc.head_dim
    k_step = _packed("k_new", k_new, hkv, d, total)
    v_step = _packed("v_new", v_new, hkv, d, total)
    at, ts = _index(k_cache), None
    if not (stream is None and _dense(at, E4M3, k_cache, v_cache) and
            _dense(at, E8M0, k_scale, v_scale) and
            _dense(at, I32, append_indptr, kv_indptr, kv_indices, kv_last_page_len) and
            (status is None or _dense(at, I32, status)) and at >= 0 and
            at == _current_device()):
        ts = _check_types(("k_cache", k_cache, E4M3), ("v_cache", v_cache, E4M3),
                          ("k_scale", k_scale, E8M0), ("v_scale", v_scale, E8M0),
                          ("append_indptr", append_indptr, I32), ("kv_indptr", kv_indptr, I32),
                          ("kv_indices", kv_indices, I32),
                          ("kv_last_page_len", kv_last_page_len, I32),
                          ("status", status, I32, True))
    _check_caches_fp8(desc, k_cache, v_cache, k_scale, v_scale)
    _check_table(batch, kv_indptr, kv_indices, kv_last_page_len, kvp, last)
    if append_indptr.numel() != batch + 1:
        raise ValueError(f"append_indptr must hold {batch + 1} entries, got "
                         f"{append_indptr.numel()}")
    if ts is not None or k_new.get_device() != at or v_new.get_device() != at:
        _check_cuda((ts or [("k_cache", k_cache)]) + [("k_new", k_new), ("v_new", v_new)], stream)
    rc = load().bia_append_paged_kv_fp8(
        ctypes.byref(desc), k_new.data_ptr(), v_new.data_ptr(), k_step, v_step, k_cache.data_ptr(),
        v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_cache.shape[0],
        append_indptr.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(),
        kv_last_page_len.data_ptr(), ap.data_ptr(), kvp.data_ptr(), last.data_ptr(), batch,
        _at(status), _handle(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_append_paged_kv_fp8")


def bia_gather_paged_kv_fp8(desc, k_cache, v_cache, k_scale, v_scale, k_out, v_out, out_indptr,
                            kv_indptr, kv_indices, kv_last_page_len, out_indptr_host,
                            kv_indptr_host, kv_last_page_len_host, status=None, stream=None):
    """Reads the first out_indptr[b+1] - out_indptr[b] keys of each request
    back from the 8-bit cache into k_out / v_out [out_indptr[batch], Hkv, D]
    bf16, packed (include/bia.h states the rule)."""
    at, ts = _index(k_cache), None
    if not (stream is None and _dense(at, E4M3, k_cache, v_cache) and
            _dense(at, E8M0, k_scale, v_scale) and _dense(at, BF16, k_out, v_out) and
            _dense(at, I32, out_indptr, kv_indptr, kv_indices, kv_last_page_len) and
            (status is None or _dense(at, I32, status)) and at >= 0 and
            at == _current_device()):
        ts = _check_types(("k_cache", k_cache, E4M3), ("v_cache", v_cache, E4M3),
                          ("k_scale", k_scale, E8M0), ("v_scale", v_scale, E8M0),
                          ("k_out", k_out, BF16), ("v_out", v_out, BF16),
                          ("out_indptr", out_indptr, I32), ("kv_indptr", kv_indptr, I32),
                          ("kv_indices", kv_indices, I32),
                          ("kv_last_page_len", kv_last_page_len, I32),
                          ("status", status, I32, True))
    _check_caches_fp8(desc, k_cache, v_cache, k_scale, v_scale)
    op, kvp, last = _host(out_indptr_host), _host(kv_indptr_host), _host(kv_last_page_len_host)
    batch = op.numel() - 1
    _check_table(batch, kv_indptr, kv_indices, kv_last_page_len, kvp, last)
    if out_indptr.numel() != batch + 1:
        raise ValueError(f"out_indptr must hold {batch + 1} entries, got {out_indptr.numel()}")
    want = (_last(op), desc.num_kv_heads, desc.head_dim)
    if k_out.shape != want or v_out.shape != want:
        raise ValueError(f"k_out and v_out must be {want}, got {tuple(k_out.shape)} and "
                         f"{tuple(v_out.shape)}")
    if ts is not None:
        _check_cuda(ts, stream)
    rc = load().bia_gather_paged_kv_fp8(
        ctypes.byref(desc), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), k_cache.shape[0], out_indptr.data_ptr(), kv_indptr.data_ptr(),
        kv_indices.data_ptr(), kv_last_page_len.data_ptr(), op.data_ptr(), kvp.data_ptr(),
        last.data_ptr(), batch, k_out.data_ptr(), v_out.data_ptr(), _at(status), _handle(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_gather_paged_kv_fp8")


def bia_decode_fp8_workspace_size(desc, kv_indptr_host, kv_last_page_len_host,
                                  split_size=0) -> int:
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    return int(load().bia_decode_fp8_workspace_size(ctypes.byref(desc), _ptr(kvp), _ptr(last),
                                                    len(kvp) - 1, int(split_size)))


def _check_decode_fp8(desc, q, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                      kv_last_page_len, workspace, out, lse, stream, kvp=None, last=None):
    at, ts = _index(q), None
    if not (stream is None and _dense(at, BF16, q, out) and _dense(at, E4M3, k_cache, v_cache) and
            _dense(at, E8M0, k_scale, v_scale) and
            _dense(at, I32, kv_indptr, kv_indices, kv_last_page_len) and
            (lse is None or _dense(at, F32, lse)) and at >= 0 and
            _index(workspace) == at == _current_device() and workspace.is_contiguous()):
        ts = _check_types(("q", q, BF16), ("k_cache", k_cache, E4M3),
                          ("v_cache", v_cache, E4M3), ("k_scale", k_scale, E8M0),
                          ("v_scale", v_scale, E8M0), ("kv_indptr", kv_indptr, I32),
                          ("kv_indices", kv_indices, I32),
                          ("kv_last_page_len", kv_last_page_len, I32),
                          ("workspace", workspace, None), ("out", out, BF16),
                          ("lse", lse, F32, True))
    _check_caches_fp8(desc, k_cache, v_cache, k_scale, v_scale)
    want = (kv_indptr.numel() - 1, desc.num_qo_heads, desc.head_dim)
    if q.shape != want or out.shape != want:
        raise ValueError(f"q and out must be {want}, got {tuple(q.shape)} and {tuple(out.shape)}")
    if lse is not None and lse.numel() != want[0] * want[1]:
        raise ValueError(f"lse must hold {want[0]} x {want[1]} floats")
    _check_table(want[0], kv_indptr, kv_indices, kv_last_page_len, kvp, last)
    if ts is not None:
        _check_cuda(ts, stream)


def bia_decode_paged_fp8(desc, q, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                         kv_last_page_len, kv_indptr_host, kv_last_page_len_host, workspace, out,
                         lse=None, split_size=0, stream=None):
    """bia_decode_paged over the 8-bit cache (include/bia.h states the format)."""
    kvp, last = _host(kv_indptr_host), _host(kv_last_page_len_host)
    _check_decode_fp8(desc, q, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                      kv_last_page_len, workspace, out, lse, stream, kvp, last)
    batch = q.shape[0]
    rc = load().bia_decode_paged_fp8(
        ctypes.byref(desc), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), k_cache.shape[0], kv_indptr.data_ptr(),
        kv_indices.data_ptr(), kv_last_page_len.data_ptr(), kvp.data_ptr(), last.data_ptr(), batch,
        int(split_size), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        out.data_ptr(), _at(lse), _handle(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_decode_paged_fp8")


def bia_decode_fp8_bounded_workspace_size(desc, bounds, batch, split_size=0) -> int:
    return int(load().bia_decode_fp8_bounded_workspace_size(
        ctypes.byref(desc), ctypes.byref(bounds), int(batch), int(split_size)))


def bia_decode_paged_fp8_bounded(desc, bounds, q, k_cache, v_cache, k_scale, v_scale, kv_indptr,
                                 kv_indices, kv_last_page_len, workspace, out, lse=None,
                                 split_size=0, stream=None):
    """bia_decode_paged_fp8 sized from `bounds` (max_kv_len): the index arrays
    are read on the device only, so a captured decode replays step after step."""
    _check_decode_fp8(desc, q, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                      kv_last_page_len, workspace, out, lse, stream)
    batch = q.shape[0]
    rc = load().bia_decode_paged_fp8_bounded(
        ctypes.byref(desc), ctypes.byref(bounds), q.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_cache.shape[0],
        kv_indptr.data_ptr(), kv_indices.data_ptr(), kv_last_page_len.data_ptr(), batch,
        int(split_size), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        out.data_ptr(), _at(lse), _handle(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_decode_paged_fp8_bounded")


# ---------------------------------------------------------------- packed prompts


def bia_prefill_ragged_workspace_size(desc, qo_indptr_host, kv_indptr_host, causal=True,
                                      split_size=0) -> int:
    qo, kvp = _host_i32(qo_indptr_host), _host_i32(kv_indptr_host)
    return int(load().bia_prefill_ragged_workspace_size(ctypes.byref(desc), _ptr(qo), _ptr(kvp),
                                                        len(qo) - 1, int(bool(causal)),
                                                        int(split_size)))


def bia_prefill_ragged(desc, q, k, v, qo_indptr, kv_indptr, qo_indptr_host, kv_indptr_host,
                       workspace, out, lse=None, causal=True, split_size=0, stream=None):
    """Attention of packed sequences: q [total_q, Hq, D] over k, v [total_kv,
    Hkv, D], each dense or a slice of a fused projection's rows
    (include/bia.h states the rule)."""
    qo, kvp = _host(qo_indptr_host), _host(kv_indptr_host)
    batch = qo.numel() - 1
    hq, hkv, d = desc.num_qo_heads, desc.num_kv_heads, desc.head_dim
    q_step = _packed("q", q, hq, d, _last(qo))
    k_step = _packed("k", k, hkv, d, _last(kvp))
    v_step = _packed("v", v, hkv, d, _last(kvp))
    at, ts = _index(out), None
    if not (stream is None and _dense(at, I32, qo_indptr, kv_indptr) and _dense(at, BF16, out) and
            (lse is None or _dense(at, F32, lse)) and at >= 0 and
            _index(workspace) == at == _current_device() and workspace.is_contiguous()):
        ts = _check_types(("qo_indptr", qo_indptr, I32), ("kv_indptr", kv_indptr, I32),
                          ("workspace", workspace, None), ("out", out, BF16),
                          ("lse", lse, F32, True))
    if out.shape != q.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, q {tuple(q.shape)}")
    if lse is not None and lse.numel() != q.shape[0] * hq:
        raise ValueError(f"lse must hold {q.shape[0]} x {hq} floats")
    for name, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("kv_indptr_host", kvp)):
        if t.numel() != batch + 1:
            raise ValueError(f"{name} must hold {batch + 1} entries, got {t.numel()}")
    if ts is not None or q.get_device() != at or k.get_device() != at or v.get_device() != at:
        _check_cuda((ts or [("out", out)]) + [("q", q), ("k", k), ("v", v)], stream)
    rc = load().bia_prefill_ragged(
        ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), q_step, k_step, v_step,
        qo_indptr.data_ptr(), kv_indptr.data_ptr(), qo.data_ptr(), kvp.data_ptr(), batch,
        int(bool(causal)), int(split_size), workspace.data_ptr(), workspace.numel() *
        workspace.element_size(), out.data_ptr(), _at(lse), _handle(stream))
    if rc != BIA_OK:
        raise BiaError(rc, "bia_prefill_ragged")


# ---------------------------------------------------------------- rotary positions


def make_rope(rot_dim, num_positions, num_axes=1, freq_axis=None, interleaved=False,
              norm_eps=1e-6) -> Rope:
    """The rotation of a model's heads (include/bia.h states the rule):
    freq_axis names the axis of each of the rot_dim / 2 frequencies where there
    are several axes, for example [16 * 0, 24 * 1, 24 * 2] or 0, 1, 2 in turn."""
    r = Rope(_int32("rot_dim", rot_dim), int(bool(interleaved)), _int32("num_axes", num_axes),
             _int32("num_positions", num_positions), float(norm_eps))
    axes = [] if freq_axis is None or num_axes == 1 else list(freq_axis)
    if num_axes > 1 and len(axes) != rot_dim // 2:
        raise ValueError(f"freq_axis must name an axis for each of {rot_dim // 2} frequencies, "
                         f"got {len(axes)}")
    if any(not 0 <= x < num_axes for x in axes):
        raise ValueError(f"freq_axis names axes 0 to {num_axes - 1}")
    if len(axes) <= 128:
        r.freq_axis[:len(axes)] = axes
    return r


def _check_rope(desc, rope, table, positions, q_weight, k_weight, total):
    if table.shape != (rope.num_positions, rope.rot_dim):
        raise ValueError(f"table must be ({rope.num_positions}, {rope.rot_dim}), got "
                         f"{tuple(table.shape)}")
    if positions is not None:
        # with one axis every shape has the same order; with more a transposed one would
        # turn by other tokens' positions
        axes = rope.num_axes
        if positions.numel() != axes * total or (axes > 1 and positions.dim() != 1 and
                                                 positions.shape != (axes, total)):
            raise ValueError(f"positions must be ({axes}, {total}), got {tuple(positions.shape)}")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and w.shape != (desc.head_dim,):
            raise ValueError(f"{name} must be ({desc.head_dim},), got {tuple(w.shape)}")


def _rope_types(table, positions, q_weight, k_weight, status):
    return _check_types(("table", table, F32), ("positions", positions, I32, True),
                        ("q_weight", q_weight, F32, True), ("k_weight", k_weight, F32, True),
                        ("status", status, I32, True))


# The calls below look at a tensor's dtype, layout and shape in as few steps as
# they can and leave its device to the library, which refuses what is not memory
# of the current device before it enqueues anything.  What is not plain (another
# stream, no tokens, a dtype or layout that is wrong), and what the library
# refused, goes through the checks above, which name the argument.


def _step(name, t, heads, head_dim, tokens) -> int:
    """_packed; what is not plain goes there."""
    if isinstance(t, torch.Tensor) and t.dtype is BF16 and tokens > 1 and \
            t.shape == (tokens, heads, head_dim):
        step, head, col = t.stride()
        if col == 1 and (head == head_dim or heads == 1) and step % 8 == 0 and \
                step >= heads * head_dim:
            return step
    return _packed(name, t, heads, head_dim, tokens)


def _check_rope_tensors(given, rows, table, positions, q_weight, k_weight, status, stream):
    """All on one device: `given`, the rotation's tensors, and the packed rows."""
    given = given + _rope_types(table, positions, q_weight, k_weight, status)
    _check_cuda(given, stream)
    for name, t in rows:
        if t is not None and t.device != given[0][1].device:
            raise ValueError(f"{name} is on {t.device}, the other arguments on "
                             f"{given[0][1].device}")


def _plain_rope(table, positions, q_weight, k_weight, status) -> bool:
    return (table.is_cuda and table.dtype is F32 and table.is_contiguous() and
            (positions is None or (positions.dtype is I32 and positions.is_contiguous())) and
            (q_weight is None or (q_weight.dtype is F32 and q_weight.is_contiguous())) and
            (k_weight is None or (k_weight.dtype is F32 and k_weight.is_contiguous())) and
            (status is None or (status.dtype is I32 and status.is_contiguous())))


def bia_norm_rope(desc, rope, table, positions, q, k, q_out, k_out, q_weight=None, k_weight=None,
                  status=None, stream=None):
    """Norms and rotates q [total, Hq, D] and k [total, Hkv, D] into q_out and
    k_out, each dense or a slice of a fused projection's rows, also in place;
    q and q_out, or k and k_out, may be None.  positions [num_axes, total]."""
    some = q if q is not None else k
    if some is None:
        raise TypeError("q or k is required")
    if not isinstance(some, torch.Tensor):
        raise TypeError(f"q and k must be torch.Tensor, got {type(some).__name__}")
    if positions is None:
        raise TypeError("positions is required")
    total = some.shape[0]
    hq, hkv, d = desc.num_qo_heads, desc.num_kv_heads, desc.head_dim
    q_step = qo_step = k_step = ko_step = 0
    if q is not None or q_out is not None:
        q_step = _step("q", q, hq, d, total)
        qo_step = _step("q_out", q_out, hq, d, total)
    if k is not None or k_out is not None:
        k_step = _step("k", k, hkv, d, total)
        ko_step = _step("k_out", k_out, hkv, d, total)

    def check():
        _check_rope_tensors([("q" if q is not None else "k", some)],
                            (("q_out", q_out), ("k", k), ("k_out", k_out)), table, positions,
                            q_weight, k_weight, status, stream)

    try:
        plain = stream is None and total > 0 and _plain_rope(table, positions, q_weight, k_weight,
                                                             status)
    except AttributeError:
        plain = False
    if not plain:
        check()
    _check_rope(desc, rope, table, positions, q_weight, k_weight, total)
    rc = load().bia_norm_rope(
        ctypes.byref(desc), ctypes.byref(rope), table.data_ptr(), positions.data_ptr(), _at(q),
        _at(k), q_step, k_step, _at(q_weight), _at(k_weight), total, _at(q_out), _at(k_out),
        qo_step, ko_step, _at(status), _handle(stream))
    if rc != BIA_OK:
        check()
        raise BiaError(rc, "bia_norm_rope")


def _append_rope(fp8, desc, rope, table, q, k_new, v_new, caches, append_indptr, kv_indptr,
                 kv_indices, kv_last_page_len, append_indptr_host, kv_indptr_host,
                 kv_last_page_len_host, q_out, k_out, positions, q_weight, k_weight, status,
                 stream):
    """The checks of the two appends, and the call."""
    ap, kvp, last = (_host(append_indptr_host), _host(kv_indptr_host),
                     _host(kv_last_page_len_host))
    batch = ap.numel() - 1
    total, hq, hkv, d = _last(ap), desc.num_qo_heads, desc.num_kv_heads, desc.head_dim
    k_cache, v_cache = caches[0], caches[1]
    q_step = qo_step = ko_step = 0
    if q is not None or q_out is not None:
        q_step = _step("q", q, hq, d, total)
        qo_step = _step("q_out", q_out, hq, d, total)
    k_step = _step("k_new", k_new, hkv, d, total)
    v_step = _step("v_new", v_new, hkv, d, total)
    if k_out is not None:
        ko_step = _step("k_out", k_out, hkv, d, total)
    kinds = (E4M3, E4M3, E8M0, E8M0) if fp8 else (BF16, BF16)

    def check():
        ts = _check_types(*zip(("k_cache", "v_cache", "k_scale", "v_scale"), caches, kinds),
                          ("append_indptr", append_indptr, I32), ("kv_indptr", kv_indptr, I32),
                          ("kv_indices", kv_indices, I32),
                          ("kv_last_page_len", kv_last_page_len, I32))
        _check_rope_tensors(ts, (("q", q), ("q_out", q_out), ("k_new", k_new), ("v_new", v_new),
                                 ("k_out", k_out)), table, positions, q_weight, k_weight, status,
                            stream)

    try:
        plain = (stream is None and total > 0 and
                 k_cache.dtype is kinds[0] and k_cache.is_contiguous() and
                 v_cache.dtype is kinds[0] and v_cache.is_contiguous() and
                 (not fp8 or (caches[2].dtype is E8M0 and caches[2].is_contiguous() and
                              caches[3].dtype is E8M0 and caches[3].is_contiguous())) and
                 append_indptr.dtype is I32 and append_indptr.is_contiguous() and
                 kv_indptr.dtype is I32 and kv_indptr.is_contiguous() and
                 kv_indices.dtype is I32 and kv_indices.is_contiguous() and
                 kv_last_page_len.dtype is I32 and kv_last_page_len.is_contiguous() and
                 _plain_rope(table, positions, q_weight, k_weight, status))
    except AttributeError:
        plain = False
    if not plain:
        check()
    if fp8:
        _check_caches_fp8(desc, *caches)
    else:
        want = (k_cache.shape[0], desc.page_size, hkv, d)
        if k_cache.shape != want or v_cache.shape != want:
            raise ValueError(f"k_cache and v_cache must be {want} (num_pages, page_size, "
                             f"num_kv_heads, head_dim) for this descriptor, got "
                             f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    _check_table(batch, kv_indptr, kv_indices, kv_last_page_len, kvp, last)
    if append_indptr.numel() != batch + 1:
        raise ValueError(f"append_indptr must hold {batch + 1} entries, got "
                         f"{append_indptr.numel()}")
    _check_rope(desc, rope, table, positions, q_weight, k_weight, total)
    if fp8:
        name, pages = "bia_append_paged_kv_fp8_rope", [c.data_ptr() for c in caches]
        tail = (_at(q_out), _at(k_out), qo_step, ko_step)
    else:
        name, pages = "bia_append_paged_kv_rope", (k_cache.data_ptr(), v_cache.data_ptr())
        tail = (_at(q_out), qo_step)
    rc = getattr(load(), name)(
        ctypes.byref(desc), ctypes.byref(rope), table.data_ptr(), _at(positions), _at(q),
        k_new.data_ptr(), v_new.data_ptr(), q_step, k_step, v_step, _at(q_weight), _at(k_weight),
        *pages, k_cache.shape[0], append_indptr.data_ptr(), kv_indptr.data_ptr(),
        kv_indices.data_ptr(), kv_last_page_len.data_ptr(), ap.data_ptr(), kvp.data_ptr(),
        last.data_ptr(), batch, *tail, _at(status), _handle(stream))
    if rc != BIA_OK:
        check()
        raise BiaError(rc, name)


def bia_append_paged_kv_rope(desc, rope, table, q, k_new, v_new, k_cache, v_cache, append_indptr,
                             kv_indptr, kv_indices, kv_last_page_len, append_indptr_host,
                             kv_indptr_host, kv_last_page_len_host, q_out, positions=None,
                             q_weight=None, k_weight=None, status=None, stream=None):
    """bia_append_paged_kv with the keys normed and rotated on the way, and the
    queries of the same tokens to q_out (q and q_out may be None).  Without
    positions a token's position is its key's."""
    _append_rope(False, desc, rope, table, q, k_new, v_new, (k_cache, v_cache), append_indptr,
                 kv_indptr, kv_indices, kv_last_page_len, append_indptr_host, kv_indptr_host,
                 kv_last_page_len_host, q_out, None, positions, q_weight, k_weight, status, stream)


def bia_append_paged_kv_fp8_rope(desc, rope, table, q, k_new, v_new, k_cache, v_cache, k_scale,
                                 v_scale, append_indptr, kv_indptr, kv_indices, kv_last_page_len,
                                 append_indptr_host, kv_indptr_host, kv_last_page_len_host, q_out,
                                 k_out=None, positions=None, q_weight=None, k_weight=None,
                                 status=None, stream=None):
    """The same into the 8-bit cache; k_out, when given, takes the rotated keys
    as bf16 rows too."""
    _append_rope(True, desc, rope, table, q, k_new, v_new, (k_cache, v_cache, k_scale, v_scale),
                 append_indptr, kv_indptr, kv_indices, kv_last_page_len, append_indptr_host,
                 kv_indptr_host, kv_last_page_len_host, q_out, k_out, positions, q_weight,
                 k_weight, status, stream)


# ---------------------------------------------------------------- window and sinks


def _window_ints(window, sinks, split_size):
    return _int32("window", window), _int32("sinks", sinks), _int32("split_size", split_size)


def _check_window_tensors(q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len, workspace,
                          out, lse, stream, qo_indptr=None):
    more = () if qo_indptr is None else (("qo_indptr", qo_indptr, I32),)
    _check_cuda(_check_types(("q", q, BF16), ("k_cache", k_cache, BF16),
                             ("v_cache", v_cache, BF16), ("kv_indptr", kv_indptr, I32),
                             ("kv_indices", kv_indices, I32),
                             ("kv_last_page_len", kv_last_page_len, I32),
                             ("workspace", workspace, None), ("out", out, BF16),
                             ("lse", lse, F32, True), *more), stream)


def _check_window(desc, q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len, workspace,
                  out, lse, stream, batch, kvp=None, last=None, qo_indptr=None):
    """The tensors of a windowed call of `batch` requests over the bf16 cache."""
    try:
        plain = (stream is None and q.is_cuda and q.dtype is BF16 and q.is_contiguous() and
                 out.dtype is BF16 and out.is_contiguous() and
                 k_cache.dtype is BF16 and k_cache.is_contiguous() and
                 v_cache.dtype is BF16 and v_cache.is_contiguous() and
                 kv_indptr.dtype is I32 and kv_indptr.is_contiguous() and
                 kv_indices.dtype is I32 and kv_indices.is_contiguous() and
                 kv_last_page_len.dtype is I32 and kv_last_page_len.is_contiguous() and
                 (lse is None or (lse.dtype is F32 and lse.is_contiguous())) and
                 (qo_indptr is None or (qo_indptr.dtype is I32 and qo_indptr.is_contiguous())) and
                 workspace.is_contiguous())
        shape, cache = q.shape, k_cache.shape
        plain = plain and shape[0] > 0
    except (AttributeError, IndexError):
        plain = False
    if not plain:
        _check_window_tensors(q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len,
                              workspace, out, lse, stream, qo_indptr)
        shape, cache = q.shape, k_cache.shape
    hq, d = desc.num_qo_heads, desc.head_dim
    rows = (cache[0], desc.page_size, desc.num_kv_heads, d)
    if cache != rows or v_cache.shape != rows:
        raise ValueError(f"k_cache and v_cache must be {rows} (num_pages, page_size, "
                         f"num_kv_heads, head_dim) for this descriptor, got "
                         f"{tuple(cache)} and {tuple(v_cache.shape)}")
    if shape != (shape[0], hq, d) or out.shape != shape:
        raise ValueError(f"q and out must be {(shape[0], hq, d)}, got {tuple(shape)} and "
                         f"{tuple(out.shape)}")
    if lse is not None and lse.numel() != shape[0] * hq:
        raise ValueError(f"lse must hold {shape[0]} x {hq} floats")
    _check_table(batch, kv_indptr, kv_indices, kv_last_page_len, kvp, last)


def bia_decode_window_workspace_size(desc, window, sinks, kv_indptr_host, kv_last_page_len_host,
                                     split_size=0) -> int:
    window, sinks, split_size = _window_ints(window, sinks, split_size)
    kvp, last = _host_i32(kv_indptr_host), _host_i32(kv_last_page_len_host)
    return int(load().bia_decode_window_workspace_size(
        ctypes.byref(desc), window, sinks, _ptr(kvp), _ptr(last), len(kvp) - 1,
        split_size))


def bia_decode_paged_window(desc, window, sinks, q, k_cache, v_cache, kv_indptr, kv_indices,
                            kv_last_page_len, kv_indptr_host, kv_last_page_len_host, workspace,
                            out, lse=None, split_size=0, stream=None):
    """bia_decode_paged where a query sees the last `window` keys and the first
    `sinks` keys of its request (include/bia.h states the rule)."""
    window, sinks, split_size = _window_ints(window, sinks, split_size)
    kvp, last = _host(kv_indptr_host), _host(kv_last_page_len_host)
    batch = q.shape[0]
    _check_window(desc, q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len, workspace,
                  out, lse, stream, batch, kvp, last)
    rc = load().bia_decode_paged_window(
        ctypes.byref(desc), window, sinks, q.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), k_cache.shape[0], kv_indptr.data_ptr(), kv_indices.data_ptr(),
        kv_last_page_len.data_ptr(), kvp.data_ptr(), last.data_ptr(), batch, split_size,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), out.data_ptr(),
        _at(lse), _handle(stream))
    if rc != BIA_OK:
        _check_window_tensors(q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len,
                              workspace, out, lse, stream)
        raise BiaError(rc, "bia_decode_paged_window")


def bia_decode_window_bounded_workspace_size(desc, bounds, window, sinks, batch,
                                             split_size=0) -> int:
    window, sinks, split_size = _window_ints(window, sinks, split_size)
    return int(load().bia_decode_window_bounded_workspace_size(
        ctypes.byref(desc), ctypes.byref(bounds), window, sinks, int(batch),
        split_size))


def bia_decode_paged_window_bounded(desc, bounds, window, sinks, q, k_cache, v_cache, kv_indptr,
                                    kv_indices, kv_last_page_len, workspace, out, lse=None,
                                    split_size=0, stream=None):
    """bia_decode_paged_window sized from `bounds` (max_kv_len): the index arrays
    are read on the device only, so a captured decode replays step after step."""
    window, sinks, split_size = _window_ints(window, sinks, split_size)
    batch = q.shape[0]
    _check_window(desc, q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len, workspace,
                  out, lse, stream, batch)
    rc = load().bia_decode_paged_window_bounded(
        ctypes.byref(desc), ctypes.byref(bounds), window, sinks, q.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), k_cache.shape[0], kv_indptr.data_ptr(),
        kv_indices.data_ptr(), kv_last_page_len.data_ptr(), batch, split_size,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), out.data_ptr(),
        _at(lse), _handle(stream))
    if rc != BIA_OK:
        _check_window_tensors(q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len,
                              workspace, out, lse, stream)
        raise BiaError(rc, "bia_decode_paged_window_bounded")


def bia_prefill_window_workspace_size(desc, window, sinks, qo_indptr_host, kv_indptr_host,
                                      kv_last_page_len_host, split_size=0) -> int:
    window, sinks, split_size = _window_ints(window, sinks, split_size)
    qo, kvp, last = (_host_i32(qo_indptr_host), _host_i32(kv_indptr_host),
                     _host_i32(kv_last_page_len_host))
    return int(load().bia_prefill_window_workspace_size(
        ctypes.byref(desc), window, sinks, _ptr(qo), _ptr(kvp), _ptr(last), len(qo) - 1,
        split_size))


def bia_prefill_paged_window(desc, window, sinks, q, k_cache, v_cache, qo_indptr, kv_indptr,
                             kv_indices, kv_last_page_len, qo_indptr_host, kv_indptr_host,
                             kv_last_page_len_host, workspace, out, lse=None, split_size=0,
                             stream=None):
    """bia_prefill_paged (causal) where a query sees the last `window` keys up to
    its own and the first `sinks` keys (include/bia.h states the rule)."""
    window, sinks, split_size = _window_ints(window, sinks, split_size)
    qo, kvp, last = (_host(qo_indptr_host), _host(kv_indptr_host),
                     _host(kv_last_page_len_host))
    batch = qo.numel() - 1
    _check_window(desc, q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len, workspace,
                  out, lse, stream, batch, kvp, last, qo_indptr)
    if qo_indptr.numel() != batch + 1:
        raise ValueError(f"qo_indptr must hold {batch + 1} entries, got {qo_indptr.numel()}")
    if q.shape[0] != _last(qo):
        raise ValueError(f"q holds {q.shape[0]} tokens, qo_indptr_host ends at {_last(qo)}")
    rc = load().bia_prefill_paged_window(
        ctypes.byref(desc), window, sinks, q.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), k_cache.shape[0], qo_indptr.data_ptr(), kv_indptr.data_ptr(),
        kv_indices.data_ptr(), kv_last_page_len.data_ptr(), qo.data_ptr(), kvp.data_ptr(),
        last.data_ptr(), batch, split_size, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), out.data_ptr(), _at(lse), _handle(stream))
    if rc != BIA_OK:
        _check_window_tensors(q, k_cache, v_cache, kv_indptr, kv_indices, kv_last_page_len,
                              workspace, out, lse, stream, qo_indptr)
        raise BiaError(rc, "bia_prefill_paged_window")
