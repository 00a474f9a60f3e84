"""ctypes binding over libfa_gb300.so (C ABI declared in include/fa.h).

The ``fa_*`` functions mirror the C entry points one to one (pointers as
Python ints, streams as ints).  ``prefill`` / ``decode`` are the two calls of
the flash-attention-cuda README's usage section, taking torch tensors: they
only check and marshal arguments, allocate the output, and call the library; so do the calls
on a paged cache at the end, whose usual arguments are read by the CPython module _paged_calls.
Every step of the computation runs in the library's CUDA kernels; if the
library is missing this module raises -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import importlib
import math
import os
import struct
import threading

from . import build as _build

FA_F16, FA_BF16, FA_F32 = 0, 1, 2
FA_FLAG_NONE, FA_FLAG_NO_CAUSAL_SKIP = 0, 1
FA_FLAG_SCHEDULE_UNITS, FA_FLAG_SCHEDULE_STREAM_K = 2, 4
FA_BWD_FLAG_NONE, FA_BWD_RECOMPUTE_DQ = 0, 1
FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_SHAPE", 3: "FA_ERR_HEAD_DIM",
    4: "FA_ERR_DTYPE", 5: "FA_ERR_ALIGN", 6: "FA_ERR_SCALE", 7: "FA_ERR_ARCH",
    8: "FA_ERR_WORKSPACE", 9: "FA_ERR_CUDA", 10: "FA_ERR_WATCHDOG",
    11: "FA_ERR_SEQ_LEN", 12: "FA_ERR_ALIAS", 13: "FA_ERR_SPLITS",
    14: "FA_ERR_PAGE",
}
(FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_HEAD_DIM, FA_ERR_DTYPE, FA_ERR_ALIGN, FA_ERR_SCALE, FA_ERR_ARCH,
 FA_ERR_WORKSPACE, FA_ERR_CUDA, FA_ERR_WATCHDOG, FA_ERR_SEQ_LEN, FA_ERR_ALIAS,
 FA_ERR_SPLITS, FA_ERR_PAGE) = range(1, 15)

_lock = threading.Lock()
_lib = None

_vp, _i, _f, _u, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint, ctypes.c_size_t
_ll = ctypes.c_longlong
_SIGNATURES = {
    "fa_prefill": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp]),
    "fa_prefill_ex": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "fa_prefill_gqa": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _u, _vp]),
    "fa_prefill_host": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _u, _vp]),
    "fa_prefill_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                               _f, _i, _i, _u, _vp]),
    "fa_prefill_lse": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _u,
                            _vp]),
    "fa_prefill_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                 _i, _f, _i, _i, _vp]),
    "fa_prefill_backward_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                    _i, _f, _i, _i, _u, _vp]),
    "fa_prefill_plan": (_i, [_i, _i, _i, _i, _i, _u, _i, _vp, _vp, _i]),
    "fa_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp]),
    "fa_decode_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz, _vp]),
    "fa_decode_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz,
                           _vp]),
    "fa_decode_gqa_choose_splits": (_i, [_i, _i, _i, _i, _i]),
    "fa_decode_splits_for_sms": (_i, [_i, _i, _i, _i, _i]),
    "fa_decode_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _vp]),
    "fa_decode_noalloc_max_bytes": (_sz, []),
    "fa_decode_choose_splits": (_i, [_i, _i, _i, _i]),
    "fa_decode_chunk_len": (_i, [_i, _i]),
    "fa_decode_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fa_cache_append": (_i, [_vp, _vp, _vp, _vp, _vp, _ll, _ll, _ll, _ll, _vp, _i, _vp, _vp, _vp,
                             _i, _i, _i, _vp, _i, _i, _i, _vp]),
    "fa_decode_paged": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_prefill_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                              _vp, _sz, _vp]),
    "fa_decode_shared": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _vp, _i, _i, _f, _i, _vp, _sz,
                              _vp]),
    "fa_paged_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fa_shared_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_last_cuda_error": (_i, []),
    "fa_device_status": (_i, [_i]),
    "fa_watchdog_selftest": (_i, [ctypes.c_longlong, _vp, _vp]),
    "fa_pool_stats": (_i, [_vp, _i]),
    "fa_read_probe": (_i, [_vp, _sz, _vp, _vp]),
    "fa_version": (_i, []),
}


class PagedCacheArg(ctypes.Structure):
    """fa_paged_cache of include/fa.h."""
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("page_stride", _ll), ("head_stride", _ll),
                ("slot_stride", _ll), ("num_pages", _i), ("num_heads", _i), ("page_size", _i),
                ("head_dim", _i), ("dtype", _i)]


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({status_string(status)})")


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = False):
    """Load libfa_gb300.so (building it first only if asked)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if not os.path.exists(path):
                if not build_if_missing:
                    raise RuntimeError(
                        f"{path} is missing: build it with attention_forward_prefill_gb300.build"
                        ".build() (there is no CPU fallback)")
                _build.build()
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


_calls = None


class _InPython:
    """In the place of _paged_calls where it is not built: every call goes through the checks in Python."""
    append = decode = prefill = shared = staticmethod(lambda *args: NotImplemented)


def _fast():
    """The module _paged_calls over the loaded library."""
    global _calls
    if _calls is None:
        lib = load()
        try:
            _paged_calls = importlib.import_module("._paged_calls", __package__)
        except ModuleNotFoundError:
            _calls = _InPython
            return _calls
        _paged_calls.init(_torch(), FaError, *(ctypes.cast(getattr(lib, n), _vp).value for n in (
            "fa_cache_append", "fa_decode_paged", "fa_prefill_paged", "fa_decode_shared")))
        _calls = _paged_calls
    return _calls


# ---------------------------------------------------------------- raw C ABI
def fa_prefill(q, k, v, out, B, H, N, d, causal, scale, stream=0) -> int:
    return load().fa_prefill(q, k, v, out, B, H, N, d, int(causal), float(scale), stream)


def fa_prefill_ex(q, k, v, out, B, H, N, d, causal, scale, in_dtype, out_dtype,
                  stream=0) -> int:
    return load().fa_prefill_ex(q, k, v, out, B, H, N, d, int(causal), float(scale),
                                in_dtype, out_dtype, stream)


def fa_prefill_gqa(q, k, v, out, B, Hq, Hkv, Nq, Nk, d, causal, scale, in_dtype, out_dtype,
                   flags=0, stream=0) -> int:
    return load().fa_prefill_gqa(q, k, v, out, B, Hq, Hkv, Nq, Nk, d, int(causal), float(scale),
                                 in_dtype, out_dtype, flags, stream)


def fa_prefill_host(q, k, v, out, B, Hq, Hkv, Nq, Nk, d, causal, scale, in_dtype, out_dtype,
                    flags=0, stream=0) -> int:
    return load().fa_prefill_host(q, k, v, out, B, Hq, Hkv, Nq, Nk, d, int(causal), float(scale),
                                  in_dtype, out_dtype, flags, stream)


def fa_prefill_varlen(q, k, v, out, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv, total_q, total_k,
                      max_seqlen_q, max_seqlen_k, d, causal, scale, in_dtype, out_dtype, flags=0,
                      stream=0) -> int:
    return load().fa_prefill_varlen(q, k, v, out, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv, total_q,
                                    total_k, max_seqlen_q, max_seqlen_k, d, int(causal),
                                    float(scale), in_dtype, out_dtype, flags, stream)


def fa_prefill_lse(q, k, v, out, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, in_dtype, out_dtype,
                   flags=0, stream=0) -> int:
    return load().fa_prefill_lse(q, k, v, out, lse, B, Hq, Hkv, Nq, Nk, d, int(causal),
                                 float(scale), in_dtype, out_dtype, flags, stream)


def fa_prefill_backward(q, k, v, out, dout, lse, dq, dk, dv, B, H, Hkv, N, d, causal, scale,
                        in_dtype, grad_dtype, stream=0) -> int:
    return load().fa_prefill_backward(q, k, v, out, dout, lse, dq, dk, dv, B, H, Hkv, N, d,
                                      int(causal), float(scale), in_dtype, grad_dtype, stream)


def fa_prefill_backward_ex(q, k, v, out, dout, lse, dq, dk, dv, B, H, Hkv, N, d, causal, scale,
                           in_dtype, grad_dtype, flags=0, stream=0) -> int:
    return load().fa_prefill_backward_ex(q, k, v, out, dout, lse, dq, dk, dv, B, H, Hkv, N, d,
                                         int(causal), float(scale), in_dtype, grad_dtype, flags,
                                         stream)


def fa_prefill_plan(B, Hq, Nq, Nk, causal, flags=0, num_sms=0, max_items=192):
    """The prefill schedule as (status, info[9], items[n][5]) -- host arithmetic only."""
    info = (ctypes.c_longlong * 9)()
    items = (ctypes.c_longlong * (5 * max_items))()
    rc = load().fa_prefill_plan(B, Hq, Nq, Nk, int(causal), flags, num_sms, info, items, max_items)
    n = int(info[5]) if rc == FA_OK else 0
    rows = [tuple(int(items[5 * i + c]) for c in range(5)) for i in range(min(n, max_items))]
    return rc, [int(x) for x in info], rows


def fa_decode(q, k_cache, v_cache, seq_lens, out, B, H, max_len, d, scale, stream=0) -> int:
    return load().fa_decode(q, k_cache, v_cache, seq_lens, out, B, H, max_len, d,
                            float(scale), stream)


def fa_decode_ex(q, k_cache, v_cache, seq_lens, out, B, H, max_len, d, scale, in_dtype,
                 out_dtype, num_splits=0, workspace=None, workspace_bytes=0, stream=0) -> int:
    return load().fa_decode_ex(q, k_cache, v_cache, seq_lens, out, B, H, max_len, d,
                               float(scale), in_dtype, out_dtype, num_splits, workspace,
                               workspace_bytes, stream)


def fa_decode_gqa(q, k_cache, v_cache, seq_lens, out, B, Hq, Hkv, max_len, d, scale, in_dtype,
                  out_dtype, num_splits=0, workspace=None, workspace_bytes=0, stream=0) -> int:
    return load().fa_decode_gqa(q, k_cache, v_cache, seq_lens, out, B, Hq, Hkv, max_len, d,
                                float(scale), in_dtype, out_dtype, num_splits, workspace,
                                workspace_bytes, stream)


def fa_decode_gqa_choose_splits(B, Hq, Hkv, max_len, device=-1) -> int:
    return load().fa_decode_gqa_choose_splits(B, Hq, Hkv, max_len, device)


def fa_decode_splits_for_sms(B, Hq, Hkv, max_len, num_sms) -> int:
    return load().fa_decode_splits_for_sms(B, Hq, Hkv, max_len, num_sms)


def fa_decode_noalloc(q, k_cache, v_cache, seq_lens, out, B, H, max_len, d, scale, in_dtype,
                      out_dtype, num_splits=0, stream=0) -> int:
    """Decode with the library's static scratch: allocates no device memory."""
    return load().fa_decode_noalloc(q, k_cache, v_cache, seq_lens, out, B, H, max_len, d,
                                    float(scale), in_dtype, out_dtype, num_splits, stream)


def fa_decode_noalloc_max_bytes() -> int:
    return load().fa_decode_noalloc_max_bytes()


def fa_decode_choose_splits(B, H, max_len, device=-1) -> int:
    return load().fa_decode_choose_splits(B, H, max_len, device)


def fa_decode_chunk_len(max_len, num_splits) -> int:
    return load().fa_decode_chunk_len(max_len, num_splits)


def fa_decode_workspace_bytes(B, H, max_len, d, num_splits) -> int:
    return load().fa_decode_workspace_bytes(B, H, max_len, d, num_splits)


def fa_cache_append(cache, q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, page_table,
                    max_pages, seq_lens, cu_seqlens, positions, B, Hq, total, rope, max_positions,
                    rope_dim, interleaved, stream=0) -> int:
    return load().fa_cache_append(ctypes.byref(cache), q, k, v, q_out, q_stride, k_stride, v_stride,
                                  q_out_stride, page_table, max_pages, seq_lens, cu_seqlens,
                                  positions, B, Hq, total, rope, max_positions, rope_dim,
                                  int(interleaved), stream)


def fa_decode_paged(cache, q, out, page_table, max_pages, seq_lens, B, Hq, scale, out_dtype,
                    workspace=None, workspace_bytes=0, stream=0) -> int:
    return load().fa_decode_paged(ctypes.byref(cache), q, out, page_table, max_pages, seq_lens, B,
                                  Hq, scale, out_dtype, workspace, workspace_bytes, stream)


def fa_prefill_paged(cache, q, out, lse, page_table, max_pages, seq_lens, cu_seqlens_q, B, Hq,
                     total_q, max_seqlen_q, causal, scale, out_dtype, workspace=None,
                     workspace_bytes=0, stream=0) -> int:
    return load().fa_prefill_paged(ctypes.byref(cache), q, out, lse, page_table, max_pages,
                                   seq_lens, cu_seqlens_q, B, Hq, total_q, max_seqlen_q,
                                   int(causal), scale, out_dtype, workspace, workspace_bytes,
                                   stream)


def fa_decode_shared(cache, q, out, prefix_table, max_prefix_pages, prefix_len, page_table,
                     max_pages, seq_lens, B, Hq, scale, out_dtype, workspace=None,
                     workspace_bytes=0, stream=0) -> int:
    return load().fa_decode_shared(ctypes.byref(cache), q, out, prefix_table, max_prefix_pages,
                                   prefix_len, page_table, max_pages, seq_lens, B, Hq, scale,
                                   out_dtype, workspace, workspace_bytes, stream)


def fa_paged_workspace_bytes(Hq, Hkv, max_seqlen_q, d, device=-1) -> int:
    return load().fa_paged_workspace_bytes(Hq, Hkv, max_seqlen_q, d, device)


def fa_shared_workspace_bytes(B, Hq, Hkv, d, device=-1) -> int:
    return load().fa_shared_workspace_bytes(B, Hq, Hkv, d, device)


def status_string(status: int) -> str:
    return load().fa_status_string(status).decode()


def fa_last_cuda_error() -> int:
    return load().fa_last_cuda_error()


def fa_device_status(reset: bool = False) -> int:
    return load().fa_device_status(int(reset))


def fa_version() -> int:
    return load().fa_version()


def fa_watchdog_selftest(limit_ns, result, stream=0) -> int:
    return load().fa_watchdog_selftest(int(limit_ns), result, stream)


def fa_pool_stats(reset_high: bool = False):
    """(status, [reserved, reserved_high, used, used_high]) of the library's scratch pool."""
    out = (ctypes.c_longlong * 4)()
    rc = load().fa_pool_stats(out, int(reset_high))
    return rc, [int(x) for x in out]


def fa_read_probe(src, nbytes, xor_out, stream=0) -> int:
    return load().fa_read_probe(src, nbytes, xor_out, stream)


# ---------------------------------------------------------------- torch calls
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.float16:
        return FA_F16
    if dt == torch.bfloat16:
        return FA_BF16
    if dt == torch.float32:
        return FA_F32
    raise TypeError(f"unsupported dtype {dt}")


def _check_cuda(name, t, shape=None, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _stream_handle(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def prefill(q, k, v, causal: bool = False, scale: float | None = None, out_dtype=None,
            flags: int = 0, out=None, sync: bool = True):
    """out = softmax(scale * q k^T [causal]) v for q [B, Hq, Nq, d] and k, v
    [B, Hkv, Nk, d] (fp16/bf16; Hq a multiple of Hkv; causal queries are the
    last Nq positions).

    CUDA inputs run on the current stream and return a CUDA tensor.  Host
    inputs go through fa_prefill_host (copies in, compute and copies out
    pipelined over chunks of heads) on the current stream and return the host
    result (pinned when q is).  With sync (the default) the call waits for the
    stream first; with sync=False it returns at once, like the C call, and the
    result is ready, and the host tensors free to reuse, once the stream has
    passed the call.
    """
    torch = _torch()
    if not q.is_cuda:
        return _prefill_host(torch, q, k, v, causal, scale, out_dtype, flags, out, sync)
    B, Hq, Nq, d = q.shape
    _check_cuda("q", q)
    _check_cuda("k", k, None, q.dtype)
    if k.dim() != 4 or k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [{B}, Hkv, Nk, {d}]")
    Hkv, Nk = k.shape[1], k.shape[2]
    _check_cuda("v", v, k.shape, q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    else:
        _check_cuda("out", out, q.shape, out_dtype)
    rc = fa_prefill_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq, Hkv, Nq,
                        Nk, d, causal, scale, dtype_code(q.dtype), dtype_code(out_dtype), flags,
                        _stream_handle(q.device))
    if rc != FA_OK:
        raise FaError(rc, "fa_prefill_gqa")
    return out


def _check_host(name, t, shape=None, dtype=None):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor when q is")
    if t.dtype not in (_torch().float16, _torch().bfloat16) and name != "out":
        raise ValueError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _prefill_host(torch, q, k, v, causal, scale, out_dtype, flags, out, sync=True):
    B, Hq, Nq, d = q.shape
    _check_host("q", q)
    _check_host("k", k, None, q.dtype)
    if k.dim() != 4 or k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [{B}, Hkv, Nk, {d}]")
    Hkv, Nk = k.shape[1], k.shape[2]
    _check_host("v", v, k.shape, q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, pin_memory=q.is_pinned())
    else:
        _check_host("out", out, q.shape, out_dtype)
    stream = torch.cuda.current_stream()
    rc = fa_prefill_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq, Hkv, Nq,
                         Nk, d, causal, scale, dtype_code(q.dtype), dtype_code(out_dtype), flags,
                         stream.cuda_stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_prefill_host")
    if sync:
        stream.synchronize()
    return out


def prefill_with_lse(q, k, v, causal: bool = False, scale: float | None = None, flags: int = 0):
    """Forward for training: returns (out, lse) with out in q's dtype and lse
    fp32 [B, Hq, Nq] (natural-log row log-sum-exp of the visible scores)."""
    torch = _torch()
    B, Hq, Nq, d = q.shape
    _check_cuda("q", q)
    _check_cuda("k", k, None, q.dtype)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check_cuda("v", v, k.shape, q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    rc = fa_prefill_lse(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B,
                        Hq, Hkv, Nq, Nk, d, causal, scale, dtype_code(q.dtype), dtype_code(q.dtype),
                        flags, _stream_handle(q.device))
    if rc != FA_OK:
        raise FaError(rc, "fa_prefill_lse")
    return out, lse


def prefill_backward(q, k, v, out, dout, lse, causal: bool = False, scale: float | None = None,
                     grad_dtype=None, flags: int = 0):
    """(dq, dk, dv) for square prefill with q, out, dout [B, H, N, d] and k, v
    [B, Hkv, N, d], from the forward's out and lse; dk, dv have k's shape.
    flags: FA_BWD_* bits (FA_BWD_RECOMPUTE_DQ)."""
    torch = _torch()
    B, H, N, d = q.shape
    for name, t in (("q", q), ("out", out), ("dout", dout)):
        _check_cuda(name, t, q.shape, q.dtype)
    _check_cuda("k", k, None, q.dtype)
    if k.dim() != 4 or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [{B}, Hkv, {N}, {d}]")
    _check_cuda("v", v, k.shape, q.dtype)
    Hkv = k.shape[1]
    _check_cuda("lse", lse, (B, H, N), torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    grad_dtype = q.dtype if grad_dtype is None else grad_dtype
    dq = torch.empty(q.shape, dtype=grad_dtype, device=q.device)
    dk, dv = (torch.empty(k.shape, dtype=grad_dtype, device=q.device) for _ in range(2))
    rc = fa_prefill_backward_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), B, H, Hkv, N, d, causal, scale, dtype_code(q.dtype),
                                dtype_code(grad_dtype), flags, _stream_handle(q.device))
    if rc != FA_OK:
        raise FaError(rc, "fa_prefill_backward_ex")
    return dq, dk, dv


def prefill_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                   causal: bool = False, scale: float | None = None, out_dtype=None,
                   flags: int = 0, out=None):
    """Packed variable-length prefill: q [total_q, Hq, d], k, v [total_k, Hkv, d],
    cu_seqlens_* int32 [B + 1] on the same device.  Returns [total_q, Hq, d]."""
    torch = _torch()
    _check_cuda("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, d]")
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    _check_cuda("k", k, (total_k, Hkv, d), q.dtype)
    _check_cuda("v", v, k.shape, q.dtype)
    B = cu_seqlens_q.shape[0] - 1
    _check_cuda("cu_seqlens_q", cu_seqlens_q, (B + 1,), torch.int32)
    _check_cuda("cu_seqlens_k", cu_seqlens_k, (B + 1,), torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    else:
        _check_cuda("out", out, q.shape, out_dtype)
    rc = fa_prefill_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Hq, Hkv, total_q,
                           total_k, int(max_seqlen_q), int(max_seqlen_k), d, causal, scale,
                           dtype_code(q.dtype), dtype_code(out_dtype), flags,
                           _stream_handle(q.device))
    if rc != FA_OK:
        raise FaError(rc, "fa_prefill_varlen")
    return out


def decode(q, k_cache, v_cache, seq_lens, scale: float | None = None, out_dtype=None,
           num_splits: int = 0, workspace=None, out=None):
    """One query row per (b, h) over the first seq_lens[b] rows of the cache.

    q: [B, Hq, 1, d]; caches: [B, Hkv, max_len, d] with Hkv dividing Hq (query
    head h reads cache head h // (Hq // Hkv)); seq_lens: int32 [B] on the same
    device.  Returns [B, Hq, 1, d].
    """
    torch = _torch()
    B, Hkv, max_len, d = k_cache.shape
    _check_cuda("k_cache", k_cache)
    _check_cuda("v_cache", v_cache, k_cache.shape, k_cache.dtype)
    _check_cuda("q", q, None, k_cache.dtype)
    if q.dim() != 4 or q.shape[0] != B or q.shape[2] != 1 or q.shape[3] != d:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [{B}, Hq, 1, {d}]")
    Hq = q.shape[1]
    _check_cuda("seq_lens", seq_lens, (B,), torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, Hq, 1, d), dtype=out_dtype, device=q.device)
    else:
        _check_cuda("out", out, (B, Hq, 1, d), out_dtype)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _check_cuda("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = fa_decode_gqa(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seq_lens.data_ptr(),
                       out.data_ptr(), B, Hq, Hkv, max_len, d, scale, dtype_code(q.dtype),
                       dtype_code(out_dtype), num_splits, ws_ptr, ws_bytes,
                       _stream_handle(q.device))
    if rc != FA_OK:
        raise FaError(rc, "fa_decode_gqa")
    return out


# ---------------------------------------------------------------- paged cache
def rope_table(positions: int, rope_dim: int, base: float = 10000.0, device="cuda"):
    """Cosines and sines of p * base^(-2 i / rope_dim) as cache_append takes them: fp32
    [positions, rope_dim], a row's cosines first.  The angles are computed in 64 bits."""
    torch = _torch()
    freq = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# A call of a few microseconds on the GPU is bound by what happens on the host, so arguments go to
# _paged_calls first, which makes the call where they are what a call mostly gets and returns
# NotImplemented otherwise; the checks here then say what is wrong, or make the call.
_PACK_CACHE = struct.Struct("@PPqqqiiiii4x").pack  # fa_paged_cache, its tail padding with it
_codes = {}


def _code_of(dtype) -> int:
    code = _codes.get(dtype)
    if code is None:
        code = _codes[dtype] = dtype_code(dtype)
    return code


def _pages(k_pages, v_pages):
    """(fa_paged_cache as bytes, heads, d) of two [pages, heads, slots, d] tensors (any strides, the
    same for both)."""
    shape, stride, dtype = k_pages.shape, k_pages.stride(), k_pages.dtype
    if not (k_pages.is_cuda and len(shape) == 4 and stride[3] == 1 and v_pages.shape == shape and
            v_pages.stride() == stride and v_pages.dtype == dtype and v_pages.device == k_pages.device):
        if not (k_pages.is_cuda and v_pages.is_cuda):
            raise ValueError("k_pages and v_pages must be CUDA tensors")
        if len(shape) != 4:
            raise ValueError(f"k_pages has shape {tuple(shape)}, expected [pages, heads, slots, d]")
        if stride[3] != 1:
            raise ValueError("the channels of a slot must be contiguous")
        raise ValueError("v_pages must have the shape, strides, dtype and device of k_pages")
    pages, heads, slots, d = shape
    return _PACK_CACHE(k_pages.data_ptr(), v_pages.data_ptr(), stride[0], stride[1], stride[2], pages, heads,
                       slots, d, _code_of(dtype)), heads, d


def _is_ints(t, device, int32, dims):
    """t is an int32 array that _check_ints has nothing to say on but its sizes."""
    return t.dtype is int32 and t.dim() == dims and t.is_contiguous() and t.device == device


def _check_ints(device, name, t, shape):
    """int32 arrays of the device: contiguous and where the cache is; a None in `shape` is any size."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, as the cache is")
    if t.dtype != _torch().int32:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.int32")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"[{', '.join('any' if n is None else str(n) for n in shape)}]")


def _stride3(t):
    stride = t.stride()
    return stride if len(stride) == 3 else (0, 0, 0)


def _check_rows(name, t, tokens, heads, k_pages):
    """[tokens, heads, d] rows in the cache's type, of which only the tokens may have a stride; returns
    it and the number of heads."""
    shape, stride, d = t.shape, t.stride(), k_pages.shape[3]
    if not (t.dtype == k_pages.dtype and t.device == k_pages.device and len(shape) == 3 and shape[0] == tokens and
            shape[2] == d and stride[2] == 1 and (stride[1] == d or shape[1] == 1) and
            (heads is None or shape[1] == heads)):
        if t.device != k_pages.device or t.dtype != k_pages.dtype:
            raise ValueError(f"{name} must have the dtype and device of the cache")
        if len(shape) != 3 or shape[0] != tokens or shape[2] != d or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} has shape {tuple(shape)}, expected [{tokens}, "
                             f"{'heads' if heads is None else heads}, {d}]")
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return stride[0], shape[1]


def _tables(device, page_table, seq_lens):
    """Checks both; the batch and the width of the table."""
    int32 = _torch().int32
    B = seq_lens.numel()
    if _is_ints(seq_lens, device, int32, 1) and _is_ints(page_table, device, int32, 2):
        rows, width = page_table.shape
        if rows == B:
            return B, width
    _check_ints(device, "seq_lens", seq_lens, (B,))
    _check_ints(device, "page_table", page_table, (B, None))
    raise AssertionError("unreachable")


def _run(name, device, *args):
    """The library's call `name` with `device` current, on its current stream."""
    torch = _torch()
    fn = getattr(_lib or load(), name)
    index = device.index
    if index == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != FA_OK:
        raise FaError(rc, name)


def _workspace(workspace, device):
    if workspace is None:
        return None, 0
    _check_cuda("workspace", workspace)
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}, as the cache is")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def cache_append(q, k, v, k_pages, v_pages, page_table, seq_lens, cu_seqlens=None, rope=None,
                 interleaved: bool = False, positions=None, out=None):
    """Put the keys and values of new tokens into their slots of a paged cache and give q and k
    their rotary positions on the way; returns the turned q (None when q is None).

    q [T, Hq, d] (or None), k, v [T, Hkv, d]: a token's heads contiguous, tokens any stride
    apart, as slices of one fused projection are.  k_pages, v_pages [pages, Hkv, slots, d], any
    strides; page_table int32 [B, max_pages].  seq_lens int32 [B]: the lengths with the new
    tokens in.  cu_seqlens int32 [B + 1]: the sequences' token offsets; None: one token each.
    rope: rope_table(...)'s rows, as wide as the channels that turn, or None.  positions int32
    [T]: the rotary positions where they are not the positions in the sequence.  out may be q;
    its rows behind the last sequence are not written.
    """
    done = (_calls or _fast()).append(q, k, v, k_pages, v_pages, page_table, seq_lens, cu_seqlens, rope, interleaved,
                                      positions, out)
    if done is not NotImplemented:
        return done
    torch = _torch()
    cache, Hkv, d = _pages(k_pages, v_pages)
    device, dtype = k_pages.device, k_pages.dtype
    total = k.shape[0]
    rows, (k_stride, k_head, k_one), (v_stride, v_head, v_one) = (total, Hkv, d), _stride3(k), _stride3(v)
    if not (k.shape == rows and v.shape == rows and k.dtype is dtype and v.dtype is dtype and k.device == device and
            v.device == device and k_one == v_one == 1 and (k_head == v_head == d or Hkv == 1)):
        _check_rows("k", k, total, Hkv, k_pages)
        _check_rows("v", v, total, Hkv, k_pages)
    B, max_pages = _tables(device, page_table, seq_lens)
    cu_ptr = pos_ptr = rope_ptr = None
    max_positions = rope_dim = 0
    if cu_seqlens is not None:
        if not (_is_ints(cu_seqlens, device, torch.int32, 1) and cu_seqlens.numel() == B + 1):
            _check_ints(device, "cu_seqlens", cu_seqlens, (B + 1,))
        cu_ptr = cu_seqlens.data_ptr()
    if positions is not None:
        _check_ints(device, "positions", positions, (total,))
        pos_ptr = positions.data_ptr()
    if rope is not None:
        if not (rope.dtype is torch.float32 and rope.dim() == 2 and rope.is_contiguous() and rope.device == device):
            raise ValueError("rope must be a contiguous float32 [positions, rope_dim] tensor beside the cache")
        max_positions, rope_dim = rope.shape
        if rope_dim:
            rope_ptr = rope.data_ptr()
    Hq = q_stride = out_stride = 0
    q_ptr = out_ptr = None
    if q is not None:
        q_stride, Hq = _check_rows("q", q, total, None, k_pages)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            out_stride = Hq * d
        else:
            out_stride, _ = _check_rows("out", out, total, Hq, k_pages)
        q_ptr, out_ptr = q.data_ptr(), out.data_ptr()
    elif out is not None:
        raise ValueError("out without q")
    if total:
        _run("fa_cache_append", device, cache, q_ptr, k.data_ptr(), v.data_ptr(), out_ptr, q_stride, k_stride,
             v_stride, out_stride, page_table.data_ptr(), max_pages, seq_lens.data_ptr(), cu_ptr, pos_ptr,
             B, Hq, total, rope_ptr, max_positions, rope_dim, 1 if interleaved else 0)
    return out


def _paged_args(q, k_pages, v_pages, page_table, seq_lens, scale, out_dtype, out):
    """The checks, defaults and output that the paged attention calls have in common."""
    torch = _torch()
    cache, _, d = _pages(k_pages, v_pages)
    device = k_pages.device
    if not (q.dtype == k_pages.dtype and q.device == device and q.is_contiguous()):
        if q.device != device or q.dtype != k_pages.dtype:
            raise ValueError("q must have the dtype and device of the cache")
        raise ValueError("q must be contiguous")
    B, max_pages = _tables(device, page_table, seq_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out_dtype is None:
        out_dtype = q.dtype
    if out is None:
        out = torch.empty_like(q, dtype=out_dtype)
    else:
        _check_cuda("out", out, q.shape, out_dtype)
        if out.device != device:
            raise ValueError("out must be on the device of the cache")
    return cache, d, device, B, max_pages, scale, _code_of(out_dtype), out


def _decode_rows(q, B, d):
    """Query heads of q [B, Hq, d] or [B, Hq, 1, d]."""
    shape = q.shape
    if not (len(shape) == 3 or (len(shape) == 4 and shape[2] == 1)) or shape[0] != B or shape[-1] != d:
        raise ValueError(f"q has shape {tuple(shape)}, expected [{B}, Hq, {d}] or [{B}, Hq, 1, {d}]")
    return shape[1]


def decode_paged(q, k_pages, v_pages, page_table, seq_lens, scale: float | None = None,
                 out_dtype=None, workspace=None, out=None):
    """One query token per sequence over the first seq_lens[b] tokens of its pages.

    q [B, Hq, d] or [B, Hq, 1, d]; k_pages, v_pages [pages, Hkv, slots, d], any strides;
    page_table int32 [B, max_pages]; seq_lens int32 [B].  Returns rows shaped as q.  The table's
    width bounds the lengths that the call is laid out for: a short call is some 5 us faster with
    one no wider than it needs.
    """
    if out_dtype is None and workspace is None:
        done = (_calls or _fast()).decode(q, k_pages, v_pages, page_table, seq_lens, scale, out)
        if done is not NotImplemented:
            return done
    cache, d, device, B, max_pages, scale, code, out = _paged_args(q, k_pages, v_pages, page_table, seq_lens, scale,
                                                                   out_dtype, out)
    ws, ws_bytes = _workspace(workspace, device)
    _run("fa_decode_paged", device, cache, q.data_ptr(), out.data_ptr(), page_table.data_ptr(), max_pages,
         seq_lens.data_ptr(), B, _decode_rows(q, B, d), scale, code, ws, ws_bytes)
    return out


def prefill_paged(q, k_pages, v_pages, page_table, seq_lens, cu_seqlens_q, max_seqlen_q: int,
                  causal: bool = False, scale: float | None = None, out_dtype=None, workspace=None,
                  out=None, lse=None):
    """Chunks of query tokens over a paged cache that already holds their keys.

    q [T, Hq, d] with sequence b's tokens at cu_seqlens_q[b] .. cu_seqlens_q[b + 1] (int32
    [B + 1]); causal queries are the last positions of their sequence's seq_lens[b] tokens.
    lse: optional fp32 [T, Hq] that receives the row log-sum-exp.  Returns [T, Hq, d]; rows
    outside every sequence are not written.
    """
    if out_dtype is None and workspace is None and lse is None:
        done = (_calls or _fast()).prefill(q, k_pages, v_pages, page_table, seq_lens, cu_seqlens_q, max_seqlen_q, causal,
                                           scale, out)
        if done is not NotImplemented:
            return done
    cache, d, device, B, max_pages, scale, code, out = _paged_args(q, k_pages, v_pages, page_table, seq_lens, scale,
                                                                   out_dtype, out)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [tokens, Hq, {d}]")
    total, Hq, _ = q.shape
    if not (_is_ints(cu_seqlens_q, device, _torch().int32, 1) and cu_seqlens_q.numel() == B + 1):
        _check_ints(device, "cu_seqlens_q", cu_seqlens_q, (B + 1,))
    lse_ptr = None
    if lse is not None:
        _check_cuda("lse", lse, (total, Hq), _torch().float32)
        if lse.device != device:
            raise ValueError("lse must be on the device of the cache")
        lse_ptr = lse.data_ptr()
    if total:
        ws, ws_bytes = _workspace(workspace, device)
        _run("fa_prefill_paged", device, cache, q.data_ptr(), out.data_ptr(), lse_ptr, page_table.data_ptr(),
             max_pages, seq_lens.data_ptr(), cu_seqlens_q.data_ptr(), B, Hq, total, int(max_seqlen_q),
             1 if causal else 0, scale, code, ws, ws_bytes)
    return out


def decode_shared(q, k_pages, v_pages, prefix_table, prefix_len, page_table, seq_lens,
                  scale: float | None = None, out_dtype=None, workspace=None, out=None):
    """decode_paged for a batch that shares a prefix: every row sees the first prefix_len tokens
    (int32 [1], on the device) of prefix_table's pages (int32 [n]), then its own.  A tile of the
    prefix is loaded once for up to 256 query rows of a kv head; a small call loads it once per
    sequence and kv head, out of L2.
    """
    if out_dtype is None and workspace is None:
        done = (_calls or _fast()).shared(q, k_pages, v_pages, prefix_table, prefix_len, page_table, seq_lens, scale, out)
        if done is not NotImplemented:
            return done
    cache, d, device, B, max_pages, scale, code, out = _paged_args(q, k_pages, v_pages, page_table, seq_lens, scale,
                                                                   out_dtype, out)
    int32 = _torch().int32
    if not (_is_ints(prefix_table, device, int32, 1) and _is_ints(prefix_len, device, int32, 1) and
            prefix_len.numel() == 1):
        _check_ints(device, "prefix_table", prefix_table, (None,))
        _check_ints(device, "prefix_len", prefix_len, (1,))
    ws, ws_bytes = _workspace(workspace, device)
    _run("fa_decode_shared", device, cache, q.data_ptr(), out.data_ptr(), prefix_table.data_ptr(),
         prefix_table.numel(), prefix_len.data_ptr(), page_table.data_ptr(), max_pages, seq_lens.data_ptr(),
         B, _decode_rows(q, B, d), scale, code, ws, ws_bytes)
    return out
