"""Thin ctypes binding of libpa (include/pa.h, include/pa_serving.h,
include/pa_request.h): argument marshalling only.

Every function takes torch tensors, checks that they are CUDA, contiguous and
of the expected dtype and shape, passes their device pointers and the current
torch stream to the C entry point of the same name, and raises ``PAError`` on a
non-zero return code.  All arithmetic happens in the CUDA kernels; if
libpa.so is missing this module raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

from . import build as _build

PA_F16, PA_BF16, PA_E4M3 = 0, 1, 2
PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA, PA_ERR_BOUNDS, \
    PA_ERR_TIMEOUT, PA_ERR_SCRATCH_LIMIT = range(8)
PA_NOALLOC_SCRATCH_BYTES = 16 << 20
PA_STATUS_BAD_BLOCK, PA_STATUS_BAD_LEN, PA_STATUS_BAD_SLOT, PA_STATUS_TIMEOUT = 1, 2, 4, 8
PA_STATUS_NO_WORKSPACE = 16
PA_STATUS_WS_DIRTY = 32
PA_F32 = 3
PA_STATUS_BAD_TOKEN = 64
PA_STATUS_BAD_ROW = 128
PA_DECODE_EARLY_PROLOGUE = 1
PA_DECODE_EARLY_COPIES = 2

# (name, argtypes, restype) of every exported entry point
_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_u32 = ctypes.c_uint
SIGNATURES = {
    "pa_version": ([], _i32),
    "pa_status_string": ([_i32], ctypes.c_char_p),
    "pa_cache_append": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_cache_append_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                             _vp], _i32),
    "pa_quantize_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_e4m3_encode": ([_vp, _vp, _i64, _vp], _i32),
    "pa_copy_blocks": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_decode_workspace_size": ([_i32, _i32, _i32, _i32], _sz),
    "pa_decode_workspace_size_rows": ([_i32, _i32, _i32, _i32, _i32], _sz),
    "pa_decode_default_splits": ([_i32], _i32),
    "pa_decode": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                   _f32, _i32, _i32, _i32, _i32, _vp, _sz, _u32, _vp], _i32),
    "pa_decode_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                       _i32, _i32, _f32, _i32, _i32, _i32, _i32, _vp, _sz, _u32, _vp], _i32),
    "pa_decode_step": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                        _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp, _sz, _u32, _vp], _i32),
    "pa_decode_step_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                            _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp, _sz, _u32,
                            _vp], _i32),
    "pa_decode_noalloc": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                           _i32, _i32, _f32, _i32, _i32, _i32, _i32, _u32, _vp], _i32),
    "pa_decode_step_synced": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                               _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp, _sz,
                               _u32, _vp, _vp], _i32),
    "pa_decode_step_fp8_synced": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                   _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32,
                                   _i32, _vp, _sz, _u32, _vp, _vp], _i32),
    "pa_decode_step_pipelined": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32,
                                  _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32,
                                  _vp, _sz, _u32, _vp, _vp, _vp], _i32),
    "pa_decode_step_fp8_pipelined": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                      _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                                      _i32, _i32, _vp, _sz, _u32, _vp, _vp, _vp], _i32),
    "pa_stream_write_value": ([_vp, _vp, _u32], _i32),
    "pa_stream_wait_value": ([_vp, _vp, _u32], _i32),
    "pa_get_status": ([_vp, ctypes.POINTER(ctypes.c_uint)], _i32),
    "pa_test_wait_timeout": ([ctypes.c_uint64, _vp], _i32),
    "pa_test_merge_timeout": ([_vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _sz,
                               ctypes.c_uint64, _vp], _i32),
}
# the entry points of include/pa_serving.h
SERVING_SIGNATURES = {
    "pa_rope": ([_vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_rope_append": ([_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                        _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_rope_append_fp8": ([_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                            _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_attention_weights_workspace_size": ([_i32, _i32, _i32, _i32, _i32], _sz),
    "pa_attention_weights": ([_vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                              _i32, _i32, _f32, _f32, _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "pa_attention_weights_fp8": ([_vp, _i64, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                  _i32, _i32, _i32, _f32, _f32, _i32, _i32, _i32, _vp, _sz, _vp],
                                 _i32),
    "pa_evict": ([_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _vp,
                  _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_evict_fp8": ([_vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i32, _vp, _i32,
                      _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_verify_drafts": ([_vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                          _vp], _i32),
}
# the entry points of include/pa_request.h
_PREFILL_TAIL = [_vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32,
                 _vp, _sz, _vp]
REQUEST_SIGNATURES = {
    "pa_prefill_workspace_size": ([_i32, _i32, _i32, _i32, _i32], _sz),
    "pa_prefill": ([_vp, _vp, _i64, _vp, _vp, *_PREFILL_TAIL], _i32),
    "pa_prefill_fp8": ([_vp, _vp, _i64, _vp, _vp, _vp, _vp, *_PREFILL_TAIL], _i32),
    "pa_alloc_pages": ([_vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp], _i32),
    "pa_free_pages": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp], _i32),
    "pa_fork_pages": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32,
                       _i32, _i32, _i32, _vp, _vp], _i32),
    "pa_compact_workspace_size": ([_i32], _sz),
    "pa_compact_pages": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                          _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "pa_process_logits": ([_vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
}
# the failure-path test of include/pa_request_test.h
REQUEST_TEST_SIGNATURES = {
    "pa_test_prefill_timeout": ([_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32,
                                 _i32, _i32, _i32, _f32, _i32, _i32, ctypes.c_uint64, _vp, _sz, _vp], _i32),
}
# the failure-path test of include/pa_serving_test.h
SERVING_TEST_SIGNATURES = {
    "pa_test_weights_timeout": ([_vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                 _i32, _f32, _i32, _i32, ctypes.c_uint64, _vp, _sz, _vp], _i32),
}

_lock = threading.Lock()
_lib = None


class PAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (code {code})")


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libpa.so (raising if it is absent, unless asked to build it)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                if not build_if_missing:
                    raise RuntimeError(f"{_build.LIB} is not built; call __graft_entry__.build() "
                                       "or python -m paged_kv_cache_179_gb300.build")
                _build.build()
            L = ctypes.CDLL(_build.LIB)
            for name, (args, res) in (*SIGNATURES.items(), *SERVING_SIGNATURES.items(),
                                      *REQUEST_SIGNATURES.items(),
                                      *REQUEST_TEST_SIGNATURES.items(),
                                      *SERVING_TEST_SIGNATURES.items()):
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def status_string(code: int) -> str:
    return load().pa_status_string(code).decode()


def _check(rc: int, where: str):
    if rc != PA_OK:
        raise PAError(rc, where)


class _Recording(threading.local):
    """Per-thread state of ``prepare``: while active, entry points record
    their C calls (with marshalled arguments) instead of making them."""
    active = False
    stream = None
    calls = None


_rec = _Recording()


def _call(fn, where: str, *args):
    if _rec.active:
        conv = []
        for t, a in zip(fn.argtypes, args):
            conv.append(a if a is None or isinstance(a, t) else t(a))
        _rec.calls.append((fn, tuple(conv), where))
        return
    _check(fn(*args), where)


class Prepared:
    """C-ABI calls recorded once, with their arguments already marshalled;
    calling the object makes them again, in order, on the recorded stream.
    Checking shapes, dtypes and devices and converting arguments is done
    once, at ``prepare``; the tensors must stay alive and in place."""

    def __init__(self, calls):
        self.calls = calls

    def __call__(self):
        for fn, args, where in self.calls:
            rc = fn(*args)
            if rc != PA_OK:
                raise PAError(rc, where)


def prepare(body, stream=None) -> Prepared:
    """Run ``body()`` (which calls entry points of this module) with every C
    call recorded instead of made, launching on ``stream`` (a
    torch.cuda.Stream; default: the current stream when the calls run).
    Returns the recorded calls as one callable: a serving loop that repeats
    a step on the same tensors pays the argument checks once."""
    if _rec.active:
        raise RuntimeError("prepare() does not nest")
    _rec.active = True
    _rec.stream = None if stream is None else ctypes.c_void_p(stream.cuda_stream)
    _rec.calls = []
    try:
        body()
        return Prepared(_rec.calls)
    finally:
        _rec.active, _rec.stream, _rec.calls = False, None, None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev) -> ctypes.c_void_p:
    if _rec.active and _rec.stream is not None:
        return _rec.stream
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, name, dtype=None, ndim=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, has {t.dim()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _flags(early_prologue: bool, early_copies: bool = False) -> int:
    if early_copies and not early_prologue:
        raise ValueError("early_copies needs early_prologue")
    return ((PA_DECODE_EARLY_PROLOGUE if early_prologue else 0) |
            (PA_DECODE_EARLY_COPIES if early_copies else 0))


def _act_code(dtype) -> int:
    if dtype == torch.float16:
        return PA_F16
    if dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"unsupported activation dtype {dtype}")


# ---------------------------------------------------------------- entry points
def pa_version() -> int:
    return load().pa_version()


def pa_cache_append(k_new, v_new, k_cache, v_cache, slot_mapping) -> None:
    """Scatter k_new/v_new [T][Hkv][D] into the pools [NB][Hkv][bs][D] at slot_mapping [T]."""
    dev = k_cache.device
    act = (torch.float16, torch.bfloat16)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, act, 3, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, k_new.dtype, 4, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    T, Hkv, D = k_new.shape
    NB, Hkv2, bs, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or v_new.shape != k_new.shape or v_cache.shape != k_cache.shape \
            or slot_mapping.shape[0] != T:
        raise ValueError("shape mismatch")
    _call(load().pa_cache_append, "pa_cache_append",
          _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), T, Hkv, D,
          bs, NB, _act_code(k_new.dtype), _stream(dev))


def pa_cache_append_fp8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, slot_mapping) -> None:
    """E4M3-encode fp16/bf16 k_new/v_new into uint8 pools: a page's first token
    sets its scales, a later token that would saturate re-scales the page."""
    dev = k_cache.device
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, (torch.float16, torch.bfloat16), 3, dev)
    _need(v_new, "v_new", k_new.dtype)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.uint8, 4, dev)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32, 2, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    T, Hkv, D = k_new.shape
    NB, _, bs, _ = k_cache.shape
    if k_scale.shape != (NB, Hkv) or v_scale.shape != (NB, Hkv) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    _call(load().pa_cache_append_fp8, "pa_cache_append_fp8",
          _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
          _ptr(slot_mapping), T, Hkv, D, bs, NB, _act_code(k_new.dtype), _stream(dev))


def pa_quantize_fp8(k_src, v_src, k_cache, v_cache, k_scale, v_scale) -> None:
    """Quantise fp16 pools [NB][Hkv][bs][D] into E4M3 pools and [NB][Hkv] fp32 scales."""
    ref = k_src if k_src is not None else v_src
    dev = ref.device
    NB, Hkv, bs, D = ref.shape
    for src, codes, sc, n in ((k_src, k_cache, k_scale, "k"), (v_src, v_cache, v_scale, "v")):
        if src is None:
            continue
        _need(src, n + "_src", torch.float16, 4, dev)
        _need(codes, n + "_cache", torch.uint8, 4, dev)
        _need(sc, n + "_scale", torch.float32, 2, dev)
        if src.shape != ref.shape or codes.shape != ref.shape or sc.shape != (NB, Hkv):
            raise ValueError("shape mismatch")
    _call(load().pa_quantize_fp8, "pa_quantize_fp8",
          _ptr(k_src), _ptr(v_src), _ptr(k_cache if k_src is not None else None),
          _ptr(v_cache if v_src is not None else None),
          _ptr(k_scale if k_src is not None else None),
          _ptr(v_scale if v_src is not None else None), NB, Hkv, D, bs, _stream(dev))


def pa_copy_blocks(k_cache, v_cache, block_mapping, k_scale=None, v_scale=None) -> None:
    """Copy whole physical blocks of both pools: block_mapping is int64
    [n][2] of (src, dst); E4M3 (uint8) pools also copy their [NB][Hkv] scales."""
    dev = k_cache.device
    fp8 = k_cache.dtype == torch.uint8
    _need(k_cache, "k_cache", (torch.float16, torch.bfloat16, torch.uint8), 4, dev)
    _need(v_cache, "v_cache", k_cache.dtype, 4, dev)
    _need(block_mapping, "block_mapping", torch.int64, 2, dev)
    NB, Hkv, bs, D = k_cache.shape
    if v_cache.shape != k_cache.shape or block_mapping.shape[1] != 2:
        raise ValueError("shape mismatch")
    if fp8:
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(t, n, torch.float32, 2, dev)
            if t.shape != (NB, Hkv):
                raise ValueError("shape mismatch")
        code = PA_E4M3
    else:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales are for E4M3 pools only")
        code = _act_code(k_cache.dtype)
    _call(load().pa_copy_blocks, "pa_copy_blocks",
          _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_mapping),
          block_mapping.shape[0], Hkv, D, bs, NB, code, _stream(dev))


def pa_e4m3_encode(x, codes) -> None:
    _need(x, "x", torch.float32, None)
    _need(codes, "codes", torch.uint8, None, x.device)
    if codes.numel() != x.numel():
        raise ValueError("size mismatch")
    _call(load().pa_e4m3_encode, "pa_e4m3_encode",
          _ptr(x), _ptr(codes), x.numel(), _stream(x.device))


def pa_decode_workspace_size(num_seqs, num_q_heads, head_dim, split_ctas=0) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, num_q_heads, head_dim, split_ctas))


def pa_decode_workspace_size_rows(num_seqs, num_q_heads, head_dim, split_ctas=0,
                                  query_rows=8) -> int:
    """Workspace bytes for calls with up to ``query_rows`` = queries_per_seq *
    (num_q_heads / num_kv_heads) query rows per (sequence, kv head)."""
    return int(load().pa_decode_workspace_size_rows(num_seqs, num_q_heads, head_dim, split_ctas,
                                                    query_rows))


def pa_decode_default_splits(pool_dtype=torch.float16) -> int:
    """CTAs a default (split_ctas=0) decode uses over pools of this dtype
    (torch.uint8 for E4M3 pools)."""
    code = PA_E4M3 if pool_dtype == torch.uint8 else _act_code(pool_dtype)
    return int(load().pa_decode_default_splits(code))


def alloc_workspace(num_seqs, num_q_heads, head_dim, split_ctas, device, query_rows=8):
    """Caller-owned workspace for pa_decode, zero-filled as the decode needs
    it (each call leaves it zero-filled again); ``query_rows``: the most
    query rows per (sequence, kv head) of the calls it serves (queries per
    sequence times the query group)."""
    n = pa_decode_workspace_size_rows(num_seqs, num_q_heads, head_dim, split_ctas, query_rows)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _decode_common(out, q, block_tables, context_lens, dev):
    """q/out [B][Hq][D], or [B][n_q][Hq][D] for n_q query tokens per sequence."""
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    if q.dim() == 3:
        (B, Hq, D), nq = q.shape, 1
    else:
        B, nq, Hq, D = q.shape
    if out.shape != q.shape or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch")
    return B, nq, Hq, D


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
              scale: float, split_ctas: int = 0, workspace=None, *, window: int = 0,
              early_prologue: bool = False, early_copies: bool = False) -> None:
    """out[b][hq] = softmax(scale q.K) V over each sequence's blocks (16-bit pools).
    early_prologue: PA_DECODE_EARLY_PROLOGUE (the kernel before this call on
    the stream must not write context_lens or block_tables).
    early_copies: PA_DECODE_EARLY_COPIES as well (the kernels before it must
    also write nothing in the pools except in each sequence's last two
    blocks, as the previous decode step of the same batch does)."""
    dev = q.device
    act = (torch.float16, torch.bfloat16)
    _need(q, "q", act, None, dev)
    _need(out, "out", q.dtype, None, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, q.dtype, 4, dev)
    B, nq, Hq, D = _decode_common(out, q, block_tables, context_lens, dev)
    NB, Hkv, bs, _ = k_cache.shape
    ws_bytes = 0
    if workspace is not None:
        _need(workspace, "workspace", None, None, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    _call(load().pa_decode, "pa_decode",
          _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
          block_tables.shape[1], _ptr(context_lens), int(max_context_len), B, Hq, Hkv, D, bs, NB,
          float(scale), int(window), nq, _act_code(q.dtype), int(split_ctas), _ptr(workspace),
          ws_bytes, _flags(early_prologue, early_copies), _stream(dev))


def pa_decode_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                  max_context_len: int, scale: float, split_ctas: int = 0, workspace=None, *,
                  window: int = 0, early_prologue: bool = False, early_copies: bool = False) -> None:
    """As pa_decode over E4M3 pools with per-(block, kv head) fp32 scales; q/out
    fp16 or bf16."""
    dev = q.device
    _need(q, "q", (torch.float16, torch.bfloat16), None, dev)
    _need(out, "out", q.dtype, None, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.uint8, 4, dev)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32, 2, dev)
    B, nq, Hq, D = _decode_common(out, q, block_tables, context_lens, dev)
    NB, Hkv, bs, _ = k_cache.shape
    ws_bytes = 0
    if workspace is not None:
        _need(workspace, "workspace", None, None, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    _call(load().pa_decode_fp8, "pa_decode_fp8",
          _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
          _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), int(max_context_len), B,
          Hq, Hkv, D, bs, NB, float(scale), int(window), nq, _act_code(q.dtype), int(split_ctas),
          _ptr(workspace), ws_bytes, _flags(early_prologue, early_copies), _stream(dev))


class StepSync(ctypes.Structure):
    """pa_step_sync: the device words and values of one step's handshake with
    the copies on other streams (see include/pa.h).  The entry points read
    the values when they are called, so a bound call sees updated values."""
    _fields_ = [("ready", ctypes.c_void_p), ("done", ctypes.c_void_p),
                ("done_count", ctypes.c_void_p), ("ready_value", ctypes.c_uint32),
                ("done_value", ctypes.c_uint32)]


class StepCopies(ctypes.Structure):
    """pa_step_copies: the host<->device copies of one pipelined step (see
    include/pa.h); ``slot_reused`` is read at each call."""
    _fields_ = [("host_in", ctypes.c_void_p), ("dev_in", ctypes.c_void_p),
                ("in_bytes", ctypes.c_size_t), ("dev_out", ctypes.c_void_p),
                ("host_out", ctypes.c_void_p), ("out_bytes", ctypes.c_size_t),
                ("copy_stream", ctypes.c_void_p), ("back_stream", ctypes.c_void_p),
                ("reuse_event", ctypes.c_void_p), ("slot_reused", ctypes.c_int)]


def _sync_ptr(sync):
    return ctypes.c_void_p(ctypes.addressof(sync))


def pa_stream_write_value(word, value: int, stream=None) -> None:
    """Stream-ordered store of ``value`` into the device int32 tensor element
    ``word`` (a 1-element view) on ``stream`` (default: the current stream)."""
    _need(word, "word", (torch.int32,), None)
    s = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(word.device)
    _call(load().pa_stream_write_value, "pa_stream_write_value", s, _ptr(word),
          int(value) & 0xffffffff)


def pa_stream_wait_value(word, value: int, stream=None) -> None:
    """Hold ``stream``'s later work until the device word reaches ``value``
    (cyclic 32-bit comparison)."""
    _need(word, "word", (torch.int32,), None)
    s = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(word.device)
    _call(load().pa_stream_wait_value, "pa_stream_wait_value", s, _ptr(word),
          int(value) & 0xffffffff)


def _ws_bytes(workspace, dev):
    if workspace is None:
        return 0
    _need(workspace, "workspace", None, None, dev)
    return workspace.numel() * workspace.element_size()


def pa_decode_step(out, q, k_new, v_new, k_cache, v_cache, slot_mapping, block_tables,
                   context_lens, max_context_len: int, scale: float, split_ctas: int = 0,
                   workspace=None, *, window: int = 0, early_prologue: bool = False, early_copies: bool = False,
                   sync: StepSync = None, copies: StepCopies = None) -> None:
    """Append k_new/v_new at slot_mapping, then decode, in one launch (16-bit
    pools); with ``sync``, pa_decode_step_synced (device-side handshake); with
    ``copies`` too, pa_decode_step_pipelined (the step's upload and read-back
    in the same call)."""
    dev = q.device
    act = (torch.float16, torch.bfloat16)
    _need(q, "q", act, 3, dev)
    _need(out, "out", q.dtype, 3, dev)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, q.dtype, 3, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, q.dtype, 4, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    B, nq, Hq, D = _decode_common(out, q, block_tables, context_lens, dev)
    if nq != 1:
        raise ValueError("the fused step takes one query token per sequence")
    NB, Hkv, bs, _ = k_cache.shape
    if k_new.shape != (B, Hkv, D) or v_new.shape != k_new.shape or slot_mapping.shape[0] != B:
        raise ValueError("shape mismatch")
    args = (_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
            _ptr(slot_mapping), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
            int(max_context_len), B, Hq, Hkv, D, bs, NB, float(scale), int(window),
            _act_code(q.dtype), int(split_ctas), _ptr(workspace), _ws_bytes(workspace, dev),
            _flags(early_prologue, early_copies))
    if sync is None:
        _call(load().pa_decode_step, "pa_decode_step", *args, _stream(dev))
    elif copies is None:
        _call(load().pa_decode_step_synced, "pa_decode_step_synced", *args, _sync_ptr(sync),
              _stream(dev))
    else:
        _call(load().pa_decode_step_pipelined, "pa_decode_step_pipelined", *args,
              _sync_ptr(sync), _sync_ptr(copies), _stream(dev))


def pa_decode_step_fp8(out, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                       block_tables, context_lens, max_context_len: int, scale: float,
                       split_ctas: int = 0, workspace=None, *, window: int = 0,
                       early_prologue: bool = False, early_copies: bool = False, sync: StepSync = None,
                       copies: StepCopies = None) -> None:
    """Append (E4M3-encode) k_new/v_new, then decode over the E4M3 pools, in one
    attention launch; q, k_new, v_new and out share one dtype (fp16 or bf16)."""
    dev = q.device
    _need(q, "q", (torch.float16, torch.bfloat16), 3, dev)
    for t, n in ((out, "out"), (k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, q.dtype, 3, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.uint8, 4, dev)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32, 2, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    B, nq, Hq, D = _decode_common(out, q, block_tables, context_lens, dev)
    if nq != 1:
        raise ValueError("the fused step takes one query token per sequence")
    NB, Hkv, bs, _ = k_cache.shape
    if k_new.shape != (B, Hkv, D) or v_new.shape != k_new.shape or slot_mapping.shape[0] != B:
        raise ValueError("shape mismatch")
    args = (_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
            _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping), _ptr(block_tables),
            block_tables.shape[1], _ptr(context_lens), int(max_context_len), B, Hq, Hkv, D, bs, NB,
            float(scale), int(window), _act_code(q.dtype), int(split_ctas), _ptr(workspace),
            _ws_bytes(workspace, dev), _flags(early_prologue, early_copies))
    if sync is None:
        _call(load().pa_decode_step_fp8, "pa_decode_step_fp8", *args, _stream(dev))
    elif copies is None:
        _call(load().pa_decode_step_fp8_synced, "pa_decode_step_fp8_synced", *args,
              _sync_ptr(sync), _stream(dev))
    else:
        _call(load().pa_decode_step_fp8_pipelined, "pa_decode_step_fp8_pipelined", *args,
              _sync_ptr(sync), _sync_ptr(copies), _stream(dev))


def pa_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens,
                      max_context_len: int, scale: float, split_ctas: int = 0,
                      window: int = 0, early_prologue: bool = False, early_copies: bool = False) -> None:
    """pa_decode with the library's static scratch instead of a workspace (allocates nothing)."""
    dev = q.device
    act = (torch.float16, torch.bfloat16)
    _need(q, "q", act, None, dev)
    _need(out, "out", q.dtype, None, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, q.dtype, 4, dev)
    B, nq, Hq, D = _decode_common(out, q, block_tables, context_lens, dev)
    NB, Hkv, bs, _ = k_cache.shape
    _call(load().pa_decode_noalloc, "pa_decode_noalloc",
          _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
          block_tables.shape[1], _ptr(context_lens), int(max_context_len), B, Hq, Hkv, D, bs, NB,
          float(scale), int(window), nq, _act_code(q.dtype), int(split_ctas),
          _flags(early_prologue, early_copies), _stream(dev))


def pa_test_wait_timeout(limit_ns: int, device=None) -> None:
    """Failure-path test: one warp's bounded mbarrier wait on a barrier that
    nothing completes gives up after ``limit_ns`` and sets PA_STATUS_TIMEOUT."""
    _call(load().pa_test_wait_timeout, "pa_test_wait_timeout", int(limit_ns),
          _stream(device or torch.cuda.current_device()))


def pa_test_merge_timeout(out, context_lens, max_context_len: int, num_kv_heads: int,
                          split_ctas: int, workspace, limit_ns: int) -> None:
    """Failure-path test: pa_decode's merge launch alone (nothing writes the
    partials it polls for) gives up after ``limit_ns`` and sets
    PA_STATUS_TIMEOUT.  out [B][Hq][D] as for pa_decode."""
    dev = out.device
    _need(out, "out", (torch.float16, torch.bfloat16), 3, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = out.shape
    _call(load().pa_test_merge_timeout, "pa_test_merge_timeout",
          _ptr(out), _ptr(context_lens), int(max_context_len), B, Hq, int(num_kv_heads), D,
          _act_code(out.dtype), int(split_ctas), _ptr(workspace), _ws_bytes(workspace, dev),
          int(limit_ns), _stream(dev))


def pa_get_status(device=None) -> tuple[int, int]:
    """(return code, raw status bits) after synchronising the current stream."""
    bits = ctypes.c_uint(0)
    rc = load().pa_get_status(_stream(device or torch.cuda.current_device()), ctypes.byref(bits))
    return rc, bits.value


# ------------------------------------------- around the decode step (pa_serving.h)
def _here(dev):
    """The tensors of a call must be on the current device (its streams and kernels are)."""
    if dev.type == "cuda" and dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _rows(t, name, dtype, device):
    """Checks a [T][H][D] tensor whose tokens may lie apart (a view of a wider
    projection) but whose heads are dense; returns the elements from one token
    to the next."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, has {t.dim()}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    T, H, D = t.shape
    if t.numel() and ((D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D)):
        raise ValueError(f"{name}: each token's heads must be contiguous")
    return t.stride(0) if T > 1 else H * D


class _RopeStruct(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("freq_axis", ctypes.c_void_p),
                ("num_axes", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("adjacent", ctypes.c_int), ("amplitude", ctypes.c_float)]


class RopeSpec:
    """A rotation (pa_rope_spec): ``inv_freq[i]`` radians per position of pair
    i, ``freq_axis[i]`` the axis of the positions it turns with (None: one
    axis), pairs (i, i + rotary_dim / 2) or, ``adjacent``, (2i, 2i + 1);
    rotary_dim is twice the number of frequencies.  Made once and kept."""

    def __init__(self, inv_freq, freq_axis=None, *, adjacent=False, amplitude=1.0, num_axes=None):
        self.inv_freq = np.ascontiguousarray(inv_freq, dtype=np.float64).reshape(-1).copy()
        self.freq_axis = None if freq_axis is None else \
            np.ascontiguousarray(freq_axis, dtype=np.int32).reshape(-1).copy()
        if self.freq_axis is not None and self.freq_axis.shape != self.inv_freq.shape:
            raise ValueError("freq_axis and inv_freq must have one entry per pair")
        if num_axes is None:
            num_axes = 1 if freq_axis is None or not self.freq_axis.size \
                else int(self.freq_axis.max()) + 1
        self.num_axes, self.rotary_dim = int(num_axes), 2 * self.inv_freq.size
        self.struct = _RopeStruct(self.inv_freq.ctypes.data,
                                  None if self.freq_axis is None else self.freq_axis.ctypes.data,
                                  self.num_axes, self.rotary_dim, int(bool(adjacent)),
                                  float(amplitude))
        self.pointer = ctypes.c_void_p(ctypes.addressof(self.struct))
        self.pointer.owner = self      # a recorded call keeps the specification alive


def _positions(positions, spec, T, dev):
    if not isinstance(spec, RopeSpec):
        raise TypeError("spec must be a RopeSpec")
    _need(positions, "positions", torch.int32, None, dev)
    if tuple(positions.shape) not in ((spec.num_axes, T),) + (((T,),) if spec.num_axes == 1 else ()):
        raise ValueError(f"positions must be [{spec.num_axes}][{T}]")


def pa_rope(q_out, q, k_out, k, positions, spec: RopeSpec) -> None:
    """Rotate q [T][Hq][D] into q_out and k [T][Hkv][D] into k_out (either pair
    may be None) by positions int32 [axes][T]; q and k may be views of one
    projection, or the outputs themselves (in place)."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    dev = ref.device
    act = (torch.float16, torch.bfloat16)
    strides, heads = [0, 0], [0, 0]
    for i, (o, t, n) in enumerate(((q_out, q, "q"), (k_out, k, "k"))):
        if (o is None) != (t is None):
            raise ValueError(f"{n} and {n}_out go together")
        if t is None:
            continue
        strides[i] = _rows(t, n, act if t is ref else ref.dtype, dev)
        _need(o, n + "_out", ref.dtype, 3, dev)
        if o.shape != t.shape or t.shape[0] != ref.shape[0] or t.shape[2] != ref.shape[2]:
            raise ValueError("shape mismatch")
        heads[i] = t.shape[1]
    T, _, D = ref.shape
    _positions(positions, spec, T, dev)
    _here(dev)
    _call(load().pa_rope, "pa_rope", _ptr(q_out), _ptr(q), strides[0], _ptr(k_out), _ptr(k),
          strides[1], _ptr(positions), spec.pointer, T, heads[0], heads[1], D,
          _act_code(ref.dtype), _stream(dev))


def _rope_append_args(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions, spec,
                      pool_dtype):
    dev = k_cache.device
    sq = _rows(q, "q", (torch.float16, torch.bfloat16), dev)
    sk, sv = _rows(k_new, "k_new", q.dtype, dev), _rows(v_new, "v_new", q.dtype, dev)
    _need(q_out, "q_out", q.dtype, 3, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, pool_dtype or q.dtype, 4, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    T, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    if q_out.shape != q.shape or k_new.shape != (T, Hkv, D) or v_new.shape != k_new.shape \
            or v_cache.shape != k_cache.shape or D2 != D or slot_mapping.shape[0] != T:
        raise ValueError("shape mismatch")
    _positions(positions, spec, T, dev)
    _here(dev)
    return (_ptr(q_out), _ptr(q), sq, _ptr(k_new), sk, _ptr(v_new), sv, _ptr(k_cache),
            _ptr(v_cache)), (_ptr(slot_mapping), _ptr(positions), spec.pointer, T, Hq, Hkv, D, bs,
                             NB, _act_code(q.dtype), _stream(dev))


def pa_rope_append(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions,
                   spec: RopeSpec) -> None:
    """pa_rope then pa_cache_append in one launch: q rotated into q_out, k
    rotated into k_cache and v copied into v_cache at slot_mapping."""
    a, b = _rope_append_args(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions,
                             spec, None)
    _call(load().pa_rope_append, "pa_rope_append", *a, *b)


def pa_rope_append_fp8(q_out, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                       positions, spec: RopeSpec) -> None:
    """pa_rope then pa_cache_append_fp8 in one launch."""
    a, b = _rope_append_args(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions,
                             spec, torch.uint8)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32, 2, k_cache.device)
        if t.shape != k_cache.shape[:2]:
            raise ValueError("shape mismatch")
    _call(load().pa_rope_append_fp8, "pa_rope_append_fp8", *a, _ptr(k_scale), _ptr(v_scale), *b)


def pa_attention_weights_workspace_size(num_seqs, num_q_heads, num_kv_heads, max_context_len,
                                        queries_per_seq=1) -> int:
    return int(load().pa_attention_weights_workspace_size(
        int(num_seqs), int(num_q_heads), int(num_kv_heads), int(max_context_len),
        int(queries_per_seq)))


def alloc_weights_workspace(num_seqs, num_q_heads, num_kv_heads, max_context_len,
                            queries_per_seq, device):
    """Caller-owned workspace for pa_attention_weights, zero-filled as it needs
    to be before its first use."""
    n = pa_attention_weights_workspace_size(num_seqs, num_q_heads, num_kv_heads, max_context_len,
                                            queries_per_seq)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _weights_args(weights, q, k_cache, block_tables, context_lens, pool_dtype, dev):
    _need(q, "q", (torch.float16, torch.bfloat16), None, dev)
    _need(weights, "weights", torch.float32, 3, dev)
    _need(k_cache, "k_cache", pool_dtype or q.dtype, 4, dev)
    B, nq, Hq, D = _decode_common(q, q, block_tables, context_lens, dev)
    NB, Hkv, bs, D2 = k_cache.shape
    if weights.shape[:2] != (B, Hkv) or D2 != D:
        raise ValueError("shape mismatch")
    _here(dev)
    return B, nq, Hq, Hkv, D, bs, NB


def pa_attention_weights(weights, q, k_cache, block_tables, context_lens, max_context_len: int,
                         scale: float, workspace, *, decay: float = 1.0,
                         fresh_tokens: int = 0) -> None:
    """weights[b][h][t] = decay * weights + the softmax weights that q's rows
    give token t (0 in the old one's place for the last fresh_tokens tokens).
    weights fp32 [B][Hkv][n >= max_context_len]; q [B][Hq][D] or [B][n_q][Hq][D]."""
    dev = q.device
    B, nq, Hq, Hkv, D, bs, NB = _weights_args(weights, q, k_cache, block_tables, context_lens,
                                              None, dev)
    _call(load().pa_attention_weights, "pa_attention_weights", _ptr(weights), weights.shape[2],
          _ptr(q), _ptr(k_cache), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
          int(max_context_len), B, Hq, Hkv, D, bs, NB, float(scale), float(decay),
          int(fresh_tokens), nq, _act_code(q.dtype), _ptr(workspace), _ws_bytes(workspace, dev),
          _stream(dev))


def pa_attention_weights_fp8(weights, q, k_cache, k_scale, block_tables, context_lens,
                             max_context_len: int, scale: float, workspace, *,
                             decay: float = 1.0, fresh_tokens: int = 0) -> None:
    """As pa_attention_weights over an E4M3 pool with [NB][Hkv] scales."""
    dev = q.device
    B, nq, Hq, Hkv, D, bs, NB = _weights_args(weights, q, k_cache, block_tables, context_lens,
                                              torch.uint8, dev)
    _need(k_scale, "k_scale", torch.float32, 2, dev)
    if k_scale.shape != (NB, Hkv):
        raise ValueError("shape mismatch")
    _call(load().pa_attention_weights_fp8, "pa_attention_weights_fp8", _ptr(weights),
          weights.shape[2], _ptr(q), _ptr(k_cache), _ptr(k_scale), _ptr(block_tables),
          block_tables.shape[1], _ptr(context_lens), int(max_context_len), B, Hq, Hkv, D, bs, NB,
          float(scale), float(decay), int(fresh_tokens), nq, _act_code(q.dtype), _ptr(workspace),
          _ws_bytes(workspace, dev), _stream(dev))


def pa_test_weights_timeout(weights, q, k_cache, block_tables, context_lens, max_context_len: int,
                            scale: float, workspace, *, silent_warp: int, limit_ns: int) -> None:
    """Failure-path test: pa_attention_weights (q [B][Hq][D], decay 0) whose warp
    ``silent_warp`` announces nothing, so that those who wait for it give up after
    ``limit_ns``, set PA_STATUS_TIMEOUT and leave their weights as they were."""
    dev = q.device
    B, nq, Hq, Hkv, D, bs, NB = _weights_args(weights, q, k_cache, block_tables, context_lens,
                                              None, dev)
    if nq != 1 or bs != 16:
        raise ValueError("one query token and blocks of 16 tokens")
    _call(load().pa_test_weights_timeout, "pa_test_weights_timeout", _ptr(weights),
          weights.shape[2], _ptr(q), _ptr(k_cache), _ptr(block_tables), block_tables.shape[1],
          _ptr(context_lens), int(max_context_len), B, Hq, Hkv, D, NB, float(scale),
          _act_code(q.dtype), int(silent_warp), int(limit_ns), _ptr(workspace),
          _ws_bytes(workspace, dev), _stream(dev))


def _evict_args(k_cache, v_cache, weights, weights_out, block_tables, context_lens,
                max_context_len, spare_tables, tables_out, new_lens, kept, dtype):
    dev = k_cache.device
    _need(k_cache, "k_cache", dtype, 4, dev)
    _need(v_cache, "v_cache", k_cache.dtype, 4, dev)
    _need(weights, "weights", torch.float32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    _need(spare_tables, "spare_tables", torch.int32, 2, dev)
    _need(new_lens, "new_lens", torch.int32, 1, dev)
    _need(kept, "kept", torch.int32, 3, dev)
    B, (NB, Hkv, bs, D) = block_tables.shape[0], k_cache.shape
    if v_cache.shape != k_cache.shape or weights.shape[:2] != (B, Hkv) or \
            kept.shape[:2] != (B, Hkv) or context_lens.shape[0] != B or \
            spare_tables.shape[0] != B or new_lens.shape[0] != B:
        raise ValueError("shape mismatch")
    if weights_out is not None:
        _need(weights_out, "weights_out", torch.float32, 3, dev)
        if weights_out.shape[:2] != (B, Hkv):
            raise ValueError("shape mismatch")
    if tables_out is not None:
        _need(tables_out, "tables_out", torch.int32, 2, dev)
        if tables_out.shape != spare_tables.shape:
            raise ValueError("shape mismatch")
    _here(dev)
    keep = kept.shape[2]
    return (_ptr(weights), weights.shape[2], _ptr(weights_out),
            0 if weights_out is None else weights_out.shape[2], _ptr(block_tables),
            block_tables.shape[1], _ptr(context_lens), int(max_context_len), _ptr(spare_tables),
            spare_tables.shape[1], _ptr(tables_out), _ptr(new_lens), _ptr(kept), B, Hkv, D, bs,
            NB, keep)


def pa_evict(k_cache, v_cache, weights, weights_out, block_tables, context_lens,
             max_context_len: int, spare_tables, tables_out, new_lens, kept, *,
             first_tokens: int = 0, recent_tokens: int = 0) -> None:
    """Cut each sequence with more than keep = kept.shape[2] tokens to the first
    first_tokens, the last recent_tokens and the heaviest of the rest, moved
    into the blocks of spare_tables; weights_out and tables_out may be None."""
    a = _evict_args(k_cache, v_cache, weights, weights_out, block_tables, context_lens,
                    max_context_len, spare_tables, tables_out, new_lens, kept,
                    (torch.float16, torch.bfloat16))
    _call(load().pa_evict, "pa_evict", _ptr(k_cache), _ptr(v_cache), *a, int(first_tokens),
          int(recent_tokens), _act_code(k_cache.dtype), _stream(k_cache.device))


def pa_evict_fp8(k_cache, v_cache, k_scale, v_scale, weights, weights_out, block_tables,
                 context_lens, max_context_len: int, spare_tables, tables_out, new_lens, kept, *,
                 first_tokens: int = 0, recent_tokens: int = 0) -> None:
    """As pa_evict over E4M3 pools: a page that is written gets the scale of the
    rows it now holds."""
    a = _evict_args(k_cache, v_cache, weights, weights_out, block_tables, context_lens,
                    max_context_len, spare_tables, tables_out, new_lens, kept, torch.uint8)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32, 2, k_cache.device)
        if t.shape != k_cache.shape[:2]:
            raise ValueError("shape mismatch")
    _call(load().pa_evict_fp8, "pa_evict_fp8", _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
          _ptr(v_scale), *a, int(first_tokens), int(recent_tokens), _stream(k_cache.device))


def _prob_rows(t, name, dtype, dev, rows):
    """Checks [B][rows][V] probabilities whose rows may be padded; the row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 3 or t.shape[1] != rows:
        raise ValueError(f"{name} must be [num_seqs][{rows}][vocab_size]")
    B, n, V = t.shape
    row = t.stride(1) if n > 1 else t.stride(0) if B > 1 else V
    if t.numel() and ((V > 1 and t.stride(2) != 1) or (B > 1 and t.stride(0) != n * row)):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
    return row


def pa_verify_drafts(out_tokens, num_accepted, target_probs, draft_probs, draft_tokens, uniforms,
                     *, num_drafts=None) -> None:
    """Accept the drafts draft_tokens int32 [B][n] in order while uniforms[b][i]
    * q_i(x_i) < p_i(x_i), then draw one more token; p = target_probs
    [B][n + 1][V], q = draft_probs [B][n][V] or None (drafts without
    probabilities), fp32, fp16 or bf16; uniforms fp32 [B][n + 1].  out_tokens
    int32 [B][n + 1] (-1 behind the drawn token), num_accepted int32 [B];
    num_drafts int32 [B]: how many drafts each sequence has (None: all n)."""
    dev = target_probs.device
    codes = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}
    if target_probs.dtype not in codes:
        raise TypeError(f"unsupported probability dtype {target_probs.dtype}")
    _need(out_tokens, "out_tokens", torch.int32, 2, dev)
    _need(num_accepted, "num_accepted", torch.int32, 1, dev)
    _need(draft_tokens, "draft_tokens", torch.int32, 2, dev)
    _need(uniforms, "uniforms", torch.float32, 2, dev)
    B, n = draft_tokens.shape
    ps = _prob_rows(target_probs, "target_probs", target_probs.dtype, dev, n + 1)
    V, qs = target_probs.shape[2], 0
    if draft_probs is not None:
        qs = _prob_rows(draft_probs, "draft_probs", target_probs.dtype, dev, n)
        if draft_probs.shape != (B, n, V):
            raise ValueError("shape mismatch")
    if num_drafts is not None:
        _need(num_drafts, "num_drafts", torch.int32, 1, dev)
        if num_drafts.shape[0] != B:
            raise ValueError("shape mismatch")
    if target_probs.shape[0] != B or out_tokens.shape != (B, n + 1) or \
            uniforms.shape != (B, n + 1) or num_accepted.shape[0] != B:
        raise ValueError("shape mismatch")
    _here(dev)
    _call(load().pa_verify_drafts, "pa_verify_drafts", _ptr(out_tokens), _ptr(num_accepted),
          _ptr(target_probs), ps, _ptr(draft_probs), qs, _ptr(draft_tokens), _ptr(num_drafts),
          _ptr(uniforms), B, n, V, codes[target_probs.dtype], _stream(dev))


# ------------------------------------------------- whole requests (pa_request.h)
def pa_prefill_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(load().pa_prefill_workspace_size(int(num_seqs), int(num_tokens), int(num_q_heads),
                                                int(num_kv_heads), int(head_dim)))


def alloc_prefill_workspace(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, device):
    """Caller-owned workspace for pa_prefill calls of up to these sizes (of any contents)."""
    n = pa_prefill_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _prefill_args(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                  query_starts, scale, workspace, window, pool_dtype, scales):
    dev = k_cache.device
    sq = _rows(q, "q", (torch.float16, torch.bfloat16), dev)
    _need(out, "out", q.dtype, 3, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, pool_dtype or q.dtype, 4, dev)
    for t, n in zip(scales, ("k_scale", "v_scale")):
        _need(t, n, torch.float32, 2, dev)
        if t.shape != k_cache.shape[:2]:
            raise ValueError("shape mismatch")
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    _need(query_starts, "query_starts", torch.int32, 1, dev)
    T, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    B = block_tables.shape[0]
    if out.shape != q.shape or v_cache.shape != k_cache.shape or D2 != D or \
            context_lens.shape[0] != B or query_starts.shape[0] != B + 1:
        raise ValueError("shape mismatch")
    _here(dev)
    return ((_ptr(out), _ptr(q), sq, _ptr(k_cache), _ptr(v_cache), *(_ptr(t) for t in scales)),
            (_ptr(block_tables), block_tables.shape[1], _ptr(context_lens), int(max_context_len),
             _ptr(query_starts), T, B, Hq, Hkv, D, bs, NB, float(scale), int(window),
             _act_code(q.dtype), _ptr(workspace), _ws_bytes(workspace, dev), _stream(dev)))


def pa_prefill(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
               query_starts, scale: float, workspace, *, window: int = 0) -> None:
    """out [T][Hq][D]: the causal attention of each sequence's last query tokens,
    q[query_starts[b]:query_starts[b + 1]] (int32 [B + 1]; any number, 0 too), over
    its cached context, their own keys and values included (16-bit pools).  q may be a
    view of one projection.  window: the last so many positions only (0: all)."""
    a, b = _prefill_args(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                         query_starts, scale, workspace, window, None, ())
    _call(load().pa_prefill, "pa_prefill", *a, *b)


def pa_prefill_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   max_context_len: int, query_starts, scale: float, workspace, *,
                   window: int = 0) -> None:
    """As pa_prefill over E4M3 pools with [NB][Hkv] scales."""
    a, b = _prefill_args(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                         query_starts, scale, workspace, window, torch.uint8, (k_scale, v_scale))
    _call(load().pa_prefill_fp8, "pa_prefill_fp8", *a, *b)


def pa_test_prefill_timeout(out, q, k_cache, v_cache, block_tables, context_lens,
                            max_context_len: int, query_starts, scale: float, workspace, *,
                            drop_tile: int, limit_ns: int) -> None:
    """Failure-path test: pa_prefill whose CTAs wait for keys that are never copied (tile
    ``drop_tile`` of each), give up after ``limit_ns`` and set PA_STATUS_TIMEOUT."""
    a, b = _prefill_args(out, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                         query_starts, scale, workspace, 0, None, ())
    tables, mbs, lens, mx, starts, T, B, Hq, Hkv, D, bs, NB, sc, _, dtype, ws, n, stream = b
    if bs != 16:
        raise ValueError("blocks of 16 tokens")
    _call(load().pa_test_prefill_timeout, "pa_test_prefill_timeout", *a, tables, mbs, lens, mx, starts,
          T, B, Hq, Hkv, D, NB, sc, dtype, int(drop_tile), int(limit_ns), ws, n, stream)


def _page_state(block_tables, num_pages, ref_counts):
    dev = block_tables.device
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(num_pages, "num_pages", torch.int32, 1, dev)
    _need(ref_counts, "ref_counts", torch.int32, 1, dev)
    if num_pages.shape[0] != block_tables.shape[0]:
        raise ValueError("shape mismatch")
    _here(dev)
    return dev


def _items(dev, n, **tensors):
    for name, t in tensors.items():
        _need(t, name, torch.int32, 1, dev)
        if t.shape[0] != n:
            raise ValueError("shape mismatch")


def pa_alloc_pages(block_tables, num_pages, rows, new_lens, ref_counts, granted) -> None:
    """Give each row of ``rows`` the pages that new_lens tokens need, the lowest
    free ones (ref_counts [NB] 0) first; granted[i] 0 where the pool did not hold
    enough for it or one before it.  All int32, all kept on the device."""
    dev = _page_state(block_tables, num_pages, ref_counts)
    _items(dev, rows.shape[0], rows=rows, new_lens=new_lens, granted=granted)
    _call(load().pa_alloc_pages, "pa_alloc_pages", _ptr(block_tables), block_tables.shape[1],
          _ptr(num_pages), block_tables.shape[0], _ptr(rows), _ptr(new_lens), rows.shape[0],
          _ptr(ref_counts), ref_counts.shape[0], 16, _ptr(granted), _stream(dev))


def pa_free_pages(block_tables, num_pages, rows, ref_counts) -> None:
    """The pages of each row of ``rows`` lose one owner; the row is empty afterwards."""
    dev = _page_state(block_tables, num_pages, ref_counts)
    _items(dev, rows.shape[0], rows=rows)
    _call(load().pa_free_pages, "pa_free_pages", _ptr(block_tables), block_tables.shape[1],
          _ptr(num_pages), block_tables.shape[0], _ptr(rows), rows.shape[0], _ptr(ref_counts),
          ref_counts.shape[0], _stream(dev))


def _page_pools(k_cache, v_cache, k_scale, v_scale, dev, NB):
    fp8 = k_cache.dtype == torch.uint8
    _need(k_cache, "k_cache", (torch.float16, torch.bfloat16, torch.uint8), 4, dev)
    _need(v_cache, "v_cache", k_cache.dtype, 4, dev)
    if v_cache.shape != k_cache.shape or k_cache.shape[0] != NB:
        raise ValueError("shape mismatch")
    if not fp8 and (k_scale is not None or v_scale is not None):
        raise ValueError("scales are for E4M3 pools only")
    if fp8:
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(t, n, torch.float32, 2, dev)
            if t.shape != k_cache.shape[:2]:
                raise ValueError("shape mismatch")
    _, Hkv, bs, D = k_cache.shape
    return Hkv, D, bs, PA_E4M3 if fp8 else _act_code(k_cache.dtype)


def pa_fork_pages(k_cache, v_cache, block_tables, num_pages, context_lens, src_rows, dst_rows,
                  ref_counts, granted, *, k_scale=None, v_scale=None) -> None:
    """Make row dst_rows[i] a fork of row src_rows[i]: the full pages shared, a
    part-full last one copied to a free page, the context length taken over."""
    dev = _page_state(block_tables, num_pages, ref_counts)
    shape = _page_pools(k_cache, v_cache, k_scale, v_scale, dev, ref_counts.shape[0])
    _items(dev, block_tables.shape[0], context_lens=context_lens)
    _items(dev, src_rows.shape[0], src_rows=src_rows, dst_rows=dst_rows, granted=granted)
    _call(load().pa_fork_pages, "pa_fork_pages", _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
          _ptr(v_scale), _ptr(block_tables), block_tables.shape[1], _ptr(num_pages),
          _ptr(context_lens), block_tables.shape[0], _ptr(src_rows), _ptr(dst_rows),
          src_rows.shape[0], _ptr(ref_counts), ref_counts.shape[0], *shape, _ptr(granted),
          _stream(dev))


def pa_compact_workspace_size(num_blocks) -> int:
    return int(load().pa_compact_workspace_size(int(num_blocks)))


def alloc_compact_workspace(num_blocks, device):
    """Caller-owned workspace for pa_compact_pages of a pool of num_blocks pages."""
    return torch.empty(max(pa_compact_workspace_size(num_blocks), 256), dtype=torch.uint8,
                       device=device)


def pa_compact_pages(k_cache, v_cache, block_tables, num_pages, ref_counts, tables_out,
                     ref_counts_out, moved_to, num_live, workspace, *, k_scale=None,
                     v_scale=None) -> None:
    """Move the live pages together at the front of the pool; tables_out and
    ref_counts_out (which may be the inputs) hold the new ids and counts, moved_to
    [NB] where each page went (-1: it was free), num_live [1] how many there are."""
    dev = _page_state(block_tables, num_pages, ref_counts)
    NB = ref_counts.shape[0]
    shape = _page_pools(k_cache, v_cache, k_scale, v_scale, dev, NB)
    _need(tables_out, "tables_out", torch.int32, 2, dev)
    if tables_out.shape != block_tables.shape:
        raise ValueError("shape mismatch")
    _items(dev, NB, ref_counts_out=ref_counts_out, moved_to=moved_to)
    _items(dev, 1, num_live=num_live)
    _call(load().pa_compact_pages, "pa_compact_pages", _ptr(k_cache), _ptr(v_cache),
          _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), block_tables.shape[1],
          _ptr(num_pages), block_tables.shape[0], _ptr(ref_counts), NB, *shape,
          _ptr(tables_out), _ptr(ref_counts_out), _ptr(moved_to), _ptr(num_live),
          _ptr(workspace), _ws_bytes(workspace, dev), _stream(dev))


class _LogitsStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "history", "history_lens", "prompt_lens", "draft_tokens", "repetition", "presence",
        "frequency", "temperature", "bias_tokens", "bias_values", "allowed")] + [
        ("history_stride", ctypes.c_int64), ("allowed_stride", ctypes.c_int64),
        ("num_bias", ctypes.c_int)]


class LogitsSpec:
    """What pa_process_logits does to logits (pa_logits_spec); every part may be
    left out.  history int32 [B][H] with history_lens int32 [B] (prompt first, then
    output) and prompt_lens int32 [B]; draft_tokens int32 [B][rows - 1]; repetition,
    presence, frequency, temperature fp32 [B]; bias_tokens int32 and bias_values
    fp32 [B][n]; allowed int32 [B][rows][words] or [B][words] (bit t % 32 of word
    t / 32).  Keeps the tensors; their contents are read by each call."""

    def __init__(self, *, history=None, history_lens=None, prompt_lens=None, draft_tokens=None,
                 repetition=None, presence=None, frequency=None, temperature=None,
                 bias_tokens=None, bias_values=None, allowed=None):
        self.tensors = dict(history=history, history_lens=history_lens, prompt_lens=prompt_lens,
                            draft_tokens=draft_tokens, repetition=repetition, presence=presence,
                            frequency=frequency, temperature=temperature, bias_tokens=bias_tokens,
                            bias_values=bias_values, allowed=allowed)
        if (history is None) != (history_lens is None):
            raise ValueError("history and history_lens go together")
        if (bias_tokens is None) != (bias_values is None):
            raise ValueError("bias_tokens and bias_values go together")
        if prompt_lens is not None and history is None:
            raise ValueError("prompt_lens needs a history")

    def _pointer(self, B, rows, V, dev):
        t = self.tensors
        for name, x in t.items():
            if x is None:
                continue
            _need(x, name, torch.float32 if name in ("repetition", "presence", "frequency",
                                                     "temperature", "bias_values") else torch.int32,
                  None, dev)
            shape = tuple(x.shape)
            n = t["bias_tokens"].shape[-1] if t["bias_tokens"] is not None else 0
            good = {"history": shape[:1] == (B,) and len(shape) == 2,
                    "draft_tokens": shape == (B, rows - 1),
                    "bias_tokens": shape == (B, n), "bias_values": shape == (B, n),
                    "allowed": shape[:-1] in ((B, rows),) + (((B,),) if rows == 1 else ()) and
                    shape[-1] >= (V + 31) // 32}
            if not good.get(name, shape == (B,)):
                raise ValueError(f"{name} has shape {shape}")
        if rows > 1 and t["draft_tokens"] is None and t["history"] is not None:
            raise ValueError("several rows a sequence need the draft_tokens between them")
        st = _LogitsStruct(*(None if x is None else x.data_ptr() for x in t.values()),
                           0 if t["history"] is None else t["history"].shape[1],
                           0 if t["allowed"] is None else t["allowed"].shape[-1],
                           0 if t["bias_tokens"] is None else t["bias_tokens"].shape[1])
        p = ctypes.c_void_p(ctypes.addressof(st))
        p.owner = (self, st)          # a recorded call keeps the struct and the tensors alive
        return p


def _logit_rows(t, name, dtypes, dev):
    """Checks [B][V] or [B][rows][V] logits whose rows may be padded; (B, rows, V, row stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [B][V] or [B][rows][V]")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    x = t if t.dim() == 3 else t[:, None]
    return (*x.shape, _prob_rows(x, name, t.dtype, dev, x.shape[1]))


def pa_process_logits(out, logits, spec: LogitsSpec, *, probs: bool = False) -> None:
    """out = logits [B][V] or [B][rows][V] (fp32, fp16 or bf16) with spec's penalties,
    biases and mask, in the logits' dtype (out may be the logits); with probs
    softmax(out / temperature) in fp32, as pa_verify_drafts takes it."""
    if not isinstance(spec, LogitsSpec):
        raise TypeError("spec must be a LogitsSpec")
    codes = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    dev = logits.device
    B, rows, V, stride = _logit_rows(logits, "logits", tuple(codes), dev)
    *shape, out_stride = _logit_rows(out, "out", (torch.float32 if probs else logits.dtype,), dev)
    if shape != [B, rows, V]:
        raise ValueError("shape mismatch")
    _here(dev)
    _call(load().pa_process_logits, "pa_process_logits", _ptr(out), out_stride, _ptr(logits),
          stride, spec._pointer(B, rows, V, dev), B, rows, V, codes[logits.dtype], int(bool(probs)),
          _stream(dev))
