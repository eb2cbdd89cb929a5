"""Thin ctypes binding of libsinkattn (argument marshalling only).

Every function here has the name of the C entry point it calls and does
nothing but turn torch tensors into pointers and sizes, allocate outputs the
caller did not pass (torch device memory), and raise on a non-zero status.
All arithmetic runs in the CUDA kernels behind the C ABI; there is no
fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsinkattn.so")
_lock = threading.Lock()
_lib = None

(OK, INVALID_ARG, UNSUPPORTED, CUDA_ERROR, TIMEOUT, BAD_LENGTHS, OUT_OF_PAGES,
 BAD_PAGES) = range(8)


class SinkAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (status_name(status), message))
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libsinkattn.so (built in-tree by ``_build.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "libsinkattn.so is not built (%s); build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            P, I32, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
            I64 = ctypes.c_int64
            L.sinkattn_prefill.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, F,
                                           I32, I32, P, P, P]
            L.sinkattn_decode_split.argtypes = [P, P, P, P, I32, I32, I32, I32, I32, I32, F, I32, I32,
                                                I32, P, P, P]
            L.sinkattn_merge.argtypes = [P, P, P, I32, I32, I32, I32, P, P, P]
            L.sinkattn_decode.argtypes = [P, P, P, P, I32, I32, I32, I32, I32, I32, F, I32, I32, I32,
                                          P, P, SZ, P, P, P]
            L.sinkattn_decode_fused.argtypes = [P, P, P, P, I32, I32, I32, I32, I32, I32, F, I32,
                                                I32, I32, P, P, P, P]
            L.sinkattn_decode_noalloc.argtypes = [P, P, P, P, I32, I32, I32, I32, I32, I32, F, I32,
                                                  I32, I32, P, P, P, P]
            L.sinkattn_decode_workspace_bytes.argtypes = [I32, I32, I32, I32, I32,
                                                          ctypes.POINTER(SZ)]
            L.sinkattn_decode_default_splits.argtypes = [I32, I32, I32, I32, I32, I32,
                                                         ctypes.POINTER(I32)]
            L.sinkattn_prefill_paged.argtypes = [P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32,
                                                 I32, I32, I32, I32, F, I32, I32, P, P, P]
            L.sinkattn_decode_split_paged.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32,
                                                      I32, I32, I32, F, I32, I32, I32, P, P, P]
            L.sinkattn_decode_paged.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32,
                                                I32, I32, F, I32, I32, I32, P, P, SZ, P, P, P]
            L.sinkattn_status_string.argtypes = [ctypes.c_int]
            L.sinkattn_status_string.restype = ctypes.c_char_p
            L.sinkattn_last_error.argtypes = []
            L.sinkattn_last_error.restype = ctypes.c_char_p
            L.sinkattn_debug_status.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
            L.sinkattn_debug_set_hooks.argtypes = [ctypes.c_longlong, ctypes.c_int]
            L.sinkattn_set_decode_kernel.argtypes = [ctypes.c_int]
            L.sinkattn_set_prefill_kernel.argtypes = [ctypes.c_int]
            L.sinkattn_decode_split_fp8.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32,
                                                    F, I32, I32, I32, P, P, P]
            L.sinkattn_decode_fp8.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, F,
                                              I32, I32, I32, P, P, SZ, P, P, P]
            L.sinkattn_decode_shared_paged.argtypes = (
                [P] * 8 + [I32] * 10 + [F] + [I32] * 4 + [P, P, SZ, P, P, P])
            L.sinkattn_decode_shared_paged_fp8.argtypes = (
                [P] * 10 + [I32] * 10 + [F] + [I32] * 4 + [P, P, SZ, P, P, P])
            L.sinkattn_decode_shared_workspace_bytes.argtypes = [I32] * 7 + [ctypes.POINTER(SZ)]
            L.sinkattn_decode_shared_default_splits.argtypes = (
                [I32] * 8 + [ctypes.POINTER(I32)] * 2)
            L.sinkattn_append_paged.argtypes = [P, P, I64, I64, P, I32, P, P, I32, I32, I32, I32, P]
            L.sinkattn_append_paged_fp8.argtypes = [P, P, I64, I64, P, I32, P, P, P, P, I32, I32,
                                                    I32, I32, P]
            T = [P, I32, I32, I32, I32]
            L.sinkattn_pages_table_ints.argtypes = [I32, I32, I32, ctypes.POINTER(I64)]
            L.sinkattn_pages_init.argtypes = T + [P]
            L.sinkattn_pages_reserve.argtypes = T + [P, P, I32, I32, P, P, I32, I64, I32, I32, P, P]
            L.sinkattn_pages_fork.argtypes = T + [P, P, I32, P]
            L.sinkattn_pages_truncate.argtypes = T + [P, P, I32, P]
            L.sinkattn_pages_compact.argtypes = T + [P, P, I32, I64, I32, I32, P, P]
            L.sinkattn_pages_lists.argtypes = T + [P, I32, P, P, P, I32, P]
            L.sinkattn_prefill_backward.argtypes = (
                [P] * 10 + [I32] * 8 + [F] + [I32] * 2 + [P] * 5 + [SZ, P])
            L.sinkattn_prefill_backward_workspace_bytes.argtypes = [I32, I32, ctypes.POINTER(SZ)]
            D = ctypes.c_double
            L.sinkattn_rope_frequencies.argtypes = [I32, D, I32, D, I32, D, D, P, P]
            L.sinkattn_rope_turns.argtypes = [P, I32, P]
            R = [P, I32, I32, F, P, P, F]   # turns .. eps
            L.sinkattn_rope_qkv.argtypes = [P] * 3 + [I64] * 3 + [P] * 2 + [I32] * 5 + R + [P] * 4
            L.sinkattn_rope_qkv_backward.argtypes = (
                [P] * 5 + [I64] * 2 + [P] * 2 + [I32] * 5 + R + [P] * 3 + [I64] * 3 + [P] * 3
                + [SZ, P])
            L.sinkattn_rope_qkv_backward_workspace_bytes.argtypes = [I32, I32, ctypes.POINTER(SZ)]
            L.sinkattn_rope_append_paged.argtypes = (
                [P] * 3 + [I64] * 3 + [P] * 2 + [I32] * 4 + R + [P] * 3 + [I32] * 2 + [P])
            L.sinkattn_rope_append_paged_fp8.argtypes = (
                [P] * 3 + [I64] * 3 + [P] * 2 + [I32] * 4 + R + [P] * 5 + [I32] * 2 + [P])
            for name in ("sinkattn_prefill", "sinkattn_decode_split", "sinkattn_merge",
                         "sinkattn_decode", "sinkattn_decode_fused", "sinkattn_decode_noalloc",
                         "sinkattn_decode_workspace_bytes", "sinkattn_decode_default_splits",
                         "sinkattn_debug_status", "sinkattn_debug_set_hooks",
                         "sinkattn_set_decode_kernel",
                         "sinkattn_set_prefill_kernel", "sinkattn_decode_split_fp8",
                         "sinkattn_decode_fp8",
                         "sinkattn_prefill_paged", "sinkattn_decode_split_paged",
                         "sinkattn_decode_paged", "sinkattn_decode_shared_paged",
                         "sinkattn_decode_shared_paged_fp8",
                         "sinkattn_decode_shared_workspace_bytes",
                         "sinkattn_decode_shared_default_splits", "sinkattn_append_paged",
                         "sinkattn_append_paged_fp8", "sinkattn_pages_table_ints",
                         "sinkattn_pages_init", "sinkattn_pages_reserve", "sinkattn_pages_fork",
                         "sinkattn_pages_truncate", "sinkattn_pages_compact",
                         "sinkattn_pages_lists", "sinkattn_prefill_backward",
                         "sinkattn_prefill_backward_workspace_bytes",
                         "sinkattn_rope_frequencies", "sinkattn_rope_turns", "sinkattn_rope_qkv",
                         "sinkattn_rope_qkv_backward",
                         "sinkattn_rope_qkv_backward_workspace_bytes",
                         "sinkattn_rope_append_paged", "sinkattn_rope_append_paged_fp8"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def status_name(status: int) -> str:
    return lib().sinkattn_status_string(int(status)).decode()


def _check(rc: int):
    if rc != OK:
        raise SinkAttnError(rc, lib().sinkattn_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t, stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _scale(sm_scale, d):
    return float(1.0 / math.sqrt(d) if sm_scale is None else sm_scale)


def sinkattn_prefill(q, k, v, sinks, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                     num_kv_heads, sm_scale=None, causal=True, window=0, out=None, lse=None,
                     return_lse=True, stream=None):
    """Varlen prefill with sink. q [total_q, Hq, d] bf16; k, v ragged HND
    [Hkv * total_k, d] bf16; sinks [Hq] fp32 or None; cu_seqlens int32 [B+1]
    on the device. Returns (out, lse) with lse None unless requested."""
    total_q, Hq, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((total_q, Hq), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(sinks), _ptr(cu_seqlens_q),
                                _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, total_q,
                                int(max_seqlen_q), int(max_seqlen_k), Hq, int(num_kv_heads), d,
                                _scale(sm_scale, d), int(bool(causal)), int(window), _ptr(out),
                                _ptr(lse), _stream(q, stream))
    _check(rc)
    return out, lse


def sinkattn_decode_split(q, k, v, kv_indptr, q_len, max_kv_len, num_kv_heads, num_splits,
                          sm_scale=None, causal=True, window=0, part_acc=None, part_md=None,
                          stream=None):
    """Split-KV step 1. q [B*q_len, Hq, d]. Returns (part_acc [B*q_len, Hq, S, d],
    part_md [B*q_len, Hq, S, 2]) fp32, without the sink."""
    rows, Hq, d = q.shape
    batch = kv_indptr.numel() - 1
    if part_acc is None:
        part_acc = torch.empty((rows, Hq, num_splits, d), dtype=torch.float32, device=q.device)
    if part_md is None:
        part_md = torch.empty((rows, Hq, num_splits, 2), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode_split(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_indptr), batch, int(q_len),
                                     int(max_kv_len), Hq, int(num_kv_heads), d,
                                     _scale(sm_scale, d), int(bool(causal)), int(window),
                                     int(num_splits), _ptr(part_acc), _ptr(part_md),
                                     _stream(q, stream))
    _check(rc)
    return part_acc, part_md


def sinkattn_merge(part_acc, part_md, sinks, out=None, lse=None, return_lse=True, stream=None):
    """Split-KV step 2: fold partials with the sink counted once. Returns (out, lse)."""
    rows, Hq, S, d = part_acc.shape
    if out is None:
        out = torch.empty((rows, Hq, d), dtype=torch.bfloat16, device=part_acc.device)
    if lse is None and return_lse:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=part_acc.device)
    rc = lib().sinkattn_merge(_ptr(part_acc), _ptr(part_md), _ptr(sinks), rows, Hq, d, S,
                              _ptr(out), _ptr(lse), _stream(part_acc, stream))
    _check(rc)
    return out, lse


def sinkattn_decode_workspace_bytes(batch, q_len, num_qo_heads, head_dim, num_splits) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().sinkattn_decode_workspace_bytes(int(batch), int(q_len), int(num_qo_heads),
                                                 int(head_dim), int(num_splits), ctypes.byref(n)))
    return int(n.value)


def sinkattn_decode_default_splits(batch, q_len, num_qo_heads, num_kv_heads, head_dim,
                                   max_kv_len) -> int:
    s = ctypes.c_int32(0)
    _check(lib().sinkattn_decode_default_splits(int(batch), int(q_len), int(num_qo_heads),
                                                int(num_kv_heads), int(head_dim), int(max_kv_len),
                                                ctypes.byref(s)))
    return int(s.value)


def sinkattn_decode(q, k, v, kv_indptr, sinks, q_len, max_kv_len, num_kv_heads, num_splits=0,
                    sm_scale=None, causal=True, window=0, workspace=None, out=None, lse=None,
                    return_lse=True, stream=None):
    """Split-KV decode / MTP in one call (split then merge on one stream).
    ``workspace``: a uint8 device tensor of at least
    sinkattn_decode_workspace_bytes() bytes (allocated here if None)."""
    rows, Hq, d = q.shape
    batch = kv_indptr.numel() - 1
    if num_splits <= 0:
        num_splits = sinkattn_decode_default_splits(batch, q_len, Hq, num_kv_heads, d, max_kv_len)
    need = sinkattn_decode_workspace_bytes(batch, q_len, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty((max(need, 256),), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_indptr), batch, int(q_len),
                               int(max_kv_len), Hq, int(num_kv_heads), d, _scale(sm_scale, d),
                               int(bool(causal)), int(window), int(num_splits), _ptr(sinks),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _ptr(out), _ptr(lse), _stream(q, stream))
    _check(rc)
    return out, lse


def sinkattn_decode_fused(q, k, v, kv_indptr, sinks, q_len, max_kv_len, num_kv_heads,
                          num_splits=0, sm_scale=None, causal=True, window=0, out=None, lse=None,
                          return_lse=True, stream=None):
    """Split-KV decode / MTP with the merge done on chip by a thread-block
    cluster (num_splits <= 16; no workspace). Returns (out, lse)."""
    rows, Hq, d = q.shape
    batch = kv_indptr.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_indptr), batch,
                                     int(q_len), int(max_kv_len), Hq, int(num_kv_heads), d,
                                     _scale(sm_scale, d), int(bool(causal)), int(window),
                                     int(num_splits), _ptr(sinks), _ptr(out), _ptr(lse),
                                     _stream(q, stream))
    _check(rc)
    return out, lse


def sinkattn_decode_noalloc(q, k, v, kv_indptr, sinks, q_len, max_kv_len, num_kv_heads,
                            num_splits=0, sm_scale=None, causal=True, window=0, out=None, lse=None,
                            return_lse=True, stream=None):
    """sinkattn_decode without a workspace, for callers that cannot allocate
    device memory: the partials go to the library's fixed 32 MiB scratch
    array. Pass ``out`` (and ``lse``) to allocate nothing here either."""
    rows, Hq, d = q.shape
    batch = kv_indptr.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    # the library looks the scratch address up in the current device's
    # context and rejects a stream of another device: make q's device current
    with torch.cuda.device(q.device):
        rc = lib().sinkattn_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_indptr), batch,
                                           int(q_len), int(max_kv_len), Hq, int(num_kv_heads), d,
                                           _scale(sm_scale, d), int(bool(causal)), int(window),
                                           int(num_splits), _ptr(sinks), _ptr(out), _ptr(lse),
                                           _stream(q, stream))
    _check(rc)
    return out, lse


DECODE_KERNELS = {"auto": 0, "warp": 1, "tcgen05": 2}


def _pages(k_pages):
    """(num_pages, Hkv, page_size, d) of a page pool."""
    num_pages, Hkv, page_size, d = k_pages.shape
    return num_pages, Hkv, page_size, d


def sinkattn_prefill_paged(q, k_pages, v_pages, sinks, cu_seqlens_q, cu_seqlens_k, page_indptr,
                           page_indices, max_seqlen_q, max_seqlen_k, sm_scale=None, causal=True,
                           window=0, out=None, lse=None, return_lse=True, stream=None):
    """sinkattn_prefill over a paged KV cache: k_pages, v_pages bf16
    [num_pages, Hkv, page_size, d]; sequence b's pages are
    page_indices[page_indptr[b]:page_indptr[b+1]] (int32, device); key
    counts come from cu_seqlens_k. Returns (out, lse)."""
    total_q, Hq, d = q.shape
    num_pages, Hkv, page_size, _ = _pages(k_pages)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((total_q, Hq), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_prefill_paged(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(sinks), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
        _ptr(page_indptr), _ptr(page_indices), num_pages, page_size, cu_seqlens_q.numel() - 1,
        total_q, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, d, _scale(sm_scale, d),
        int(bool(causal)), int(window), _ptr(out), _ptr(lse), _stream(q, stream))
    _check(rc)
    return out, lse


def sinkattn_decode_split_paged(q, k_pages, v_pages, kv_indptr, page_indptr, page_indices, q_len,
                                max_kv_len, num_splits, sm_scale=None, causal=True, window=0,
                                part_acc=None, part_md=None, stream=None):
    """sinkattn_decode_split over a paged KV cache (layout as in
    sinkattn_prefill_paged). Returns (part_acc, part_md) without the sink."""
    rows, Hq, d = q.shape
    num_pages, Hkv, page_size, _ = _pages(k_pages)
    batch = kv_indptr.numel() - 1
    if part_acc is None:
        part_acc = torch.empty((rows, Hq, num_splits, d), dtype=torch.float32, device=q.device)
    if part_md is None:
        part_md = torch.empty((rows, Hq, num_splits, 2), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode_split_paged(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kv_indptr), _ptr(page_indptr),
        _ptr(page_indices), num_pages, page_size, batch, int(q_len), int(max_kv_len), Hq, Hkv, d,
        _scale(sm_scale, d), int(bool(causal)), int(window), int(num_splits), _ptr(part_acc),
        _ptr(part_md), _stream(q, stream))
    _check(rc)
    return part_acc, part_md


def sinkattn_decode_paged(q, k_pages, v_pages, kv_indptr, page_indptr, page_indices, sinks, q_len,
                          max_kv_len, num_splits=0, sm_scale=None, causal=True, window=0,
                          workspace=None, out=None, lse=None, return_lse=True, stream=None):
    """sinkattn_decode over a paged KV cache (layout as in
    sinkattn_prefill_paged). Returns (out, lse)."""
    rows, Hq, d = q.shape
    num_pages, Hkv, page_size, _ = _pages(k_pages)
    batch = kv_indptr.numel() - 1
    if num_splits <= 0:
        num_splits = sinkattn_decode_default_splits(batch, q_len, Hq, Hkv, d, max_kv_len)
    need = sinkattn_decode_workspace_bytes(batch, q_len, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty((max(need, 256),), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode_paged(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kv_indptr), _ptr(page_indptr),
        _ptr(page_indices), num_pages, page_size, batch, int(q_len), int(max_kv_len), Hq, Hkv, d,
        _scale(sm_scale, d), int(bool(causal)), int(window), int(num_splits), _ptr(sinks),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
        _stream(q, stream))
    _check(rc)
    return out, lse


def sinkattn_set_decode_kernel(kind) -> None:
    """Selects the split-KV partial kernel process-wide: "auto", "warp" or
    "tcgen05" (or the integer codes of include/sinkattn.h)."""
    code = DECODE_KERNELS[kind] if isinstance(kind, str) else int(kind)
    _check(lib().sinkattn_set_decode_kernel(code))
    _shared_sizes.cache_clear()   # (the default split counts go by the kernel)


def sinkattn_decode_split_fp8(q, k, v, k_scale, v_scale, kv_indptr, q_len, max_kv_len,
                              num_splits, sm_scale=None, causal=True, window=0, part_acc=None,
                              part_md=None, stream=None):
    """sinkattn_decode_split over an FP8 KV cache: k, v uint8 e4m3 codes in
    the ragged HND layout [Hkv * total_k, d]; k_scale, v_scale fp32 [Hkv]
    per-KV-head scales (device). Returns (part_acc, part_md) without the sink."""
    rows, Hq, d = q.shape
    Hkv = k_scale.numel()
    batch = kv_indptr.numel() - 1
    if part_acc is None:
        part_acc = torch.empty((rows, Hq, num_splits, d), dtype=torch.float32, device=q.device)
    if part_md is None:
        part_md = torch.empty((rows, Hq, num_splits, 2), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode_split_fp8(
        _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(kv_indptr), batch,
        int(q_len), int(max_kv_len), Hq, Hkv, d, _scale(sm_scale, d), int(bool(causal)),
        int(window), int(num_splits), _ptr(part_acc), _ptr(part_md), _stream(q, stream))
    _check(rc)
    return part_acc, part_md


def sinkattn_decode_fp8(q, k, v, k_scale, v_scale, kv_indptr, sinks, q_len, max_kv_len,
                        num_splits=0, sm_scale=None, causal=True, window=0, workspace=None,
                        out=None, lse=None, return_lse=True, stream=None):
    """sinkattn_decode over an FP8 KV cache (layout as in
    sinkattn_decode_split_fp8). Returns (out, lse)."""
    rows, Hq, d = q.shape
    Hkv = k_scale.numel()
    batch = kv_indptr.numel() - 1
    if num_splits <= 0:
        num_splits = sinkattn_decode_default_splits(batch, q_len, Hq, Hkv, d, max_kv_len)
    need = sinkattn_decode_workspace_bytes(batch, q_len, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty((max(need, 256),), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    rc = lib().sinkattn_decode_fp8(
        _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(kv_indptr), batch,
        int(q_len), int(max_kv_len), Hq, Hkv, d, _scale(sm_scale, d), int(bool(causal)),
        int(window), int(num_splits), _ptr(sinks), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(q, stream))
    _check(rc)
    return out, lse


def _bad(t, what, dtype, dev, shape):
    """Raises what is wrong with a tensor that _need did not take."""
    if not torch.is_tensor(t):
        text = "%s must be a tensor" % what
    elif t.dtype is not dtype:
        text = "%s must be %s, not %s" % (what, dtype, t.dtype)
    elif t.device != dev:
        text = "%s must be on %s, not %s" % (what, dev, t.device)
    elif not t.is_contiguous():
        text = "%s must be contiguous" % what
    elif isinstance(shape, int):
        text = "%s must have %d dimension(s), not shape %s" % (what, shape, tuple(t.shape))
    else:
        text = "%s must have shape %s, not %s" % (what, tuple(shape), tuple(t.shape))
    raise SinkAttnError(INVALID_ARG, text)


def _need(t, what, dtype, dev, shape):
    """The address of a tensor that the kernels read or write, once it is known
    to have the type, device, layout and shape (a tuple, or the number of
    dimensions) that they take it for. A call of the paged-cache functions
    costs a few microseconds on the GPU, so this is one expression when all is well."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.is_contiguous()
            and (t.dim() == shape if shape.__class__ is int else t.shape == shape)):
        return t.data_ptr()
    _bad(t, what, dtype, dev, shape)


def _need_cuda(t, what):
    if not torch.is_tensor(t) or not t.is_cuda:
        raise SinkAttnError(INVALID_ARG, "%s must be a CUDA tensor" % what)
    return t.device


def _i32(*sizes):
    """The sizes as integers that the entry points' 32-bit arguments hold (ctypes would
    drop the upper bits)."""
    sizes = [int(x) for x in sizes]
    for x in sizes:
        if not -2 ** 31 <= x < 2 ** 31:
            raise SinkAttnError(INVALID_ARG, "%d does not fit a 32-bit size" % x)
    return sizes


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(dev, stream):
    if stream is None:
        return (_raw_stream(dev.index) if _raw_stream is not None
                else torch.cuda.current_stream(dev).cuda_stream)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(shape, dtype, dev, stream, kept=True):
    """A tensor for kernels on `stream`, taken from that stream's memory: what
    its bytes held before may still be read on another stream. One that the
    caller gets (`kept`) is used on the current stream too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    here = torch.cuda.current_stream(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_of(dev, stream), device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if kept and stream.cuda_stream != here.cuda_stream:
        t.record_stream(here)
    return t


def _launch(dev, entry, *args):
    """Calls a C entry point with `dev` current; raises on a non-zero status."""
    if dev.index == torch.cuda.current_device():
        rc = entry(*args)
    else:
        with torch.cuda.device(dev):
            rc = entry(*args)
    if rc != OK:
        _check(rc)


def sinkattn_decode_shared_default_splits(batch, q_len, num_qo_heads, num_kv_heads, head_dim,
                                          num_groups, max_prefix_len, max_suffix_len):
    """(prefix_splits, num_splits) the shared-prefix decode uses by default."""
    a, b = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().sinkattn_decode_shared_default_splits(
        *_i32(batch, q_len, num_qo_heads, num_kv_heads, head_dim, num_groups, max_prefix_len,
              max_suffix_len), ctypes.byref(a), ctypes.byref(b)))
    return int(a.value), int(b.value)


def sinkattn_decode_shared_workspace_bytes(batch, q_len, num_qo_heads, head_dim, num_groups,
                                           prefix_splits, num_splits) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().sinkattn_decode_shared_workspace_bytes(
        *_i32(batch, q_len, num_qo_heads, head_dim, num_groups, prefix_splits, num_splits),
        ctypes.byref(n)))
    return int(n.value)


@functools.lru_cache(maxsize=256)
def _shared_sizes(device_index, prefix_splits, num_splits, batch, q_len, Hq, Hkv, d, groups,
                  max_prefix_len, max_suffix_len):
    """(prefix_splits, num_splits, workspace bytes) of these sizes (host arithmetic only)."""
    _i32(prefix_splits, num_splits, max_prefix_len, max_suffix_len)
    if num_splits <= 0 or prefix_splits <= 0:
        ps, ss = sinkattn_decode_shared_default_splits(batch, q_len, Hq, Hkv, d, groups,
                                                       max_prefix_len, max_suffix_len)
        prefix_splits = prefix_splits if prefix_splits > 0 else ps
        num_splits = num_splits if num_splits > 0 else ss
    return prefix_splits, num_splits, sinkattn_decode_shared_workspace_bytes(
        batch, q_len, Hq, d, groups, prefix_splits, num_splits)


def _decode_shared(entry, pool_dtype, scales, q, k_pages, v_pages, kv_indptr, page_indptr,
                   page_indices, group_indptr, prefix_lens, sinks, q_len, max_prefix_len,
                   max_suffix_len, num_splits, prefix_splits, sm_scale, causal, window, workspace,
                   out, lse, return_lse, stream):
    dev = _need_cuda(q, "q")
    i32, f32 = torch.int32, torch.float32
    q_p = _need(q, "q", torch.bfloat16, dev, 3)
    rows, Hq, d = q.shape
    k_p = _need(k_pages, "k_pages", pool_dtype, dev, 4)
    num_pages, Hkv, page_size, kd = k_pages.shape
    if kd != d:
        raise SinkAttnError(INVALID_ARG, "q has head_dim %d, the pools %d" % (d, kd))
    v_p = _need(v_pages, "v_pages", pool_dtype, dev, k_pages.shape)
    scale_p = [_need(t, what, f32, dev, (Hkv,)) for t, what in zip(scales, ("k_scale", "v_scale"))]
    kv_p = _need(kv_indptr, "kv_indptr", i32, dev, 1)
    batch, q_len = kv_indptr.shape[0] - 1, int(q_len)
    if batch < 0 or rows != batch * q_len:
        raise SinkAttnError(INVALID_ARG, "q has %d rows, batch * q_len is %d" % (rows, batch * q_len))
    pp_p = _need(page_indptr, "page_indptr", i32, dev, (batch + 1,))
    pi_p = _need(page_indices, "page_indices", i32, dev, 1)
    pl_p = _need(prefix_lens, "prefix_lens", i32, dev, 1)
    groups = prefix_lens.shape[0]
    gp_p = _need(group_indptr, "group_indptr", i32, dev, (groups + 1,))
    sinks_p = None if sinks is None else _need(sinks, "sinks", f32, dev, (Hq,))
    max_prefix_len, max_suffix_len = int(max_prefix_len), int(max_suffix_len)
    prefix_splits, num_splits, need = _shared_sizes(
        dev.index, int(prefix_splits), int(num_splits), batch, q_len, Hq, Hkv, d, groups,
        max_prefix_len, max_suffix_len)
    if workspace is None:
        workspace = _new((need,), torch.uint8, dev, stream, kept=False)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise SinkAttnError(INVALID_ARG, "workspace must be contiguous and on %s" % dev)
    if out is None:
        out = _new(q.shape, torch.bfloat16, dev, stream)
        out_p = out.data_ptr()
    else:
        out_p = _need(out, "out", torch.bfloat16, dev, q.shape)
    lse_p = None
    if lse is not None:
        lse_p = _need(lse, "lse", f32, dev, (rows, Hq))
    elif return_lse:
        lse = _new((rows, Hq), f32, dev, stream)
        lse_p = lse.data_ptr()
    if batch == 0:   # (an empty tensor has no address to check)
        return out, lse
    _launch(dev, entry, q_p, k_p, v_p, *scale_p, kv_p, pp_p, pi_p, gp_p, pl_p, groups, num_pages,
            page_size, batch, q_len, max_prefix_len, max_suffix_len, Hq, Hkv, d,
            _scale(sm_scale, d), 1 if causal else 0, min(int(window), 2 ** 31 - 1), prefix_splits,
            num_splits, sinks_p, workspace.data_ptr(), workspace.numel() * workspace.element_size(), out_p,
            lse_p, _stream_of(dev, stream))
    return out, lse


def sinkattn_decode_shared_paged(q, k_pages, v_pages, kv_indptr, page_indptr, page_indices,
                                 group_indptr, prefix_lens, sinks, q_len, max_prefix_len,
                                 max_suffix_len, num_splits=0, prefix_splits=0, sm_scale=None,
                                 causal=True, window=0, workspace=None, out=None, lse=None,
                                 return_lse=True, stream=None):
    """sinkattn_decode_paged for a batch whose sequences share prefixes: group
    g holds sequences group_indptr[g] .. group_indptr[g+1] - 1 (int32, device),
    whose first prefix_lens[g] keys (int32, device; a multiple of the page
    size) are the same; they are read once, from the first sequence's page
    list. max_prefix_len bounds prefix_lens, max_suffix_len the keys of a
    sequence past its prefix (at least q_len each). Where these say that the
    call has few keys, every sequence reads its own, unless prefix_splits > 0.
    Returns (out, lse)."""
    return _decode_shared(lib().sinkattn_decode_shared_paged, torch.bfloat16, (), q, k_pages,
                          v_pages, kv_indptr, page_indptr, page_indices, group_indptr, prefix_lens,
                          sinks, q_len, max_prefix_len, max_suffix_len, num_splits, prefix_splits,
                          sm_scale, causal, window, workspace, out, lse, return_lse, stream)


def sinkattn_decode_shared_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, kv_indptr, page_indptr,
                                     page_indices, group_indptr, prefix_lens, sinks, q_len,
                                     max_prefix_len, max_suffix_len, num_splits=0, prefix_splits=0,
                                     sm_scale=None, causal=True, window=0, workspace=None,
                                     out=None, lse=None, return_lse=True, stream=None):
    """sinkattn_decode_shared_paged over pools of e4m3 codes (uint8) with
    per-KV-head fp32 scales [Hkv]. Returns (out, lse)."""
    return _decode_shared(lib().sinkattn_decode_shared_paged_fp8, torch.uint8, (k_scale, v_scale),
                          q, k_pages, v_pages, kv_indptr, page_indptr, page_indices, group_indptr,
                          prefix_lens, sinks, q_len, max_prefix_len, max_suffix_len, num_splits,
                          prefix_splits, sm_scale, causal, window, workspace, out, lse, return_lse,
                          stream)


def _append(entry, pool_dtype, scales, k, v, slots, k_pages, v_pages, stream):
    dev = _need_cuda(k_pages, "k_pages")
    kp_p = _need(k_pages, "k_pages", pool_dtype, dev, 4)
    num_pages, Hkv, page_size, d = k_pages.shape
    vp_p = _need(v_pages, "v_pages", pool_dtype, dev, k_pages.shape)
    s_p = _need(slots, "slots", torch.int32, dev, 1)
    tokens = slots.shape[0]
    strides = []
    for t, what in ((k, "k"), (v, "v")):
        if (not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.device != dev
                or t.shape != (tokens, Hkv, d)):
            raise SinkAttnError(INVALID_ARG, "%s must be bfloat16 %s on %s" % (
                what, (tokens, Hkv, d), dev))
        at, head, el = t.stride()
        if tokens > 0 and (el != 1 or (head != d and Hkv > 1)):
            raise SinkAttnError(INVALID_ARG, "the rows of a token of %s must be contiguous" % what)
        strides.append(at if tokens > 1 else Hkv * d)
    scale_p = [_need(t, what, torch.float32, dev, (Hkv,))
               for t, what in zip(scales, ("k_scale", "v_scale"))]
    _launch(dev, entry, k.data_ptr(), v.data_ptr(), strides[0], strides[1], s_p, tokens, *scale_p,
            kp_p, vp_p, num_pages, page_size, Hkv, d, _stream_of(dev, stream))


def sinkattn_append_paged(k, v, slots, k_pages, v_pages, stream=None):
    """Writes new keys and values, bf16 [tokens, Hkv, d] (rows of a token
    contiguous, any token stride that is a multiple of 8), to the slots (int32
    [tokens], page * page_size + position; outside the pool: left out) of the
    pools [num_pages, Hkv, page_size, d]."""
    _append(lib().sinkattn_append_paged, torch.bfloat16, (), k, v, slots, k_pages, v_pages, stream)


def sinkattn_append_paged_fp8(k, v, slots, k_scale, v_scale, k_pages, v_pages, stream=None):
    """sinkattn_append_paged into pools of e4m3 codes (uint8): the code
    nearest to x / scale[head] (ties to even, saturating at 448)."""
    _append(lib().sinkattn_append_paged_fp8, torch.uint8, (k_scale, v_scale), k, v, slots, k_pages,
            v_pages, stream)


def sinkattn_pages_table_ints(num_pages, max_seqs, max_pages) -> int:
    n = ctypes.c_int64(0)
    _check(lib().sinkattn_pages_table_ints(*_i32(num_pages, max_seqs, max_pages), ctypes.byref(n)))
    return int(n.value)


class PageTable:
    """A page table's buffer and sizes. ``state``: an int32 device tensor of at
    least sinkattn_pages_table_ints() words that holds a table already; without
    one, a new buffer on ``device`` is allocated and initialised (every page
    free, every sequence empty). The parts are views of ``state``."""
    __slots__ = ("_args", "_state", "device")

    def __init__(self, state, num_pages, page_size, max_seqs, max_pages, device="cuda",
                 stream=None):
        num_pages, page_size, max_seqs, max_pages = _i32(num_pages, page_size, max_seqs, max_pages)
        need = 16 + max_seqs * (8 + max_pages) + 4 * num_pages
        new = state is None
        if new:
            words = sinkattn_pages_table_ints(num_pages, max_seqs, max_pages)
            state = _new((words,), torch.int32, torch.device(device), stream)
        self.device = _need_cuda(state, "state")
        ptr = _need(state, "state", torch.int32, self.device, 1)
        if state.shape[0] < need:
            raise SinkAttnError(INVALID_ARG, "state has %d words, a table of these sizes %d" % (
                state.shape[0], need))
        self._state = state
        # what every entry point takes first (the buffer stays where it is while the table lives)
        self._args = (ptr, num_pages, page_size, max_seqs, max_pages)
        if new:
            sinkattn_pages_init(self, stream=stream)

    state = property(lambda self: self._state)
    num_pages = property(lambda self: self._args[1])
    page_size = property(lambda self: self._args[2])
    max_seqs = property(lambda self: self._args[3])
    max_pages = property(lambda self: self._args[4])

    def _part(self, at, n):
        return self._state[at:at + n]

    @property
    def free_count(self):
        return self._part(0, 1)

    @property
    def seq_lens(self):
        return self._part(16, self.max_seqs)

    @property
    def page_list(self):
        return self._part(16 + self.max_seqs, self.max_seqs * self.max_pages).view(
            self.max_seqs, self.max_pages)

    @property
    def refcount(self):
        return self._part(16 + self.max_seqs * (1 + self.max_pages), self.num_pages)

    @property
    def free_list(self):
        return self._part(16 + self.max_seqs * (1 + self.max_pages) + self.num_pages,
                          self.num_pages)


def _pools(table, k_pages, v_pages):
    """(k, v, layers, layer stride, Hkv, row bytes) of the pools of one layer,
    [num_pages, Hkv, page_size, d], or of several, [layers, ...]."""
    for t, what in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if not isinstance(t, torch.Tensor) or t.device != table.device or t.dim() not in (4, 5):
            raise SinkAttnError(INVALID_ARG, "%s must be a tensor of 4 or 5 dimensions on %s" % (
                what, table.device))
    shape, strides = k_pages.shape, k_pages.stride()
    if shape != v_pages.shape or strides != v_pages.stride() or k_pages.dtype is not v_pages.dtype:
        raise SinkAttnError(INVALID_ARG, "k_pages and v_pages must have one shape, type and stride")
    if not k_pages.is_contiguous() and not (len(shape) == 5 and shape[0] > 0
                                            and k_pages[0].is_contiguous()):
        raise SinkAttnError(INVALID_ARG, "each layer of k_pages and v_pages must be contiguous")
    num_pages, Hkv, page_size, d = shape[-4:]
    if num_pages != table.num_pages or page_size != table.page_size:
        raise SinkAttnError(INVALID_ARG, "the pools have %d pages of %d, the table %d of %d" % (
            num_pages, page_size, table.num_pages, table.page_size))
    el = k_pages.element_size()
    layers = shape[0] if len(shape) == 5 else 1
    return (k_pages.data_ptr(), v_pages.data_ptr(), layers, strides[0] * el if layers > 1 else 0,
            Hkv, d * el)


def sinkattn_pages_init(table, stream=None) -> None:
    """Every page free (page 0 is the first to be taken), every sequence empty."""
    dev = table.device
    _launch(dev, lib().sinkattn_pages_init, *table._args, _stream_of(dev, stream))


def sinkattn_pages_reserve(table, seq_ids, cu_new, total_new, k_pages, v_pages, slots=None,
                           stream=None):
    """Room for cu_new[i+1] - cu_new[i] more tokens in sequence seq_ids[i]
    (int32, device). Returns the new tokens' slots, int32 [total_new]. A
    partly filled page that other sequences hold too is copied first, in the
    pools of all layers."""
    dev = table.device
    ids_p = _need(seq_ids, "seq_ids", torch.int32, dev, 1)
    n = seq_ids.shape[0]
    cu_p = _need(cu_new, "cu_new", torch.int32, dev, (n + 1,))
    total_new, = _i32(total_new)
    if slots is None:
        slots = _new((max(total_new, 0),), torch.int32, dev, stream)
        slots_p = slots.data_ptr()
    else:
        slots_p = _need(slots, "slots", torch.int32, dev, (total_new,))
    _launch(dev, lib().sinkattn_pages_reserve, *table._args, ids_p, cu_p, n, total_new,
            *_pools(table, k_pages, v_pages), slots_p, _stream_of(dev, stream))
    return slots


def sinkattn_pages_fork(table, src_ids, dst_ids, stream=None) -> None:
    """dst_ids[i] (empty sequences) become copies of src_ids[i] that share all
    their pages (int32, device)."""
    dev = table.device
    src_p = _need(src_ids, "src_ids", torch.int32, dev, 1)
    dst_p = _need(dst_ids, "dst_ids", torch.int32, dev, src_ids.shape)
    _launch(dev, lib().sinkattn_pages_fork, *table._args, src_p, dst_p, src_ids.shape[0],
            _stream_of(dev, stream))


def sinkattn_pages_truncate(table, seq_ids, new_lens=None, stream=None) -> None:
    """Shortens seq_ids[i] to new_lens[i] tokens (int32, device; None: 0, which
    frees the sequences); pages that no sequence holds any more become free."""
    dev = table.device
    ids_p = _need(seq_ids, "seq_ids", torch.int32, dev, 1)
    new_p = None if new_lens is None else _need(new_lens, "new_lens", torch.int32, dev,
                                                seq_ids.shape)
    _launch(dev, lib().sinkattn_pages_truncate, *table._args, ids_p, new_p, seq_ids.shape[0],
            _stream_of(dev, stream))


def sinkattn_pages_compact(table, k_pages, v_pages, page_map=None, stream=None):
    """Moves the pages in use to the front of the pools (all layers). Returns
    page_map, int32 [num_pages]: each old page's new index, -1 where it was free."""
    dev = table.device
    if page_map is None:
        page_map = _new((table.num_pages,), torch.int32, dev, stream)
        map_p = page_map.data_ptr()
    else:
        map_p = _need(page_map, "page_map", torch.int32, dev, (table.num_pages,))
    _launch(dev, lib().sinkattn_pages_compact, *table._args, *_pools(table, k_pages, v_pages),
            map_p, _stream_of(dev, stream))
    return page_map


def sinkattn_pages_lists(table, seq_ids, kv_indptr=None, page_indptr=None, page_indices=None,
                         stream=None):
    """What the paged attention reads of the sequences seq_ids: returns
    (kv_indptr [n+1], page_indptr [n+1], page_indices), int32."""
    dev = table.device
    ids_p = _need(seq_ids, "seq_ids", torch.int32, dev, 1)
    n = seq_ids.shape[0]
    if kv_indptr is None:
        kv_indptr = _new((n + 1,), torch.int32, dev, stream)
    if page_indptr is None:
        page_indptr = _new((n + 1,), torch.int32, dev, stream)
    if page_indices is None:
        page_indices = _new((n * table.max_pages,), torch.int32, dev, stream)
    kv_p = _need(kv_indptr, "kv_indptr", torch.int32, dev, (n + 1,))
    pp_p = _need(page_indptr, "page_indptr", torch.int32, dev, (n + 1,))
    pi_p = _need(page_indices, "page_indices", torch.int32, dev, 1)
    _launch(dev, lib().sinkattn_pages_lists, *table._args, ids_p, n, kv_p, pp_p, pi_p,
            page_indices.shape[0], _stream_of(dev, stream))
    return kv_indptr, page_indptr, page_indices


def sinkattn_prefill_backward_workspace_bytes(total_q, num_qo_heads) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().sinkattn_prefill_backward_workspace_bytes(*_i32(total_q, num_qo_heads),
                                                           ctypes.byref(n)))
    return int(n.value)


_back_bytes = functools.lru_cache(maxsize=256)(sinkattn_prefill_backward_workspace_bytes)


def _given_or_new(t, what, shape, dtype, dev, stream):
    if t is None:
        return _new(shape, dtype, dev, stream)
    _need(t, what, dtype, dev, tuple(shape))
    return t


def _workspace(t, need, dev, stream):
    if t is None:
        return _new((max(need, 256),), torch.uint8, dev, stream, kept=False)
    if not torch.is_tensor(t) or t.device != dev or not t.is_contiguous():
        raise SinkAttnError(INVALID_ARG, "workspace must be contiguous and on %s" % dev)
    return t


def sinkattn_prefill_backward(dout, q, k, v, out, lse, sinks, cu_seqlens_q, cu_seqlens_k,
                              max_seqlen_q, max_seqlen_k, num_kv_heads, sm_scale=None, causal=True,
                              window=0, dlse=None, dq=None, dk=None, dv=None, dsinks=None,
                              workspace=None, stream=None):
    """Gradients of sinkattn_prefill: dout bf16 [total_q, Hq, d] is that of
    out, dlse fp32 [total_q, Hq] (or None) that of lse; out and lse are what
    the forward call returned for the same q, k, v, sinks. Returns (dq, dk, dv,
    dsinks), bf16 in the inputs' layouts and fp32 [Hq] (None without sinks). Rows
    behind the last sequence are not written: give zeroed tensors where a padded
    batch's gradients go on."""
    dev = _need_cuda(q, "q")
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    _need(q, "q", bf16, dev, 3)
    total_q, Hq, d = q.shape
    _need(k, "k", bf16, dev, 2)
    Hkv, = _i32(num_kv_heads)
    if Hkv < 1 or k.shape[1] != d or k.shape[0] % Hkv:
        raise SinkAttnError(INVALID_ARG, "k must have shape [%d * total_k, %d], not %s" % (
            Hkv, d, tuple(k.shape)))
    total_k = k.shape[0] // Hkv
    _need(v, "v", bf16, dev, k.shape)
    _need(dout, "dout", bf16, dev, q.shape)
    _need(out, "out", bf16, dev, q.shape)
    _need(lse, "lse", f32, dev, (total_q, Hq))
    if sinks is not None:
        _need(sinks, "sinks", f32, dev, (Hq,))
    elif dsinks is not None:
        raise SinkAttnError(INVALID_ARG, "dsinks without sinks")
    if dlse is not None:
        _need(dlse, "dlse", f32, dev, (total_q, Hq))
    _need(cu_seqlens_q, "cu_seqlens_q", i32, dev, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", i32, dev, cu_seqlens_q.shape)
    batch = cu_seqlens_q.shape[0] - 1
    if batch < 0:
        raise SinkAttnError(INVALID_ARG, "cu_seqlens_q must have an entry at least")
    max_seqlen_q, max_seqlen_k = _i32(max_seqlen_q, max_seqlen_k)
    dq = _given_or_new(dq, "dq", q.shape, bf16, dev, stream)
    dk = _given_or_new(dk, "dk", k.shape, bf16, dev, stream)
    dv = _given_or_new(dv, "dv", k.shape, bf16, dev, stream)
    if sinks is not None:
        dsinks = _given_or_new(dsinks, "dsinks", (Hq,), f32, dev, stream)
    need = _back_bytes(total_q, Hq)
    workspace = _workspace(workspace, need, dev, stream)
    _launch(dev, lib().sinkattn_prefill_backward, dout.data_ptr(), q.data_ptr(), k.data_ptr(),
            v.data_ptr(), out.data_ptr(), lse.data_ptr(),
            None if sinks is None else sinks.data_ptr(),
            None if dlse is None else dlse.data_ptr(), cu_seqlens_q.data_ptr(),
            cu_seqlens_k.data_ptr(), batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv,
            d, _scale(sm_scale, d), 1 if causal else 0, min(int(window), 2 ** 31 - 1),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
            None if dsinks is None else dsinks.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_of(dev, stream))
    return dq, dk, dv, dsinks


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def sinkattn_rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0,
                              original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(angles per position of the rotary_dim / 2 pairs, attention factor) of
    plain, "linear", "ntk" or "yarn" scaled rotary positions; host arithmetic only.
    ("yarn" blends linearly in the pair's index, between borders that are not
    rounded; Rope takes the frequencies of another rule as ``inv_freq``.)"""
    if isinstance(scaling, str) and scaling not in ROPE_SCALINGS:
        raise SinkAttnError(INVALID_ARG, "scaling must be one of %s" % ", ".join(ROPE_SCALINGS))
    code = ROPE_SCALINGS[scaling] if isinstance(scaling, str) else scaling
    rotary_dim, original_len, code = _i32(rotary_dim, original_len, code)
    inv = (ctypes.c_double * max(rotary_dim // 2, 1))()
    att = ctypes.c_float(0.0)
    _check(lib().sinkattn_rope_frequencies(rotary_dim, float(base), code, float(factor),
                                           original_len, float(beta_fast), float(beta_slow), inv,
                                           ctypes.addressof(att)))
    return list(inv)[:rotary_dim // 2], float(att.value)


def sinkattn_rope_turns(inv_freq):
    """Frequencies as the kernels take them: turns per position in units of
    2^-64, as a list of integers in [0, 2^64)."""
    n = len(inv_freq)
    freq = (ctypes.c_double * max(n, 1))(*[float(x) for x in inv_freq])
    turns = (ctypes.c_uint64 * max(n, 1))()
    _check(lib().sinkattn_rope_turns(freq, n, turns))
    return list(turns)[:n]


class Rope:
    """Rotary positions of a head's first ``rotary_dim`` elements, in the half
    layout (pairs (i, i + rotary_dim / 2)) or the ``interleaved`` one (pairs
    (2i, 2i + 1)). The frequencies are those of sinkattn_rope_frequencies, or
    ``inv_freq`` (a sequence of rotary_dim / 2 angles per position) with
    ``attention_factor``, which overrides the scaling's own where given. They
    live on ``device``, so make the object once and keep it; it does not change."""
    __slots__ = ("_turns", "_args", "_inv_freq", "_device")

    def __init__(self, rotary_dim, base=10000.0, interleaved=False, scaling="none", factor=1.0,
                 original_len=0, beta_fast=32.0, beta_slow=1.0, inv_freq=None,
                 attention_factor=None, device="cuda"):
        r, = _i32(rotary_dim)
        if inv_freq is None:
            inv_freq, own = sinkattn_rope_frequencies(r, base, scaling, factor, original_len,
                                                      beta_fast, beta_slow)
        else:
            inv_freq, own = [float(x) for x in inv_freq], 1.0
            if r < 0 or 2 * len(inv_freq) != r:
                raise SinkAttnError(INVALID_ARG, "inv_freq must have rotary_dim / 2 entries")
        own = float(own if attention_factor is None else attention_factor)
        if not math.isfinite(own):
            raise SinkAttnError(INVALID_ARG, "attention_factor must be finite")
        self._inv_freq = tuple(inv_freq)
        # (int64 holds the unsigned words)
        words = [t - 2 ** 64 if t >= 2 ** 63 else t for t in sinkattn_rope_turns(inv_freq)]
        self._turns = torch.tensor(words or [0], dtype=torch.int64).to(device)
        self._device = _need_cuda(self._turns, "device")
        # what every entry point takes beside the words, whose number goes by the first (their
        # address is asked for at each call: a copy of the object has words of its own)
        self._args = (r, 1 if interleaved else 0, own)

    turns = property(lambda self: self._turns)
    rotary_dim = property(lambda self: self._args[0])
    interleaved = property(lambda self: bool(self._args[1]))
    attention_factor = property(lambda self: self._args[2])
    inv_freq = property(lambda self: self._inv_freq)
    device = property(lambda self: self._device)


def _rope_rows(t, what, dev, heads, d, tokens):
    """(address, token stride) of rows [tokens, heads, d] bf16."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.device != dev
            or t.dim() != 3 or t.shape != (tokens, heads, d)):
        raise SinkAttnError(INVALID_ARG, "%s must be bfloat16 %s on %s" % (
            what, (tokens, heads, d), dev))
    at, head, el = t.stride()
    if tokens > 0 and (el != 1 or (head != d and heads > 1)):
        raise SinkAttnError(INVALID_ARG, "the rows of a token of %s must be contiguous" % what)
    return t.data_ptr(), at if tokens > 1 else heads * d


def _rope_common(q, k, v, rope, q_weight, k_weight, positions):
    """(device, tokens, Hq, Hkv, d, addresses and strides, positions, rotation arguments without eps)."""
    dev = _need_cuda(q, "q")
    if q.dim() != 3 or not torch.is_tensor(k) or k.dim() != 3:
        raise SinkAttnError(INVALID_ARG, "q and k must have 3 dimensions")
    tokens, Hq, d = q.shape
    Hkv = k.shape[1]
    rows = [_rope_rows(t, what, dev, heads, d, tokens)
            for t, what, heads in ((q, "q", Hq), (k, "k", Hkv), (v, "v", Hkv))]
    return dev, tokens, Hq, Hkv, d, rows, *_rope_args(rope, q_weight, k_weight, positions, dev, d,
                                                      tokens)


def _rope_args(rope, q_weight, k_weight, positions, dev, d, tokens):
    if not isinstance(rope, Rope) or rope._device != dev:
        raise SinkAttnError(INVALID_ARG, "rope must be a Rope on %s" % dev)
    qw, kw = [None if t is None else _need(t, what, torch.float32, dev, (d,))
              for t, what in ((q_weight, "q_weight"), (k_weight, "k_weight"))]
    pos = None if positions is None else _need(positions, "positions", torch.int32, dev, (tokens,))
    return pos, (rope._turns.data_ptr(), *rope._args, qw, kw)


def sinkattn_rope_qkv(q, k, v, cu_seqlens, rope, q_weight=None, k_weight=None, eps=1e-6,
                      positions=None, q_out=None, k_out=None, v_out=None, stream=None):
    """From a fused projection's rows to what sinkattn_prefill reads: q bf16
    [tokens, Hq, d], k and v [tokens, Hkv, d] (heads of a token contiguous, any
    token stride that is a multiple of 8) are normed per head (q_weight,
    k_weight fp32 [d]; None: not), q and k rotated by ``rope`` at ``positions``
    (int32 [tokens]; None: the index in the sequence). Returns (q [tokens, Hq,
    d], k, v ragged HND [Hkv * tokens, d]); rows behind the last sequence are not
    written."""
    dev, tokens, Hq, Hkv, d, rows, pos, args = _rope_common(q, k, v, rope, q_weight, k_weight,
                                                            positions)
    cu = _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    if cu_seqlens.shape[0] < 1:
        raise SinkAttnError(INVALID_ARG, "cu_seqlens must have an entry at least")
    bf16 = torch.bfloat16
    q_out = _given_or_new(q_out, "q_out", (tokens, Hq, d), bf16, dev, stream)
    k_out = _given_or_new(k_out, "k_out", (Hkv * tokens, d), bf16, dev, stream)
    v_out = _given_or_new(v_out, "v_out", (Hkv * tokens, d), bf16, dev, stream)
    _launch(dev, lib().sinkattn_rope_qkv, *[r[0] for r in rows], *[r[1] for r in rows], cu, pos,
            cu_seqlens.shape[0] - 1, tokens, Hq, Hkv, d, *args, float(eps), q_out.data_ptr(),
            k_out.data_ptr(), v_out.data_ptr(), _stream_of(dev, stream))
    return q_out, k_out, v_out


def sinkattn_rope_qkv_backward_workspace_bytes(tokens, head_dim) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().sinkattn_rope_qkv_backward_workspace_bytes(*_i32(tokens, head_dim),
                                                            ctypes.byref(n)))
    return int(n.value)


_rope_back_bytes = functools.lru_cache(maxsize=256)(sinkattn_rope_qkv_backward_workspace_bytes)


def sinkattn_rope_qkv_backward(dq, dk, dv, cu_seqlens, rope, q=None, k=None, q_weight=None,
                               k_weight=None, eps=1e-6, positions=None, dq_in=None, dk_in=None,
                               dv_in=None, dq_weight=None, dk_weight=None, workspace=None,
                               stream=None):
    """Gradients of sinkattn_rope_qkv from those of its outputs: dq bf16
    [tokens, Hq, d], dk and dv ragged HND. q and k, its inputs, are read where
    they are normed. Returns (dq_in, dk_in, dv_in, dq_weight, dk_weight); by default the
    first three are slices of one [tokens, (Hq + 2 Hkv) * d] gradient of the
    projection's output. Rows behind the last sequence are not written: give zeroed
    tensors where a padded batch's gradients go on."""
    dev = _need_cuda(dq, "dq")
    bf16, f32 = torch.bfloat16, torch.float32
    _need(dq, "dq", bf16, dev, 3)
    tokens, Hq, d = dq.shape
    _need(dk, "dk", bf16, dev, 2)
    if dk.shape[1] != d or (tokens > 0 and (dk.shape[0] % tokens or dk.shape[0] == 0)):
        raise SinkAttnError(INVALID_ARG, "dk must have shape [Hkv * %d, %d], not %s" % (
            tokens, d, tuple(dk.shape)))
    _need(dv, "dv", bf16, dev, dk.shape)
    if tokens > 0:
        Hkv = dk.shape[0] // tokens
    else:   # (the layout of no rows does not tell)
        Hkv = next((t.shape[1] for t in (k, dk_in, dv_in) if torch.is_tensor(t) and t.dim() == 3), 1)
    cu = _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    if cu_seqlens.shape[0] < 1:
        raise SinkAttnError(INVALID_ARG, "cu_seqlens must have an entry at least")
    pos, args = _rope_args(rope, q_weight, k_weight, positions, dev, d, tokens)
    ins = [(None, 0), (None, 0)]
    if q_weight is not None:
        ins[0] = _rope_rows(q, "q", dev, Hq, d, tokens)
    if k_weight is not None:
        ins[1] = _rope_rows(k, "k", dev, Hkv, d, tokens)
    given = (dq_in, dk_in, dv_in)
    if any(t is None for t in given):
        rows = _new((tokens, Hq + 2 * Hkv, d), bf16, dev, stream)
        dq_in, dk_in, dv_in = [a if t is None else t
                               for t, a in zip(given, rows.split((Hq, Hkv, Hkv), 1))]
    outs = [_rope_rows(t, what, dev, heads, d, tokens) for t, what, heads in (
        (dq_in, "dq_in", Hq), (dk_in, "dk_in", Hkv), (dv_in, "dv_in", Hkv))]
    if q_weight is not None:
        dq_weight = _given_or_new(dq_weight, "dq_weight", (d,), f32, dev, stream)
    elif dq_weight is not None:
        raise SinkAttnError(INVALID_ARG, "dq_weight without q_weight")
    if k_weight is not None:
        dk_weight = _given_or_new(dk_weight, "dk_weight", (d,), f32, dev, stream)
    elif dk_weight is not None:
        raise SinkAttnError(INVALID_ARG, "dk_weight without k_weight")
    ws_p, ws_n = None, 0
    if q_weight is not None or k_weight is not None:
        need = _rope_back_bytes(tokens, d)
        workspace = _workspace(workspace, need, dev, stream)
        ws_p, ws_n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(dev, lib().sinkattn_rope_qkv_backward, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
            ins[0][0], ins[1][0], ins[0][1], ins[1][1], cu, pos, cu_seqlens.shape[0] - 1, tokens,
            Hq, Hkv, d, *args, float(eps), *[o[0] for o in outs], *[o[1] for o in outs],
            None if dq_weight is None else dq_weight.data_ptr(),
            None if dk_weight is None else dk_weight.data_ptr(), ws_p, ws_n,
            _stream_of(dev, stream))
    return dq_in, dk_in, dv_in, dq_weight, dk_weight


def _rope_append(entry, pool_dtype, scales, q, k, v, positions, slots, rope, k_pages, v_pages,
                 q_weight, k_weight, eps, q_out, stream):
    dev, tokens, Hq, Hkv, d, rows, pos, args = _rope_common(q, k, v, rope, q_weight, k_weight,
                                                            positions)
    if pos is None:
        raise SinkAttnError(INVALID_ARG, "positions must be a tensor")
    s_p = _need(slots, "slots", torch.int32, dev, (tokens,))
    kp_p = _need(k_pages, "k_pages", pool_dtype, dev, 4)
    num_pages, pool_heads, page_size, pool_d = k_pages.shape
    if pool_heads != Hkv or pool_d != d:
        raise SinkAttnError(INVALID_ARG, "k has %d heads of %d, the pools %d of %d" % (
            Hkv, d, pool_heads, pool_d))
    vp_p = _need(v_pages, "v_pages", pool_dtype, dev, k_pages.shape)
    scale_p = [_need(t, what, torch.float32, dev, (Hkv,))
               for t, what in zip(scales, ("k_scale", "v_scale"))]
    q_out = _given_or_new(q_out, "q_out", (tokens, Hq, d), torch.bfloat16, dev, stream)
    _launch(dev, entry, *[r[0] for r in rows], *[r[1] for r in rows], pos, s_p, tokens, Hq, Hkv, d,
            *args, float(eps), *scale_p, q_out.data_ptr(), kp_p, vp_p, num_pages, page_size,
            _stream_of(dev, stream))
    return q_out


def sinkattn_rope_append_paged(q, k, v, positions, slots, rope, k_pages, v_pages, q_weight=None,
                               k_weight=None, eps=1e-6, q_out=None, stream=None):
    """sinkattn_append_paged with the norm and rotation of sinkattn_rope_qkv on
    the way: q, k, v are a fused projection's rows, positions and slots int32
    [tokens]. k and v go to the pools; returns the rotated q, [tokens, Hq, d]."""
    return _rope_append(lib().sinkattn_rope_append_paged, torch.bfloat16, (), q, k, v, positions,
                        slots, rope, k_pages, v_pages, q_weight, k_weight, eps, q_out, stream)


def sinkattn_rope_append_paged_fp8(q, k, v, positions, slots, rope, k_scale, v_scale, k_pages,
                                   v_pages, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
                                   stream=None):
    """sinkattn_rope_append_paged into pools of e4m3 codes (uint8): the code
    nearest to the fp32 quotient of the rotated key and scale[head] (ties to even,
    saturating at 448)."""
    return _rope_append(lib().sinkattn_rope_append_paged_fp8, torch.uint8, (k_scale, v_scale), q, k,
                        v, positions, slots, rope, k_pages, v_pages, q_weight, k_weight, eps,
                        q_out, stream)


PREFILL_KERNELS = {"auto": 0, "one_block": 1, "persistent": 2}


def sinkattn_set_prefill_kernel(kind) -> None:
    """Selects the prefill launch process-wide: "auto", "one_block" or
    "persistent" (or the integer codes of include/sinkattn.h)."""
    code = PREFILL_KERNELS[kind] if isinstance(kind, str) else int(kind)
    _check(lib().sinkattn_set_prefill_kernel(code))


def sinkattn_status_string(status: int) -> str:
    return status_name(status)


def sinkattn_last_error() -> str:
    return lib().sinkattn_last_error().decode()


def sinkattn_debug_status(stream=None) -> int:
    st = ctypes.c_int(0)
    s = ctypes.c_void_p(0) if stream is None and not torch.cuda.is_available() else (
        _stream(torch.empty(0, device="cuda"), stream))
    _check(lib().sinkattn_debug_status(s, ctypes.byref(st)))
    return int(st.value)


def sinkattn_debug_set_hooks(wait_limit_cycles: int = 0, skip_tile: int = -1) -> None:
    """Test only: bounded-wait limit in SM clock cycles (0: the default) and
    the KV tile the first thread block's producer leaves out (-1: none)."""
    _check(lib().sinkattn_debug_set_hooks(int(wait_limit_cycles), int(skip_tile)))
