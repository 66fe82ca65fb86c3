"""Paged-KV attention for GB300 (sm_103a): Python binding of libpa.so.

Thin ctypes marshalling over the C ABI declared in include/pa.h: every
function here checks tensor dtypes/devices, passes raw pointers, sizes and
the current CUDA stream to the library, and raises PagedAttentionError on a
non-OK status.  All computation happens in the library's CUDA kernels; there
is no CPU or PyTorch fallback, and importing the binding fails loudly when
libpa.so has not been built (see build.py).

Entry points (same names as the C ABI without the ``pa_`` prefix):
  store_kvcache, slot_mapping_decode, slot_mapping_prefill,
  decode_workspace_size, decode, decode_static, prefill_varlen,
  sample_gumbel, set_checked, get_device_error;
  kvcache_q8, store_kvcache_q8, load_kvcache_q8, decode_q8_workspace,
  decode_q8 (the 8-bit pool); logprobs;
  rope_frequencies, rope, rope_store_kvcache, tree_metadata,
  decode_tree_workspace, decode_tree, verify_drafts, compact_kvcache
  (speculative decoding);
  block_manager.BlockManager wraps the host block manager (pa_bm_*).
"""
from __future__ import annotations

import ctypes as C
import math
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA, PA_ERR_DEVICE_CHECK = range(6)
(PA_DEV_TIMEOUT, PA_DEV_BAD_SLOT, PA_DEV_BAD_CONTEXT, PA_DEV_BAD_BLOCK, PA_DEV_BAD_SEQLENS, PA_DEV_SMEM_ALIGN,
 PA_DEV_BAD_TEMPERATURE, PA_DEV_BAD_TOKEN, PA_DEV_BAD_TREE) = range(1, 10)
PA_Q8_E4M3, PA_Q8_INT8 = range(2)
PA_ROPE_PLAIN, PA_ROPE_LINEAR, PA_ROPE_NTK, PA_ROPE_YARN = range(4)

# Every symbol include/pa.h declares, with its ctypes signature.
_i32, _i64, _sz, _f32, _vp = C.c_int32, C.c_int64, C.c_size_t, C.c_float, C.c_void_p
SIGNATURES = {
    "pa_version": (C.c_int, []),
    "pa_status_str": (C.c_char_p, [C.c_int]),
    "pa_last_error_message": (C.c_char_p, []),
    "pa_store_kvcache": (C.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _vp]),
    "pa_slot_mapping_decode": (C.c_int, [_vp, _vp, _i32, _vp, _i32, _i32, _vp]),
    "pa_slot_mapping_prefill": (C.c_int, [_vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp]),
    "pa_decode_workspace_size": (_sz, [_i32, _i32, _i32]),
    "pa_decode": (C.c_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                            _i32, _f32, _vp, _sz, _vp]),
    "pa_decode_static": (C.c_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                   _i32, _f32, _vp]),
    "pa_decode_static_scratch": (C.c_int, [C.POINTER(_vp), C.POINTER(_sz)]),
    "pa_decode_shared_prefix_workspace_size": (_sz, [_i32, _i32, _i32]),
    "pa_decode_shared_prefix": (C.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                          _i32, _i32, _i32, _i32, _f32, _vp, _sz, _vp]),
    "pa_decode_store": (C.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                  _i32, _i32, _i32, _i32, _f32, _vp, _sz, _vp]),
    "pa_prefill_varlen": (C.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i32,
                                    _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp]),
    "pa_prefill_store_workspace_size": (C.c_size_t, []),
    "pa_prefill_store_varlen": (C.c_int, [_vp, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp,
                                          _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp,
                                          C.c_size_t, _vp]),
    "pa_sample_gumbel": (C.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _i32, _vp]),
    "pa_logprobs": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _vp]),
    "pa_store_kvcache_q8": (C.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                      _i32, _vp]),
    "pa_load_kvcache_q8": (C.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                     _i32, _vp]),
    "pa_decode_q8_workspace_size": (_sz, [_i32, _i32, _i32]),
    "pa_decode_q8": (C.c_int, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                               _i32, _i32, _f32, _vp, _sz, _vp]),
    "pa_decode_store_q8": (C.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32,
                                     _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _sz, _vp]),
    "pa_rope_frequencies": (C.c_int, [_vp, C.POINTER(C.c_float), _i32, C.c_double, _i32, C.c_double, C.c_double,
                                      C.c_double, C.c_double]),
    "pa_rope": (C.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _f32, _i32,
                          _i32, _i32, _i32, _vp]),
    "pa_rope_store_kvcache": (C.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _f32, _vp,
                                        _vp, _f32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _vp]),
    "pa_tree_metadata": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]),
    "pa_decode_tree_workspace_size": (_sz, [_i32, _i32, _i32, _i32]),
    "pa_decode_tree": (C.c_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                 _i32, _f32, _vp, _sz, _vp]),
    "pa_verify_drafts": (C.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _i32, _vp,
                                   _i32, _i32, _i32, _vp]),
    "pa_compact_kvcache": (C.c_int, [_vp, _i64, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                     _i32, _i32, _vp]),
    "pa_set_checked": (C.c_int, [_i32]),
    # host block manager
    "pa_bm_create": (C.c_int, [_i32, _i32, C.POINTER(_vp)]),
    "pa_bm_destroy": (None, [_vp]),
    "pa_bm_seq_add": (C.c_int, [_vp, _vp, _i32, C.POINTER(_i32)]),
    "pa_bm_seq_append_token": (C.c_int, [_vp, _i32, _i64]),
    "pa_bm_seq_set_num_cached_tokens": (C.c_int, [_vp, _i32, _i32]),
    "pa_bm_seq_info": (C.c_int, [_vp, _i32, C.POINTER(_i32), C.POINTER(_i32), C.POINTER(_i32)]),
    "pa_bm_can_allocate": (_i32, [_vp, _i32]),
    "pa_bm_allocate": (C.c_int, [_vp, _i32, _i32]),
    "pa_bm_deallocate": (C.c_int, [_vp, _i32]),
    "pa_bm_can_append": (_i32, [_vp, _i32]),
    "pa_bm_may_append": (C.c_int, [_vp, _i32]),
    "pa_bm_hash_blocks": (C.c_int, [_vp, _i32, _i32]),
    "pa_bm_seq_block_table": (_i32, [_vp, _i32, _vp, _i32]),
    "pa_bm_block_tables": (C.c_int, [_vp, _vp, _i32, _vp, _i32]),
    "pa_bm_free_block_ids": (_i32, [_vp, _vp, _i32]),
    "pa_bm_block_info": (C.c_int, [_vp, _i32, C.POINTER(_i32), C.POINTER(_i32), C.POINTER(C.c_uint64),
                                   C.POINTER(_i32)]),
    "pa_bm_lookup_hash": (_i32, [_vp, C.c_uint64]),
    "pa_bm_num_hashes": (_i32, [_vp]),
    "pa_bm_block_hash": (C.c_uint64, [_vp, _i32, _i32, C.c_uint64]),
    "pa_bm_xxh64": (C.c_uint64, [_vp, _sz, C.c_uint64]),
    "pa_get_device_error": (C.c_int, [_vp, C.POINTER(_i32), C.POINTER(_i64)]),
}

_LIB = None


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [status {status}]")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load libpa.so and declare its signatures (no GPU needed)."""
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with paged_kv_cache_store_gb300.build.build()")
    lib = C.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def lib():
    global _LIB
    if _LIB is None:
        _LIB = load_library()
    return _LIB


def _check(status: int, what: str):
    if status != PA_OK:
        L = lib()
        msg = (L.pa_last_error_message() or b"").decode(errors="replace")
        name = (L.pa_status_str(status) or b"").decode()
        raise PagedAttentionError(status, f"{what}: {name}: {msg}")


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _row_stride(t, name):
    """Elements between rows of a [N, ...] tensor whose trailing dims are contiguous."""
    inner = 1
    for d in t.shape[1:]:
        inner *= d
    if t.shape[0] == 0:
        return inner
    if t.dim() > 1 and not t[0].is_contiguous():
        raise ValueError(f"{name}: each row must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else inner


def store_kvcache(key, value, k_cache, v_cache, slot_mapping, stream=None):
    """Scatter key/value [N, Hkv, D] (bf16, rows may be strided) into the pool
    [num_blocks, B, Hkv, D] at slot_mapping (int32 [N], negatives skipped)."""
    for t, n in ((key, "key"), (value, "value"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(slot_mapping, torch.int32, "slot_mapping")
    nb, B, hkv, d = k_cache.shape
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    n = key.shape[0]
    if slot_mapping.numel() != n or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous with one entry per token")
    _check(lib().pa_store_kvcache(_ptr(key), _row_stride(key, "key"), _ptr(value),
                                  _row_stride(value, "value"), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(slot_mapping), n, hkv, d, nb * B, _stream(stream)),
           "pa_store_kvcache")


def slot_mapping_decode(block_tables, context_lens, block_size, out=None, stream=None):
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    batch = context_lens.numel()
    if out is None:
        out = torch.empty(batch, dtype=torch.int32, device=context_lens.device)
    _check(lib().pa_slot_mapping_decode(_ptr(out), _ptr(block_tables.contiguous()), block_tables.shape[1],
                                        _ptr(context_lens), batch, block_size, _stream(stream)),
           "pa_slot_mapping_decode")
    return out


def slot_mapping_prefill(block_tables, cu_seqlens_q, cu_seqlens_k, block_size, total_q=None,
                         out=None, stream=None):
    _need(block_tables, torch.int32, "block_tables")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    num_seqs = cu_seqlens_q.numel() - 1
    if total_q is None:
        total_q = int(cu_seqlens_q[-1].item())
    if out is None:
        out = torch.empty(total_q, dtype=torch.int32, device=cu_seqlens_q.device)
    _check(lib().pa_slot_mapping_prefill(_ptr(out), _ptr(block_tables.contiguous()), block_tables.shape[1],
                                         _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), num_seqs, total_q,
                                         block_size, _stream(stream)),
           "pa_slot_mapping_prefill")
    return out


def decode_workspace_size(num_q_heads, num_kv_heads, head_dim) -> int:
    return int(lib().pa_decode_workspace_size(num_q_heads, num_kv_heads, head_dim))


def decode_workspace(num_q_heads, num_kv_heads, head_dim, device="cuda", shared_prefix=False):
    """Allocate (with torch) a zero-filled workspace for pa_decode (at most
    about 6.4 MB; it depends only on the GQA group), or, with shared_prefix,
    for pa_decode_shared_prefix (about 8.6 MB more).  The calls leave it
    zeroed, so it can be reused by any number of calls on one stream."""
    n = (int(lib().pa_decode_shared_prefix_workspace_size(num_q_heads, num_kv_heads, head_dim)) if shared_prefix
         else decode_workspace_size(num_q_heads, num_kv_heads, head_dim))
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def decode(q, k_cache, v_cache, block_tables, context_lens, softmax_scale=None, workspace=None, out=None,
           stream=None, new_k=None, new_v=None, shared_prefix=False):
    """Paged decode attention.  q [batch, Hq, D] bf16 (rows may be strided);
    caches [num_blocks, B, Hkv, D]; block_tables int32 [batch, max_blocks];
    context_lens int32 [batch].  Returns out [batch, Hq, D] bf16.  With
    new_k / new_v ([batch, Hkv, D] bf16, rows may be strided) the kernel first
    stores them at position context_lens-1 (pa_decode_store); no other row's
    context may hold a position that is stored (store_kvcache first there).  With
    shared_prefix, sequences that share leading blocks read them once
    (pa_decode_shared_prefix; its workspace is larger)."""
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    batch, hq, d = q.shape
    nb, B, hkv, _ = k_cache.shape
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and block_tables.is_contiguous()):
        raise ValueError("caches and block_tables must be contiguous")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    mb = block_tables.shape[1]
    if workspace is None:
        workspace = decode_workspace(hq, hkv, d, q.device, shared_prefix=shared_prefix)
    if out is None:
        out = torch.empty(batch, hq, d, dtype=torch.bfloat16, device=q.device)
    if shared_prefix:
        if new_k is not None or new_v is not None:
            _need(new_k, torch.bfloat16, "new_k")
            _need(new_v, torch.bfloat16, "new_v")
        nk_args = ((_ptr(new_k), _row_stride(new_k, "new_k"), _ptr(new_v), _row_stride(new_v, "new_v"))
                   if new_k is not None else (None, 0, None, 0))
        _check(lib().pa_decode_shared_prefix(_ptr(out), _ptr(q), _row_stride(q, "q"), *nk_args, _ptr(k_cache),
                                             _ptr(v_cache), _ptr(block_tables), mb, _ptr(context_lens), batch, hq, hkv,
                                             d, B, nb, float(softmax_scale), _ptr(workspace), workspace.numel(),
                                             _stream(stream)),
               "pa_decode_shared_prefix")
        return out
    if new_k is not None or new_v is not None:
        _need(new_k, torch.bfloat16, "new_k")
        _need(new_v, torch.bfloat16, "new_v")
        _check(lib().pa_decode_store(_ptr(out), _ptr(q), _row_stride(q, "q"), _ptr(new_k), _row_stride(new_k, "new_k"),
                                     _ptr(new_v), _row_stride(new_v, "new_v"), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(block_tables), mb, _ptr(context_lens), batch, hq, hkv, d, B, nb,
                                     float(softmax_scale), _ptr(workspace), workspace.numel(), _stream(stream)),
               "pa_decode_store")
        return out
    _check(lib().pa_decode(_ptr(out), _ptr(q), _row_stride(q, "q"), _ptr(k_cache), _ptr(v_cache),
                           _ptr(block_tables), mb, _ptr(context_lens), batch, hq, hkv, d, B, nb,
                           float(softmax_scale), _ptr(workspace), workspace.numel(), _stream(stream)),
           "pa_decode")
    return out


def decode_static(q, k_cache, v_cache, block_tables, context_lens, softmax_scale=None, out=None, stream=None):
    """pa_decode without a workspace: for callers that must not allocate device
    memory.  The split scratch is an 8 MiB array built into the library (shared
    by all calls, so calls that may overlap on the GPU must be serialised).
    Only `out` is allocated here, and only when the caller passes none."""
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    batch, hq, d = q.shape
    nb, B, hkv, _ = k_cache.shape
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(batch, hq, d, dtype=torch.bfloat16, device=q.device)
    _check(lib().pa_decode_static(_ptr(out), _ptr(q), _row_stride(q, "q"), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), batch, hq, hkv,
                                  d, B, nb, float(softmax_scale), _stream(stream)),
           "pa_decode_static")
    return out


def prefill_store_workspace(device="cuda"):
    """Zero-filled workspace for prefill_varlen(..., new_k=, new_v=) (a grid
    barrier's counter; the call leaves it as found, reusable on one stream)."""
    n = int(lib().pa_prefill_store_workspace_size())
    return torch.zeros(n, dtype=torch.uint8, device=device)


def prefill_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale=None,
                   block_tables=None, causal=True, out=None, stream=None, new_k=None, new_v=None, workspace=None):
    """Varlen prefill attention.  q [total_q, Hq, D]; with block_tables, k/v are
    the caches [num_blocks, B, Hkv, D]; without, contiguous [total_k, Hkv, D].
    With new_k / new_v ([total_q, Hkv, D], the uncached suffix in q's order;
    block_tables required) the same launch first stores them into the caches
    (pa_prefill_store_varlen)."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    tq, hq, d = q.shape
    if block_tables is not None:
        _need(block_tables, torch.int32, "block_tables")
        nb, B, hkv, _ = k.shape
        mb, kv_stride, tk = block_tables.shape[1], 0, 0
    else:
        tk, hkv, _ = k.shape
        nb, B, mb, kv_stride = 0, 16, 0, _row_stride(k, "k")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(tq, hq, d, dtype=torch.bfloat16, device=q.device)
    if new_k is not None or new_v is not None:
        if new_k is None or new_v is None or block_tables is None:
            raise ValueError("the fused store needs new_k, new_v and block_tables")
        _need(new_k, torch.bfloat16, "new_k")
        _need(new_v, torch.bfloat16, "new_v")
        if new_k.shape[0] != tq or new_v.shape[0] != tq:
            raise ValueError("new_k / new_v need one row per query token")
        if workspace is None:
            workspace = prefill_store_workspace(q.device)
        _check(lib().pa_prefill_store_varlen(
            _ptr(out), _ptr(q), _row_stride(q, "q"), tq, _ptr(new_k), _row_stride(new_k, "new_k"), _ptr(new_v),
            _row_stride(new_v, "new_v"), _ptr(k), _ptr(v), _ptr(block_tables), mb, _ptr(cu_seqlens_q),
            _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k), hq, hkv, d, B, nb,
            float(softmax_scale), 1 if causal else 0, _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream)), "pa_prefill_store_varlen")
        return out
    _check(lib().pa_prefill_varlen(_ptr(out), _ptr(q), _row_stride(q, "q"), tq, _ptr(k), _ptr(v), kv_stride, tk,
                                   _ptr(block_tables), mb, _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                   cu_seqlens_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k), hq, hkv,
                                   d, B, nb, float(softmax_scale), 1 if causal else 0, _stream(stream)),
           "pa_prefill_varlen")
    return out


def sample_gumbel(logits, temperatures, exp_noise, out=None, stream=None):
    """One token per row: argmax softmax(logits / T) / max(E, 1e-10) (Gumbel-max).
    logits [batch, vocab] bf16 or fp32 (rows may be strided); temperatures
    fp32 [batch]; exp_noise fp32 [batch, vocab] of Exp(1) draws (the caller's
    random state).  Returns int32 [batch]."""
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("logits must be bfloat16 or float32")
    _need(temperatures, torch.float32, "temperatures")
    _need(exp_noise, torch.float32, "exp_noise")
    batch, vocab = logits.shape
    if tuple(exp_noise.shape) != (batch, vocab) or tuple(temperatures.shape) != (batch,):
        raise ValueError("exp_noise must be [batch, vocab] and temperatures [batch]")
    if logits.stride(1) != 1 or exp_noise.stride(1) != 1 or not temperatures.is_contiguous():
        raise ValueError("rows must be contiguous")
    if out is None:
        out = torch.empty(batch, dtype=torch.int32, device=logits.device)
    _check(lib().pa_sample_gumbel(_ptr(out), _ptr(logits), logits.stride(0), 1 if logits.dtype == torch.float32 else 0,
                                  _ptr(temperatures), _ptr(exp_noise), exp_noise.stride(0), batch, vocab,
                                  _stream(stream)),
           "pa_sample_gumbel")
    return out


# ---------------------------------------------------------------------------
# The 8-bit pool: codes [num_blocks, Hkv, B, 128] (float8_e4m3fn or int8) and
# one scale byte per token and head [num_blocks, Hkv, B] (uint8).
# ---------------------------------------------------------------------------
_Q8_FORMATS = {torch.float8_e4m3fn: PA_Q8_E4M3, torch.int8: PA_Q8_INT8}


def kvcache_q8(num_blocks, block_size, num_kv_heads, head_dim=128, dtype=torch.float8_e4m3fn, device="cuda"):
    """Allocate one layer's 8-bit pool, zero-filled: (k_cache, v_cache, k_scale, v_scale)."""
    if dtype not in _Q8_FORMATS:
        raise TypeError(f"dtype must be float8_e4m3fn or int8, got {dtype}")
    shape = (num_blocks, num_kv_heads, block_size, head_dim)
    return (*(torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2)),
            *(torch.zeros(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)))


def _q8_pool(k_cache, v_cache, k_scale, v_scale):
    """Checks the four tensors of an 8-bit pool; returns its shape and format."""
    dtype = k_cache.dtype
    fmt = _Q8_FORMATS.get(dtype)
    shape = k_cache.shape
    if fmt is None or len(shape) != 4:
        raise TypeError("k_cache must be a [num_blocks, Hkv, B, D] tensor of float8_e4m3fn or int8")
    if v_cache.dtype is not dtype or k_scale.dtype is not torch.uint8 or v_scale.dtype is not torch.uint8:
        raise TypeError(f"v_cache must be {dtype} and k_scale / v_scale {torch.uint8}, got {v_cache.dtype}, "
                        f"{k_scale.dtype}, {v_scale.dtype}")
    if v_cache.shape != shape or not (k_scale.shape == v_scale.shape == shape[:3]):
        raise ValueError("k_cache / v_cache must be [num_blocks, Hkv, B, D] and k_scale / v_scale [num_blocks, Hkv, B]")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous()):
        raise ValueError("caches and scales must be contiguous")
    return shape, fmt


def _placed(stream, first, *others):
    """Where a call runs: on its tensors' device (which all must share) and on
    `stream`, default that device's current stream.  Returns None when both are
    current already, else a context in which they are, so that what the call
    allocates belongs to the stream that it runs on."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    if dev < 0:
        raise TypeError("tensors must be CUDA tensors")
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError(f"stream of device {stream.device_index}, tensors on {first.device}")
        return torch.cuda.stream(stream)  # makes its device current as well
    return None if dev == _current_device() else torch.cuda.device(dev)


def _rows(t, name, n, heads, d):
    """Elements between the rows of a bf16 [n, heads, d] tensor (n None: any),
    each contiguous."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or (n is not None and shape[0] != n):
        raise ValueError(f"{name} must be [{'N' if n is None else n}, {heads}, {d}], got {list(shape)}")
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (heads > 1 and s1 != d):
        raise ValueError(f"{name}: each row must be contiguous")
    return s0 if shape[0] > 1 else heads * d


def _fits(n, name):
    """Sizes are int32 in the library, and ctypes would cut longer ones down."""
    if not -(1 << 31) <= n < 1 << 31:
        raise ValueError(f"{name} {n} does not fit 32 bits")


def _slots(slot_mapping, n=None):
    _need(slot_mapping, torch.int32, "slot_mapping")
    if slot_mapping.dim() != 1 or not slot_mapping.is_contiguous() or (n is not None and slot_mapping.shape[0] != n):
        raise ValueError("slot_mapping must be contiguous with one entry per token")
    _fits(slot_mapping.shape[0], "number of tokens")


def _raw_stream():
    """The current device's current stream (torch's raw getter takes 0.1 us,
    building a Stream object 3 us)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())


def store_kvcache_q8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, stream=None):
    """Quantise key/value [N, Hkv, 128] (bf16, rows may be strided) into the
    8-bit pool at slot_mapping (int32 [N], negatives skipped)."""
    (nb, hkv, B, d), fmt = _q8_pool(k_cache, v_cache, k_scale, v_scale)
    ks = _rows(key, "key", None, hkv, d)
    n = key.shape[0]
    vs = _rows(value, "value", n, hkv, d)
    _slots(slot_mapping, n)
    ctx = _placed(stream, key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping)
    if ctx is not None:
        with ctx:
            return store_kvcache_q8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping)
    _check(lib().pa_store_kvcache_q8(key.data_ptr(), ks, value.data_ptr(), vs, k_cache.data_ptr(),
                                     v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                     slot_mapping.data_ptr(), n, hkv, d, B, nb, fmt, _raw_stream()),
           "pa_store_kvcache_q8")


def load_kvcache_q8(k_cache, v_cache, k_scale, v_scale, slot_mapping, out_k=None, out_v=None, stream=None):
    """Read rows of the 8-bit pool back: (k, v), bf16 [N, Hkv, 128], the rows of
    slots slot_mapping (int32 [N], may repeat; zeros for negatives).  out_k /
    out_v may be given (rows may be strided)."""
    (nb, hkv, B, d), fmt = _q8_pool(k_cache, v_cache, k_scale, v_scale)
    _slots(slot_mapping)
    n = slot_mapping.shape[0]
    ctx = _placed(stream, k_cache, v_cache, k_scale, v_scale, slot_mapping, out_k, out_v)
    if ctx is not None:
        with ctx:
            return load_kvcache_q8(k_cache, v_cache, k_scale, v_scale, slot_mapping, out_k, out_v)
    ks = hkv * d if out_k is None else _rows(out_k, "out_k", n, hkv, d)
    vs = hkv * d if out_v is None else _rows(out_v, "out_v", n, hkv, d)
    k = torch.empty(n, hkv, d, dtype=torch.bfloat16, device=k_cache.device) if out_k is None else out_k
    v = torch.empty(n, hkv, d, dtype=torch.bfloat16, device=k_cache.device) if out_v is None else out_v
    _check(lib().pa_load_kvcache_q8(k.data_ptr(), ks, v.data_ptr(), vs, k_cache.data_ptr(), v_cache.data_ptr(),
                                    k_scale.data_ptr(), v_scale.data_ptr(), slot_mapping.data_ptr(), n, hkv, d, B, nb,
                                    fmt, _raw_stream()), "pa_load_kvcache_q8")
    return k, v


def decode_q8_workspace(num_q_heads, num_kv_heads, head_dim=128, device="cuda"):
    """Zero-filled workspace for decode_q8 (its size depends only on the GQA
    group; one of a larger group serves the smaller ones too); the calls leave
    it ready for the next one on the same stream."""
    n = int(lib().pa_decode_q8_workspace_size(num_q_heads, num_kv_heads, head_dim))
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def decode_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, softmax_scale=None, workspace=None,
              out=None, stream=None, new_k=None, new_v=None):
    """Paged decode attention over the 8-bit pool.  q [batch, Hq, 128] bf16
    (rows may be strided); block_tables int32 [batch, max_blocks];
    context_lens int32 [batch].  Returns out [batch, Hq, 128] bf16.  With
    new_k / new_v ([batch, Hkv, 128] bf16, rows may be strided) the kernel first
    stores them at position context_lens-1 (pa_decode_store_q8); no other row's
    context may hold a position that is stored (store_kvcache_q8 first there)."""
    (nb, hkv, B, d), fmt = _q8_pool(k_cache, v_cache, k_scale, v_scale)
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    if q.dim() != 3:
        raise ValueError(f"q must be [batch, Hq, {d}]")
    batch, hq, _ = q.shape
    qs = _rows(q, "q", batch, hq, d)
    if block_tables.dim() != 2 or block_tables.shape[0] != batch or context_lens.shape != (batch,):
        raise ValueError("block_tables must be [batch, max_blocks] and context_lens [batch]")
    _fits(batch, "batch")
    _fits(block_tables.shape[1], "width of block_tables")
    if not (block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("block_tables and context_lens must be contiguous")
    if out is not None:
        _need(out, torch.bfloat16, "out")
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be contiguous and of q's shape")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    stores = new_k is not None or new_v is not None
    if stores:
        if new_k is None or new_v is None:
            raise ValueError("the fused store needs new_k and new_v")
        nks, nvs = _rows(new_k, "new_k", batch, hkv, d), _rows(new_v, "new_v", batch, hkv, d)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    ctx = _placed(stream, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, workspace, out, new_k,
                  new_v)
    if ctx is not None:
        with ctx:
            return decode_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, workspace, out,
                             None, new_k, new_v)
    if workspace is None:
        workspace = decode_q8_workspace(hq, hkv, d, q.device)
    if out is None:
        out = torch.empty(batch, hq, d, dtype=torch.bfloat16, device=q.device)
    if stores:
        _check(lib().pa_decode_store_q8(out.data_ptr(), q.data_ptr(), qs, new_k.data_ptr(), nks, new_v.data_ptr(), nvs,
                                        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), batch,
                                        hq, hkv, d, B, nb, fmt, scale, workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), _raw_stream()),
               "pa_decode_store_q8")
        return out
    _check(lib().pa_decode_q8(out.data_ptr(), q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(),
                              k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
                              context_lens.data_ptr(), batch, hq, hkv, d, B, nb, fmt, scale, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _raw_stream()), "pa_decode_q8")
    return out


class Logprobs(NamedTuple):
    """What logprobs returns; the last two are None for top_k == 0."""
    logprobs: torch.Tensor                # fp32 [rows]
    entropy: torch.Tensor                 # fp32 [rows]
    top_ids: Optional[torch.Tensor]       # int32 [rows, top_k]
    top_logprobs: Optional[torch.Tensor]  # fp32 [rows, top_k]


def logprobs(logits, tokens, top_k=0, temperatures=None, out=None, stream=None):
    """Log probabilities of tokens (int32 [rows]) under softmax(logits / T),
    the entropy and the top_k largest entries per row.  logits [rows, vocab]
    bf16 or fp32 (rows may be strided); temperatures fp32 [rows] or None.
    `out`, a Logprobs of contiguous tensors, is filled and returned."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("logits must be a bfloat16 or float32 tensor")
    _need(tokens, torch.int32, "tokens")
    if logits.dim() != 2 or tokens.shape != logits.shape[:1]:
        raise ValueError("logits must be [rows, vocab] and tokens [rows]")
    rows, vocab = logits.shape
    top_k = int(top_k)
    for n, name in ((rows, "number of rows"), (vocab, "vocabulary"), (top_k, "top_k")):
        _fits(n, name)
    if not tokens.is_contiguous() or (vocab > 1 and logits.stride(1) != 1):
        raise ValueError("rows must be contiguous")
    if temperatures is not None:
        _need(temperatures, torch.float32, "temperatures")
        if temperatures.shape != (rows,) or not temperatures.is_contiguous():
            raise ValueError("temperatures must be contiguous [rows]")
    if out is not None:
        for t, dtype, shape, name in ((out[0], torch.float32, (rows,), "logprobs"),
                                      (out[1], torch.float32, (rows,), "entropy"),
                                      (out[2], torch.int32, (rows, top_k), "top_ids"),
                                      (out[3], torch.float32, (rows, top_k), "top_logprobs")):
            if t is None and top_k == 0 and len(shape) == 2:
                continue
            _need(t, dtype, name)
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"out.{name} must be contiguous {list(shape)}")
    ctx = _placed(stream, logits, tokens, temperatures, *(out or ()))
    if ctx is not None:
        with ctx:
            return logprobs(logits, tokens, top_k, temperatures, out)
    if out is None:
        dev, k = logits.device, min(max(top_k, 0), vocab)
        out = Logprobs(torch.empty(rows, dtype=torch.float32, device=dev),
                       torch.empty(rows, dtype=torch.float32, device=dev),
                       torch.empty(rows, k, dtype=torch.int32, device=dev) if k else None,
                       torch.empty(rows, k, dtype=torch.float32, device=dev) if k else None)
    # A lone row's stride does not matter; the library wants it well-formed.
    stride = logits.stride(0) if rows > 1 else -(-vocab // 8) * 8
    tops = (None, None) if out[2] is None or out[3] is None else (out[2].data_ptr(), out[3].data_ptr())
    _check(lib().pa_logprobs(out[0].data_ptr(), out[1].data_ptr(), *tops, logits.data_ptr(), stride,
                             1 if logits.dtype is torch.float32 else 0,
                             None if temperatures is None else temperatures.data_ptr(), tokens.data_ptr(), rows, vocab,
                             top_k, _raw_stream()), "pa_logprobs")
    return out


# ---------------------------------------------------------------------------
# Speculative decoding: trees of drafted tokens, node 0 the token that they
# continue, node i > 0 under parents[i] < i; at most 64 nodes a sequence.
# ---------------------------------------------------------------------------
class Rope(NamedTuple):
    """Rotary frequencies as rope_frequencies makes them."""
    freqs: torch.Tensor  # int64 [rotary_dim / 2] on the GPU: turns per position, fractions of 2^64
    gain: float          # multiplies what is rotated (1 but for yarn)
    interleaved: bool    # pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2)


_ROPE_SCALINGS = {"linear": PA_ROPE_LINEAR, "ntk": PA_ROPE_NTK, "yarn": PA_ROPE_YARN}


def rope_frequencies(rotary_dim=128, theta=10000.0, scaling=None, interleaved=False, device="cuda"):
    """Rotary frequencies for rope / rope_store_kvcache, made once per model.
    scaling: None, ("linear", factor), ("ntk", factor) or ("yarn", factor,
    original_context[, beta_fast, beta_slow])."""
    kind, args = PA_ROPE_PLAIN, ()
    if scaling is not None:
        if not isinstance(scaling, (tuple, list)) or not scaling or scaling[0] not in _ROPE_SCALINGS:
            raise ValueError(f"scaling must be None or a tuple that starts with one of {sorted(_ROPE_SCALINGS)}")
        kind, args = _ROPE_SCALINGS[scaling[0]], tuple(float(x) for x in scaling[1:])
        if len(args) not in ((2, 4) if kind == PA_ROPE_YARN else (1,)):
            raise ValueError("scaling must be (kind, factor), for yarn (kind, factor, original_context"
                             "[, beta_fast, beta_slow])")
    factor, original, fast, slow = args + (1.0, 0.0, 32.0, 1.0)[len(args):]
    rotary_dim = int(rotary_dim)
    _fits(rotary_dim, "rotary_dim")
    freqs, gain = (C.c_uint64 * max(64, 1))(), C.c_float()
    _check(lib().pa_rope_frequencies(freqs, C.byref(gain), rotary_dim, float(theta), kind, factor, original, fast,
                                     slow), "pa_rope_frequencies")
    host = torch.tensor([f - (1 << 64) if f >> 63 else f for f in freqs[:rotary_dim // 2]], dtype=torch.int64)
    return Rope(host.to(device), gain.value, bool(interleaved))


_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _current_device():
    get = getattr(torch._C, "_cuda_getDevice", None)  # (0.1 us; torch.cuda.current_device takes 0.5)
    return torch.cuda.current_device() if get is None else get()


def _stream_of(dev):
    """The raw current stream of the current device, dev."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream().cuda_stream if raw is None else raw(dev)


def _rope_args(q, k, positions, frequencies, q_norm, k_norm, out_q):
    """Checks what rope and rope_store_kvcache share; returns (tokens, q heads, kv heads, D, strides)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q and k must be [N, heads, 128]")
    n, hq, d = q.shape
    hkv = k.shape[1]
    if n > 0x7fffffff or hq > 0x7fffffff or hkv > 0x7fffffff:
        raise ValueError("number of tokens or heads does not fit 32 bits")
    qs, ks = _rows(q, "q", n, hq, d), _rows(k, "k", n, hkv, d)
    freqs = frequencies.freqs
    if positions.dtype is not _I32 or freqs.dtype is not _I64:
        raise TypeError(f"positions must be {_I32} and frequencies.freqs {_I64}, got {positions.dtype}, {freqs.dtype}")
    if positions.dim() != 1 or positions.shape[0] != n or not positions.is_contiguous():
        raise ValueError("positions must be contiguous [N]")
    if freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("frequencies.freqs must be contiguous [rotary_dim / 2]")
    for w in (q_norm, k_norm):
        if w is not None:
            if w.dtype is not _BF16:
                raise TypeError(f"q_norm and k_norm must be {_BF16}, got {w.dtype}")
            if w.dim() != 1 or w.shape[0] != d or not w.is_contiguous():
                raise ValueError(f"q_norm and k_norm must be contiguous [{d}]")
    return n, hq, hkv, d, qs, ks, hq * d if out_q is None else _rows(out_q, "out_q", n, hq, d)


def rope(q, k, positions, frequencies, q_norm=None, k_norm=None, eps=1e-6, out_q=None, out_k=None, stream=None):
    """Per-head norm (weights q_norm / k_norm, bf16 [128] or None) and rotation of
    q [N, Hq, 128] and k [N, Hkv, 128] (bf16, rows may be strided) at positions
    (int32 [N]), frequencies from rope_frequencies.  Returns (out_q, out_k); out_q may be q itself, out_k may be k."""
    n, hq, hkv, d, qs, ks, oqs = _rope_args(q, k, positions, frequencies, q_norm, k_norm, out_q)
    oks = hkv * d if out_k is None else _rows(out_k, "out_k", n, hkv, d)
    freqs = frequencies.freqs
    ctx = _placed(stream, q, k, positions, freqs, q_norm, k_norm, out_q, out_k)
    if ctx is not None:
        with ctx:
            return rope(q, k, positions, frequencies, q_norm, k_norm, eps, out_q, out_k)
    if out_q is None:
        out_q = torch.empty(n, hq, d, dtype=_BF16, device=q.device)
    if out_k is None:
        out_k = torch.empty(n, hkv, d, dtype=_BF16, device=k.device)
    _check(lib().pa_rope(out_q.data_ptr(), oqs, out_k.data_ptr(), oks, q.data_ptr(), qs, k.data_ptr(), ks,
                         positions.data_ptr(), freqs.data_ptr(), 2 * freqs.shape[0],
                         1 if frequencies.interleaved else 0, frequencies.gain,
                         None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                         eps, n, hq, hkv, d, _stream_of(q.get_device())), "pa_rope")
    return out_q, out_k


def _bf16_pool(k_cache, v_cache):
    """The shape of a bf16 pool [num_blocks, B, Hkv, 128]."""
    shape = k_cache.shape
    if k_cache.dtype is not _BF16 or v_cache.dtype is not _BF16:
        raise TypeError(f"caches must be {_BF16}, got {k_cache.dtype}, {v_cache.dtype}")
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be of one shape, [num_blocks, B, Hkv, 128]")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    return shape


def rope_store_kvcache(q, key, value, positions, frequencies, k_cache, v_cache, slot_mapping, q_norm=None,
                       k_norm=None, eps=1e-6, out_q=None, stream=None):
    """rope of q [N, Hq, 128] and key [N, Hkv, 128], the rotated keys and value
    [N, Hkv, 128] written into the pool [num_blocks, B, Hkv, 128] at slot_mapping
    (int32 [N], negatives skipped).  Returns the rotated q (out_q may be q itself)."""
    n, hq, hkv, d, qs, ks, oqs = _rope_args(q, key, positions, frequencies, q_norm, k_norm, out_q)
    vs = _rows(value, "value", n, hkv, d)
    nb, B, ch, cd = _bf16_pool(k_cache, v_cache)
    if ch != hkv or cd != d:
        raise ValueError(f"caches must be [num_blocks, B, {hkv}, {d}]")
    _slots(slot_mapping, n)
    freqs = frequencies.freqs
    ctx = _placed(stream, q, key, value, positions, freqs, k_cache, v_cache, slot_mapping, q_norm, k_norm, out_q)
    if ctx is not None:
        with ctx:
            return rope_store_kvcache(q, key, value, positions, frequencies, k_cache, v_cache, slot_mapping, q_norm,
                                      k_norm, eps, out_q)
    if out_q is None:
        out_q = torch.empty(n, hq, d, dtype=_BF16, device=q.device)
    _check(lib().pa_rope_store_kvcache(
        out_q.data_ptr(), oqs, q.data_ptr(), qs, key.data_ptr(), ks, value.data_ptr(), vs, positions.data_ptr(),
        freqs.data_ptr(), 2 * freqs.shape[0], 1 if frequencies.interleaved else 0, frequencies.gain,
        None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(), eps,
        k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), n, hq, hkv, d, nb * B,
        _stream_of(q.get_device())), "pa_rope_store_kvcache")
    return out_q


def _int_rows(t, name, shape, dtype=_I32):
    """The address of a contiguous tensor of this shape and type; None stays None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a tensor of {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _tables(block_tables, context_lens, batch):
    """Checks a batch's tables and lengths; returns the tables' width."""
    if block_tables.dtype is not _I32 or context_lens.dtype is not _I32:
        raise TypeError(f"block_tables and context_lens must be {_I32}")
    if block_tables.dim() != 2 or block_tables.shape[0] != batch or context_lens.shape != (batch,):
        raise ValueError("block_tables must be [batch, max_blocks] and context_lens [batch]")
    if not (block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("block_tables and context_lens must be contiguous")
    width = block_tables.shape[1]
    if batch > 0x7fffffff or width > 0x7fffffff:
        raise ValueError("batch or width of block_tables does not fit 32 bits")
    return width


class TreeMetadata(NamedTuple):
    """What tree_metadata returns, node by node."""
    tree_mask: torch.Tensor     # int64 [batch, num_drafts]
    positions: torch.Tensor     # int32 [batch * num_drafts]
    slot_mapping: torch.Tensor  # int32 [batch * num_drafts]


def tree_metadata(parents, context_lens, block_tables, block_size, draft_lens=None, num_drafts=None, stream=None):
    """Masks, rotary positions and slots of a step's trees.  parents int32
    [batch, num_drafts], or None with num_drafts given (chains); context_lens
    int32 [batch] counts all keys, the step's nodes the last of them; draft_lens
    int32 [batch] or None (num_drafts everywhere)."""
    batch = context_lens.shape[0] if isinstance(context_lens, torch.Tensor) and context_lens.dim() == 1 else -1
    width = _tables(block_tables, context_lens, batch)
    if parents is None:
        if num_drafts is None:
            raise ValueError("num_drafts is needed without parents")
        t = int(num_drafts)
    else:
        if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
            raise ValueError("parents must be [batch, num_drafts]")
        t = parents.shape[1]
        if num_drafts is not None and num_drafts != t:
            raise ValueError("num_drafts is not the width of parents")
    _fits(t, "num_drafts")
    _fits(int(block_size), "block size")
    par, lens = _int_rows(parents, "parents", (batch, t)), _int_rows(draft_lens, "draft_lens", (batch,))
    ctx = _placed(stream, context_lens, block_tables, parents, draft_lens)
    if ctx is not None:
        with ctx:
            return tree_metadata(parents, context_lens, block_tables, block_size, draft_lens, t)
    size, dev = max(t, 0), context_lens.device
    out = TreeMetadata(torch.empty(batch, size, dtype=_I64, device=dev),
                       torch.empty(batch * size, dtype=_I32, device=dev),
                       torch.empty(batch * size, dtype=_I32, device=dev))
    _check(lib().pa_tree_metadata(out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), par,
                                  context_lens.data_ptr(), lens, block_tables.data_ptr(), width, batch, t,
                                  int(block_size), _stream_of(context_lens.get_device())), "pa_tree_metadata")
    return out


def decode_tree_workspace(num_q_heads, num_kv_heads, head_dim=128, num_drafts=64, device="cuda"):
    """Workspace for decode_tree (its size depends on the query heads per kv head
    and on num_drafts; a larger one serves smaller calls too).  It holds nothing
    between calls; calls that may run at the same time need one each."""
    n = int(lib().pa_decode_tree_workspace_size(num_q_heads, num_kv_heads, head_dim, num_drafts))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def decode_tree(q, k_cache, v_cache, block_tables, context_lens, tree_mask=None, softmax_scale=None, draft_lens=None,
                workspace=None, out=None, stream=None):
    """Paged attention of the drafted tokens of each sequence.  q [batch,
    num_drafts, Hq, 128] bf16 (tokens may be strided evenly); caches [num_blocks,
    B, Hkv, 128]; context_lens int32 [batch] counts all keys, the drafts the last
    of them (stored before the call); tree_mask int64 [batch, num_drafts]: bit j
    where the draft sees draft j (None: chains); draft_lens int32 [batch] or None.
    Returns out, of q's shape; zeros for padding."""
    nb, B, hkv, d = _bf16_pool(k_cache, v_cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError(f"q must be [batch, num_drafts, Hq, {d}]")
    shape = q.shape
    batch, t, hq, qd = shape
    if q.dtype is not _BF16:
        raise TypeError(f"q must be {_BF16}, got {q.dtype}")
    s0, s1, s2, s3 = q.stride()
    if qd != d or (d > 1 and s3 != 1) or (hq > 1 and s2 != d) or (batch > 1 and t > 1 and s0 != t * s1):
        raise ValueError(f"q must be [batch, num_drafts, Hq, {d}], each token contiguous and all evenly spaced")
    qs = s1 if t > 1 else s0 if batch > 1 else hq * d
    width = _tables(block_tables, context_lens, batch)
    if t > 0x7fffffff or hq > 0x7fffffff:
        raise ValueError("num_drafts or number of q heads does not fit 32 bits")
    mask = _int_rows(tree_mask, "tree_mask", (batch, t), _I64)
    lens = _int_rows(draft_lens, "draft_lens", (batch,))
    if out is not None:
        if out.dtype is not _BF16:
            raise TypeError(f"out must be {_BF16}, got {out.dtype}")
        if out.shape != shape or not out.is_contiguous():
            raise ValueError("out must be contiguous and of q's shape")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
    ctx = _placed(stream, q, k_cache, v_cache, block_tables, context_lens, tree_mask, draft_lens, workspace, out)
    if ctx is not None:
        with ctx:
            return decode_tree(q, k_cache, v_cache, block_tables, context_lens, tree_mask, scale, draft_lens, workspace,
                               out)
    if workspace is None:
        workspace = decode_tree_workspace(hq, hkv, d, t, q.device)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
    _check(lib().pa_decode_tree(out.data_ptr(), q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(),
                                block_tables.data_ptr(), width, context_lens.data_ptr(), lens, mask, batch, t, hq, hkv,
                                d, B, nb, scale, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_of(q.get_device())), "pa_decode_tree")
    return out


class Verified(NamedTuple):
    """What verify_drafts returns; -1 after a row's `counts` entries."""
    tokens: torch.Tensor  # int32 [batch, num_nodes]: the kept tokens, then the next one
    nodes: torch.Tensor   # int32 [batch, num_nodes]: 0 and the kept nodes
    counts: torch.Tensor  # int32 [batch]


def _flat_rows(t, name):
    """Shape of a [batch, rows, vocab] tensor, and elements between its rows, evenly spaced."""
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions")
    b, r, v = t.shape
    s0, s1, s2 = t.stride()
    if (v > 1 and s2 != 1) or (b > 1 and r > 1 and s0 != r * s1):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
    return b, r, v, s1 if r > 1 else s0 if b > 1 else -(-v // 8) * 8


def verify_drafts(logits, tokens, parents, uniforms, exp_noise, temperatures, draft_probs=None, draft_lens=None,
                  out=None, stream=None):
    """Speculative sampling: which drafted tokens the target keeps, and the next
    token.  logits [batch, num_nodes, vocab] bf16 or fp32 (rows may be strided
    evenly), the target's at every node; tokens / parents int32 [batch,
    num_nodes] (parents None: chains); uniforms fp32 [batch, num_nodes] in [0, 1);
    exp_noise fp32 [batch, vocab] of Exp(1) draws; temperatures fp32 [batch];
    draft_probs fp32 [batch, at least num_nodes - 1, vocab], the distributions
    that the nodes' children were drawn from, or None (chosen candidates);
    draft_lens int32 [batch], nodes of each tree, or None.  `out`, a Verified of
    contiguous tensors, is filled and returned."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (_BF16, _F32):
        raise TypeError("logits must be a bfloat16 or float32 tensor")
    batch, n, vocab, ls = _flat_rows(logits, "logits")
    if batch > 0x7fffffff or n > 0x7fffffff or vocab > 0x7fffffff:
        raise ValueError("batch, number of nodes or vocabulary does not fit 32 bits")
    rows = (batch, n)
    tok, par = _int_rows(tokens, "tokens", rows), _int_rows(parents, "parents", rows)
    uni, temp = _int_rows(uniforms, "uniforms", rows, _F32), _int_rows(temperatures, "temperatures", (batch,), _F32)
    lens = _int_rows(draft_lens, "draft_lens", (batch,))
    if exp_noise.dtype is not _F32:
        raise TypeError(f"exp_noise must be {_F32}, got {exp_noise.dtype}")
    if exp_noise.shape != (batch, vocab) or (vocab > 1 and exp_noise.stride(1) != 1):
        raise ValueError("exp_noise must be [batch, vocab] with contiguous rows")
    es = exp_noise.stride(0) if batch > 1 else -(-vocab // 4) * 4
    probs, ps, pr = None, 0, 0
    if draft_probs is not None:
        if draft_probs.dtype is not _F32:
            raise TypeError(f"draft_probs must be {_F32}, got {draft_probs.dtype}")
        pb, pr, pv, ps = _flat_rows(draft_probs, "draft_probs")
        if pb != batch or pv != vocab or not n - 1 <= pr <= 0x7fffffff:
            raise ValueError("draft_probs must be [batch, at least num_nodes - 1, vocab]")
        probs = draft_probs.data_ptr()
    if out is not None:
        for t, shape, name in ((out[0], rows, "tokens"), (out[1], rows, "nodes"), (out[2], (batch,), "counts")):
            if _int_rows(t, f"out.{name}", shape) is None:
                raise TypeError(f"out.{name} must be a CUDA tensor")
    ctx = _placed(stream, logits, tokens, parents, uniforms, exp_noise, temperatures, draft_probs, draft_lens,
                  *(out or ()))
    if ctx is not None:
        with ctx:
            return verify_drafts(logits, tokens, parents, uniforms, exp_noise, temperatures, draft_probs, draft_lens,
                                 out)
    if out is None:
        out = Verified(torch.empty_like(tokens), torch.empty_like(tokens),
                       torch.empty(batch, dtype=_I32, device=tokens.device))
    _check(lib().pa_verify_drafts(out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), logits.data_ptr(), ls,
                                  1 if logits.dtype is _F32 else 0, tok, par, uni, exp_noise.data_ptr(), es, temp,
                                  probs, ps, pr, lens, batch, n, vocab, _stream_of(logits.get_device())),
           "pa_verify_drafts")
    return out


def compact_kvcache(k_cache, v_cache, block_tables, context_lens, nodes, counts, draft_lens=None, stream=None):
    """Move the kept nodes' K and V rows next to the context: position base +
    nodes[b, j] to base + j for j < counts[b], base = context_lens[b] minus the
    tree's size (draft_lens, or nodes' width).  Caches [num_blocks, B, Hkv, 128], or
    [layers, num_blocks, B, Hkv, 128] for all layers in one call (each layer
    contiguous); nodes int32 [batch, num_nodes] and counts int32 [batch] as
    verify_drafts returns them."""
    layers, ks, vs = 1, 0, 0
    if k_cache.dim() == 5 and v_cache.dim() == 5:
        layers, nb, B, hkv, d = shape = k_cache.shape
        if k_cache.dtype is not _BF16 or v_cache.dtype is not _BF16:
            raise TypeError(f"caches must be {_BF16}, got {k_cache.dtype}, {v_cache.dtype}")
        if v_cache.shape != shape or layers > 0x7fffffff:
            raise ValueError("k_cache and v_cache must be of one shape, [layers, num_blocks, B, Hkv, 128]")
        if not (k_cache.is_contiguous() and v_cache.is_contiguous()):  # then each layer has to be
            for t in (k_cache, v_cache):
                if layers > 0 and not t[0].is_contiguous():
                    raise ValueError("each layer must be contiguous")
        ks, vs = k_cache.stride(0), v_cache.stride(0)
        if layers > 1 and min(ks, vs) < nb * B * hkv * d:
            raise ValueError("layers overlap")
    else:
        nb, B, hkv, d = _bf16_pool(k_cache, v_cache)
    if not isinstance(nodes, torch.Tensor) or nodes.dim() != 2:
        raise ValueError("nodes must be [batch, num_nodes]")
    batch, n = nodes.shape
    width = _tables(block_tables, context_lens, batch)
    if n > 0x7fffffff:
        raise ValueError("number of nodes does not fit 32 bits")
    lens, node_ptr = _int_rows(draft_lens, "draft_lens", (batch,)), _int_rows(nodes, "nodes", (batch, n))
    count_ptr = _int_rows(counts, "counts", (batch,))
    ctx = _placed(stream, k_cache, v_cache, block_tables, context_lens, nodes, counts, draft_lens)
    if ctx is not None:
        with ctx:
            return compact_kvcache(k_cache, v_cache, block_tables, context_lens, nodes, counts, draft_lens)
    _check(lib().pa_compact_kvcache(k_cache.data_ptr(), ks, v_cache.data_ptr(), vs, block_tables.data_ptr(), width,
                                    context_lens.data_ptr(), lens, node_ptr, count_ptr, batch, n, layers, hkv, d, B, nb,
                                    _stream_of(k_cache.get_device())), "pa_compact_kvcache")


def set_checked(enabled: bool):
    _check(lib().pa_set_checked(1 if enabled else 0), "pa_set_checked")


def get_device_error(stream=None):
    """Synchronise the stream; return (code, where) of the first device-side
    error since the last call ((0, 0) if none) and clear it."""
    code, where = _i32(0), _i64(0)
    st = lib().pa_get_device_error(_stream(stream), C.byref(code), C.byref(where))
    if st not in (PA_OK, PA_ERR_DEVICE_CHECK):
        _check(st, "pa_get_device_error")
    return int(code.value), int(where.value)
