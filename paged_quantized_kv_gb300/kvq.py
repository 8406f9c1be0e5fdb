"""Thin Python binding of libkvq (ctypes).

Argument marshalling only: torch tensors supply device pointers, sizes and
strides, and ``torch.cuda.current_stream()`` supplies the stream; every step
of the computation runs in the CUDA kernels behind ``include/kvq.h``.  If
``libkvq.so`` is missing or cannot be loaded the calls raise -- there is no
fallback path.

The operations keep the argument order of the pages' ops where there is
one:

* ``kvq_store_nvfp4(key, value, key_cache, value_cache, slot_mapping,
  k_scale, v_scale)`` -- vLLM ``reshape_and_cache_nvfp4_dispatch``
  (nvfp4_kv_cache_kernels.cu, commit 7ce4c8e): ``key_cache`` /
  ``value_cache`` are ``kv_cache[:, 0]`` / ``kv_cache[:, 1]`` in the logical
  order [num_blocks, block_size, num_heads, head_size/2 + head_size/16],
  their strides telling HND from NHD.
* ``kvq_gather_indexer_k(kv_cache, k_fp8, k_scale, block_table,
  cu_seq_lens)`` -- vLLM ``cp_gather_indexer_k_quant_cache`` (PR #25931,
  PR #26456).
* ``kvq_load_nvfp4(key_cache, value_cache, block_table, cu_seq_lens,
  k_scale, v_scale, key_out, value_out)`` -- the read side of the store.
* ``kvq_store_indexer_k(k, kv_cache, slot_mapping)`` -- the write side of
  the indexer cache the gather reads.

Additions of this library (no counterpart in the pages):

* ``kvq_chunk_attention_nvfp4`` -- causal attention of chunks of new tokens
  over the NVFP4 pages.
* ``kvq_tree_attention_nvfp4`` -- the same for trees of drafted tokens.
* ``kvq_quantize_indexer_q``, ``kvq_score_blocks_indexer_k``,
  ``kvq_select_blocks``, ``kvq_sparse_attention_nvfp4`` -- attention over
  blocks of the context that an indexer selects for each query.
* ``kvq_extend_sequences``, ``kvq_fork_sequences``,
  ``kvq_compact_sequences``, ``kvq_free_sequences`` -- the state of a paged
  cache (``alloc_page_pool``) on the device.
* ``kvq_copy_pages``, ``kvq_move_tokens_nvfp4`` -- the bytes that go with
  them.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK = 0
KVQ_ERR_NULL = -1
KVQ_ERR_SHAPE = -2
KVQ_ERR_ALIGN = -3
KVQ_ERR_DTYPE = -4
KVQ_ERR_LAYOUT = -5
KVQ_ERR_CUDA = -6
KVQ_ERR_ARG = -7
KVQ_ERR_SCRATCH = -8
KVQ_NOALLOC_SCRATCH_BYTES = 32 << 20

KVQ_LAYOUT_HND = 0
KVQ_LAYOUT_NHD = 1
KVQ_DTYPE_BF16 = 0
KVQ_DTYPE_FP16 = 1
KVQ_F_SWIZZLE_K_SCALE = 1
KVQ_F_PDL = 2
KVQ_F_PDL_EARLY_META = 4
KVQ_F_PDL_EARLY_READ = 1 << 4
KVQ_DEVERR_SLOT = 1
KVQ_DEVERR_BLOCK = 2
KVQ_DEVERR_SEQ = 4
KVQ_DEVERR_TIMEOUT = 8
KVQ_DEVERR_REF = 16
KVQ_DEVERR_FULL = 32

_HALF_TYPES = {torch.bfloat16: KVQ_DTYPE_BF16,
               torch.float16: KVQ_DTYPE_FP16}

_lock = threading.Lock()
_lib = None


class KvqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {kvq_status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libkvq.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m paged_quantized_kv_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        c = ctypes
        P = c.c_void_p
        L.kvq_store_nvfp4.argtypes = [
            P, c.c_int64, P, c.c_int64, c.c_int32, c.c_int32, c.c_int32,
            c.c_int32, P, P, c.c_int64, c.c_int32, c.c_int64, c.c_int32, P,
            P, P, c.c_uint32, P, P]
        L.kvq_store_nvfp4.restype = c.c_int
        L.kvq_gather_indexer_k.argtypes = [
            P, c.c_int64, c.c_int64, c.c_int32, c.c_int32, P, c.c_int64,
            c.c_int32, P, c.c_int32, c.c_int64, P, P, c.c_uint32, P, P]
        L.kvq_gather_indexer_k.restype = c.c_int
        L.kvq_load_nvfp4.argtypes = [
            P, P, c.c_int64, c.c_int32, c.c_int64, c.c_int32, c.c_int32,
            c.c_int32, P, c.c_int64, c.c_int32, P, c.c_int32, c.c_int64, P,
            P, c.c_int32, P, P, c.c_int64, c.c_uint32, P, P]
        L.kvq_load_nvfp4.restype = c.c_int
        L.kvq_store_indexer_k.argtypes = [
            P, c.c_int64, c.c_int32, c.c_int32, c.c_int32, P, c.c_int64,
            c.c_int32, c.c_int64, P, c.c_uint32, P, P]
        L.kvq_store_indexer_k.restype = c.c_int
        L.kvq_paged_attention_nvfp4.argtypes = [
            P, c.c_int64, c.c_int32, c.c_int32, c.c_int32, c.c_int32,
            c.c_int32, P, P, c.c_int64, c.c_int32, c.c_int64, c.c_int32, P,
            c.c_int64, c.c_int32, P, c.c_int32, P, P, c.c_float, c.c_int32,
            P, P, P, P, c.c_int64, c.c_uint32, P, P]
        L.kvq_paged_attention_nvfp4.restype = c.c_int
        L.kvq_paged_attention_nvfp4_noalloc.argtypes = [
            P, c.c_int64, c.c_int32, c.c_int32, c.c_int32, c.c_int32,
            c.c_int32, P, P, c.c_int64, c.c_int32, c.c_int64, c.c_int32, P,
            c.c_int64, c.c_int32, P, c.c_int32, P, P, c.c_float, c.c_int32,
            P, c.c_int64, c.c_uint32, P, P]
        L.kvq_paged_attention_nvfp4_noalloc.restype = c.c_int
        L.kvq_chunk_attention_nvfp4.argtypes = [
            P, c.c_int64, c.c_int32, c.c_int64, c.c_int32, P, c.c_int32,
            c.c_int32, c.c_int32, c.c_int32, P, P, c.c_int64, c.c_int32,
            c.c_int64, c.c_int32, P, c.c_int64, c.c_int32, P, c.c_int32, P,
            P, c.c_float, P, c.c_int64, P, c.c_int64, c.c_uint32, P, P]
        L.kvq_chunk_attention_nvfp4.restype = c.c_int
        L.kvq_chunk_attention_workspace_bytes.argtypes = []
        L.kvq_chunk_attention_workspace_bytes.restype = c.c_int64
        attention = L.kvq_chunk_attention_nvfp4.argtypes
        L.kvq_tree_attention_nvfp4.argtypes = attention[:21] + [
            P, c.c_int64, c.c_int32] + attention[21:]
        L.kvq_tree_attention_nvfp4.restype = c.c_int
        L.kvq_sparse_attention_nvfp4.argtypes = attention[:21] + [
            P, c.c_int64, c.c_int32, c.c_int32] + attention[21:]
        L.kvq_sparse_attention_nvfp4.restype = c.c_int
        L.kvq_sparse_attention_workspace_bytes.argtypes = [
            c.c_int64] + [c.c_int32] * 7
        L.kvq_sparse_attention_workspace_bytes.restype = c.c_int64
        L.kvq_quantize_indexer_q.argtypes = [
            P, c.c_int64, c.c_int32, P, c.c_int64, c.c_float, c.c_int64,
            c.c_int32, c.c_int32, P, P, c.c_uint32, P]
        L.kvq_quantize_indexer_q.restype = c.c_int
        L.kvq_score_blocks_indexer_k.argtypes = [
            P, c.c_int64, P, c.c_int64, c.c_int64, c.c_int32, P, c.c_int32,
            c.c_int32, c.c_int32, P, c.c_int64, c.c_int64, c.c_int32, P,
            c.c_int64, c.c_int32, P, c.c_int32, P, c.c_int64, c.c_int32,
            c.c_uint32, P, P]
        L.kvq_score_blocks_indexer_k.restype = c.c_int
        L.kvq_select_blocks.argtypes = [
            P, c.c_int64, c.c_int32, c.c_int64, c.c_int32, P, P, c.c_int32,
            c.c_int32, c.c_int32, P, c.c_int64, c.c_int32, c.c_uint32, P, P]
        L.kvq_select_blocks.restype = c.c_int
        pool = [P, c.c_int64, P, c.c_int64, c.c_int32, c.c_int32, P]
        L.kvq_extend_sequences.argtypes = pool + [
            c.c_int32, P, P, c.c_int32, P, c.c_int64, c.c_uint32, P, P]
        L.kvq_extend_sequences.restype = c.c_int
        L.kvq_fork_sequences.argtypes = pool + [
            c.c_int32, P, P, c.c_int32, P, P, c.c_uint32, P, P]
        L.kvq_fork_sequences.restype = c.c_int
        L.kvq_compact_sequences.argtypes = pool + [
            c.c_int32, P, P, P, c.c_int32, P, P, c.c_int64, c.c_uint32, P,
            P]
        L.kvq_compact_sequences.restype = c.c_int
        L.kvq_free_sequences.argtypes = pool + [
            P, c.c_int32, c.c_uint32, P, P]
        L.kvq_free_sequences.restype = c.c_int
        L.kvq_copy_pages.argtypes = [
            P, c.c_int32, c.c_int64, c.c_int64, c.c_int64, P, P, c.c_int32,
            c.c_uint32, P, P]
        L.kvq_copy_pages.restype = c.c_int
        L.kvq_move_tokens_nvfp4.argtypes = [
            P, c.c_int32, c.c_int64, c.c_int64, c.c_int64, c.c_int32,
            c.c_int32, c.c_int32, c.c_int32, P, P, c.c_int64, P, c.c_int32,
            c.c_uint32, P, P]
        L.kvq_move_tokens_nvfp4.restype = c.c_int
        L.kvq_status_string.argtypes = [c.c_int]
        L.kvq_status_string.restype = c.c_char_p
        L.kvq_version.argtypes = []
        L.kvq_version.restype = c.c_int32
        _lib = L
        return L


def kvq_status_string(status: int) -> str:
    return lib().kvq_status_string(int(status)).decode()


def kvq_version() -> int:
    return int(lib().kvq_version())


def _stream_of(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _check(fn: str, status: int) -> None:
    if status != KVQ_OK:
        raise KvqError(fn, status)


def kvq_store_nvfp4(key: torch.Tensor, value: torch.Tensor,
                    key_cache: torch.Tensor, value_cache: torch.Tensor,
                    slot_mapping: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, flags: int = 0,
                    dev_error: torch.Tensor | None = None,
                    stream: int | None = None) -> None:
    """NVFP4 paged store (see ``include/kvq.h``).

    key, value: bf16 or fp16 [T, H, D], last two dims contiguous.  key_cache,
    value_cache: uint8 [num_blocks, block_size, H, D/2 + D/16] views whose
    stride(0) is the page stride and whose stride(2) > stride(1) marks HND.
    slot_mapping: int64 [T].  k_scale, v_scale: fp32 device scalars."""
    dtypes = {torch.bfloat16: KVQ_DTYPE_BF16, torch.float16: KVQ_DTYPE_FP16}
    if key.dtype not in dtypes or value.dtype != key.dtype:
        raise KvqError("kvq_store_nvfp4", KVQ_ERR_DTYPE)
    T, H, D = key.shape
    if (key.stride(2) != 1 or key.stride(1) != D or value.stride(2) != 1
            or value.stride(1) != D or tuple(value.shape) != (T, H, D)):
        raise KvqError("kvq_store_nvfp4", KVQ_ERR_SHAPE)
    if key_cache.dim() != 4 or key_cache.dtype != torch.uint8:
        raise KvqError("kvq_store_nvfp4", KVQ_ERR_SHAPE)
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() < T:
        raise KvqError("kvq_store_nvfp4", KVQ_ERR_SHAPE)
    layout = (KVQ_LAYOUT_HND if key_cache.stride(2) > key_cache.stride(1)
              else KVQ_LAYOUT_NHD)
    st = lib().kvq_store_nvfp4(
        key.data_ptr(), key.stride(0), value.data_ptr(), value.stride(0),
        dtypes[key.dtype], T, H, D, key_cache.data_ptr(),
        value_cache.data_ptr(), key_cache.stride(0), key_cache.size(1),
        key_cache.size(0), layout, slot_mapping.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), int(flags),
        _ptr(dev_error), _stream_of(key) if stream is None else stream)
    _check("kvq_store_nvfp4", st)


def kvq_gather_indexer_k(kv_cache: torch.Tensor, k_fp8: torch.Tensor,
                         k_scale: torch.Tensor, block_table: torch.Tensor,
                         cu_seq_lens: torch.Tensor, block_size: int | None = None,
                         flags: int = 0,
                         dev_error: torch.Tensor | None = None,
                         stream: int | None = None) -> None:
    """Indexer-K gather (see ``include/kvq.h``).

    kv_cache: uint8 [num_blocks, block_size, head_dim + 4] (or
    [num_blocks, bytes] with ``block_size`` given); each block holds
    [block_size*head_dim K bytes | block_size*4 scale bytes].
    k_fp8: [total, head_dim] 1-byte elements; k_scale: [total, 4] uint8 (or
    [total] float32).  block_table int32 [num_seqs, max_blocks];
    cu_seq_lens int32 [num_seqs + 1]; total = k_fp8.size(0)."""
    if kv_cache.element_size() != 1 or k_fp8.element_size() != 1:
        raise KvqError("kvq_gather_indexer_k", KVQ_ERR_DTYPE)
    if block_table.dtype != torch.int32 or cu_seq_lens.dtype != torch.int32:
        raise KvqError("kvq_gather_indexer_k", KVQ_ERR_DTYPE)
    total, head_dim = k_fp8.shape
    if block_size is None:
        if kv_cache.dim() != 3:
            raise KvqError("kvq_gather_indexer_k", KVQ_ERR_SHAPE)
        block_size = kv_cache.size(1)
    if (k_fp8.stride(0) != head_dim or k_fp8.stride(1) != 1
            or k_scale.numel() * k_scale.element_size() < 4 * total
            or not k_scale.is_contiguous() or block_table.stride(1) != 1):
        raise KvqError("kvq_gather_indexer_k", KVQ_ERR_SHAPE)
    st = lib().kvq_gather_indexer_k(
        kv_cache.data_ptr(), kv_cache.stride(0), kv_cache.size(0),
        int(block_size), int(head_dim), block_table.data_ptr(),
        block_table.stride(0), block_table.size(1), cu_seq_lens.data_ptr(),
        cu_seq_lens.numel() - 1, int(total), k_fp8.data_ptr(),
        k_scale.data_ptr(), int(flags), _ptr(dev_error),
        _stream_of(kv_cache) if stream is None else stream)
    _check("kvq_gather_indexer_k", st)


def kvq_load_nvfp4(key_cache: torch.Tensor, value_cache: torch.Tensor,
                   block_table: torch.Tensor, cu_seq_lens: torch.Tensor,
                   k_scale: torch.Tensor, v_scale: torch.Tensor,
                   key_out: torch.Tensor, value_out: torch.Tensor,
                   flags: int = 0, dev_error: torch.Tensor | None = None,
                   stream: int | None = None) -> None:
    """NVFP4 paged load (see ``include/kvq.h``): the tokens the block table
    names, dequantised into key_out / value_out (bf16 [total, H, D], last two
    dims contiguous; total = key_out.size(0)).  key_cache / value_cache are
    the store's 4-D page views."""
    if key_out.dtype != torch.bfloat16 or value_out.dtype != torch.bfloat16:
        raise KvqError("kvq_load_nvfp4", KVQ_ERR_DTYPE)
    T, H, D = key_out.shape
    if (key_out.stride(2) != 1 or key_out.stride(1) != D
            or tuple(value_out.shape) != (T, H, D)
            or value_out.stride(0) != key_out.stride(0)
            or value_out.stride(2) != 1 or value_out.stride(1) != D):
        raise KvqError("kvq_load_nvfp4", KVQ_ERR_SHAPE)
    if key_cache.dim() != 4 or key_cache.dtype != torch.uint8:
        raise KvqError("kvq_load_nvfp4", KVQ_ERR_SHAPE)
    if block_table.dtype != torch.int32 or cu_seq_lens.dtype != torch.int32:
        raise KvqError("kvq_load_nvfp4", KVQ_ERR_DTYPE)
    layout = (KVQ_LAYOUT_HND if key_cache.stride(2) > key_cache.stride(1)
              else KVQ_LAYOUT_NHD)
    st = lib().kvq_load_nvfp4(
        key_cache.data_ptr(), value_cache.data_ptr(), key_cache.stride(0),
        key_cache.size(1), key_cache.size(0), layout, H, D,
        block_table.data_ptr(), block_table.stride(0), block_table.size(1),
        cu_seq_lens.data_ptr(), cu_seq_lens.numel() - 1, T,
        k_scale.data_ptr(), v_scale.data_ptr(), KVQ_DTYPE_BF16,
        key_out.data_ptr(), value_out.data_ptr(), key_out.stride(0),
        int(flags), _ptr(dev_error),
        _stream_of(key_out) if stream is None else stream)
    _check("kvq_load_nvfp4", st)


def kvq_store_indexer_k(k: torch.Tensor, kv_cache: torch.Tensor,
                        slot_mapping: torch.Tensor,
                        block_size: int | None = None, flags: int = 0,
                        dev_error: torch.Tensor | None = None,
                        stream: int | None = None) -> None:
    """Indexer-K store (see ``include/kvq.h``): k bf16/fp16 [T, head_dim]
    (last dim contiguous) into kv_cache uint8 [num_blocks, block_size,
    head_dim + 4] (or [num_blocks, bytes] with ``block_size`` given)."""
    dtypes = {torch.bfloat16: KVQ_DTYPE_BF16, torch.float16: KVQ_DTYPE_FP16}
    if k.dtype not in dtypes or kv_cache.element_size() != 1:
        raise KvqError("kvq_store_indexer_k", KVQ_ERR_DTYPE)
    T, D = k.shape
    if block_size is None:
        if kv_cache.dim() != 3:
            raise KvqError("kvq_store_indexer_k", KVQ_ERR_SHAPE)
        block_size = kv_cache.size(1)
    if (k.stride(1) != 1 or slot_mapping.dtype != torch.int64
            or slot_mapping.numel() < T):
        raise KvqError("kvq_store_indexer_k", KVQ_ERR_SHAPE)
    st = lib().kvq_store_indexer_k(
        k.data_ptr(), k.stride(0), dtypes[k.dtype], T, D,
        kv_cache.data_ptr(), kv_cache.stride(0), int(block_size),
        kv_cache.size(0), slot_mapping.data_ptr(), int(flags),
        _ptr(dev_error), _stream_of(k) if stream is None else stream)
    _check("kvq_store_indexer_k", st)


def attention_scratch(num_seqs: int, num_q_heads: int, max_context_len: int,
                      partition_size: int = 512, head_size: int = 128,
                      device="cuda"):
    """(exp_sums, max_logits, tmp_out) fp32 scratch for
    kvq_paged_attention_nvfp4, or (None, None, None) when every context fits
    one partition."""
    parts = -(-int(max_context_len) // int(partition_size))
    if parts <= 1:
        return None, None, None
    shape = (num_seqs, num_q_heads, parts)
    return (torch.empty(shape, dtype=torch.float32, device=device),
            torch.empty(shape, dtype=torch.float32, device=device),
            torch.empty(shape + (head_size,), dtype=torch.float32,
                        device=device))


def kvq_paged_attention_nvfp4(query: torch.Tensor, key_cache: torch.Tensor,
                              value_cache: torch.Tensor,
                              block_table: torch.Tensor,
                              context_lens: torch.Tensor,
                              k_scale: torch.Tensor, v_scale: torch.Tensor,
                              scale: float, out: torch.Tensor,
                              max_context_len: int,
                              partition_size: int = 512,
                              exp_sums: torch.Tensor | None = None,
                              max_logits: torch.Tensor | None = None,
                              tmp_out: torch.Tensor | None = None,
                              flags: int = 0,
                              dev_error: torch.Tensor | None = None,
                              stream: int | None = None) -> None:
    """Paged decode attention over the NVFP4 cache (see ``include/kvq.h``).

    query / out: bf16 or fp16 [num_seqs, Hq, 128] (last two dims
    contiguous); key_cache / value_cache: the store's 4-D page views;
    block_table int32 [num_seqs, max_blocks]; context_lens int32
    [num_seqs].  The fp32 scratch (``attention_scratch``) is allocated here
    when it is needed and not given."""
    dtypes = {torch.bfloat16: KVQ_DTYPE_BF16, torch.float16: KVQ_DTYPE_FP16}
    if query.dtype not in dtypes or out.dtype != query.dtype:
        raise KvqError("kvq_paged_attention_nvfp4", KVQ_ERR_DTYPE)
    n, Hq, D = query.shape
    if (query.stride(2) != 1 or query.stride(1) != D or out.stride(2) != 1
            or out.stride(1) != D or tuple(out.shape) != (n, Hq, D)):
        raise KvqError("kvq_paged_attention_nvfp4", KVQ_ERR_SHAPE)
    if key_cache.dim() != 4 or key_cache.dtype != torch.uint8:
        raise KvqError("kvq_paged_attention_nvfp4", KVQ_ERR_SHAPE)
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise KvqError("kvq_paged_attention_nvfp4", KVQ_ERR_DTYPE)
    layout = (KVQ_LAYOUT_HND if key_cache.stride(2) > key_cache.stride(1)
              else KVQ_LAYOUT_NHD)
    if exp_sums is None and max_logits is None and tmp_out is None:
        exp_sums, max_logits, tmp_out = attention_scratch(
            n, Hq, max_context_len, partition_size, D, query.device)
    st = lib().kvq_paged_attention_nvfp4(
        query.data_ptr(), query.stride(0), dtypes[query.dtype], n, Hq,
        key_cache.size(2), D, key_cache.data_ptr(), value_cache.data_ptr(),
        key_cache.stride(0), key_cache.size(1), key_cache.size(0), layout,
        block_table.data_ptr(), block_table.stride(0), block_table.size(1),
        context_lens.data_ptr(), int(max_context_len), k_scale.data_ptr(),
        v_scale.data_ptr(), float(scale), int(partition_size),
        _ptr(exp_sums), _ptr(max_logits), _ptr(tmp_out), out.data_ptr(),
        out.stride(0), int(flags), _ptr(dev_error),
        _stream_of(query) if stream is None else stream)
    _check("kvq_paged_attention_nvfp4", st)


def kvq_paged_attention_nvfp4_noalloc(query: torch.Tensor,
                                      key_cache: torch.Tensor,
                                      value_cache: torch.Tensor,
                                      block_table: torch.Tensor,
                                      context_lens: torch.Tensor,
                                      k_scale: torch.Tensor,
                                      v_scale: torch.Tensor, scale: float,
                                      out: torch.Tensor, max_context_len: int,
                                      partition_size: int = 512,
                                      flags: int = 0,
                                      dev_error: torch.Tensor | None = None,
                                      stream: int | None = None) -> None:
    """kvq_paged_attention_nvfp4 for callers that cannot allocate device
    memory (see ``include/kvq.h``): the same arguments without the scratch
    tensors; the library's built-in scratch array is used instead, and
    nothing is allocated here either."""
    dtypes = {torch.bfloat16: KVQ_DTYPE_BF16, torch.float16: KVQ_DTYPE_FP16}
    if query.dtype not in dtypes or out.dtype != query.dtype:
        raise KvqError("kvq_paged_attention_nvfp4_noalloc", KVQ_ERR_DTYPE)
    n, Hq, D = query.shape
    if (query.stride(2) != 1 or query.stride(1) != D or out.stride(2) != 1
            or out.stride(1) != D or tuple(out.shape) != (n, Hq, D)):
        raise KvqError("kvq_paged_attention_nvfp4_noalloc", KVQ_ERR_SHAPE)
    if key_cache.dim() != 4 or key_cache.dtype != torch.uint8:
        raise KvqError("kvq_paged_attention_nvfp4_noalloc", KVQ_ERR_SHAPE)
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise KvqError("kvq_paged_attention_nvfp4_noalloc", KVQ_ERR_DTYPE)
    layout = (KVQ_LAYOUT_HND if key_cache.stride(2) > key_cache.stride(1)
              else KVQ_LAYOUT_NHD)
    st = lib().kvq_paged_attention_nvfp4_noalloc(
        query.data_ptr(), query.stride(0), dtypes[query.dtype], n, Hq,
        key_cache.size(2), D, key_cache.data_ptr(), value_cache.data_ptr(),
        key_cache.stride(0), key_cache.size(1), key_cache.size(0), layout,
        block_table.data_ptr(), block_table.stride(0), block_table.size(1),
        context_lens.data_ptr(), int(max_context_len), k_scale.data_ptr(),
        v_scale.data_ptr(), float(scale), int(partition_size),
        out.data_ptr(), out.stride(0), int(flags), _ptr(dev_error),
        _stream_of(query) if stream is None else stream)
    _check("kvq_paged_attention_nvfp4_noalloc", st)


def _here(fn: str, *tensors) -> int:
    """The current device's stream, once every tensor given is on that
    device, else KVQ_ERR_ARG: a host or foreign pointer must not reach a
    kernel.  (Raw calls: these checks are most of a small call's time.)"""
    here = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1
    for t in tensors:
        if t is not None and (here < 0 or t.get_device() != here):
            raise KvqError(fn, KVQ_ERR_ARG)
    return torch._C._cuda_getCurrentRawStream(here)


def _vector(fn: str, dtype: torch.dtype, *tensors) -> None:
    for t in tensors:
        if t.dtype is not dtype:
            raise KvqError(fn, KVQ_ERR_DTYPE)
        if t.dim() != 1 or (t.stride(0) != 1 and t.numel() > 1):
            raise KvqError(fn, KVQ_ERR_SHAPE)


def _dev_error_ok(fn: str, t) -> None:
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1):
        raise KvqError(fn, KVQ_ERR_DTYPE)


def _page_views(fn: str, key_cache, value_cache) -> int:
    """Checks the store's 4-D page views; returns their layout."""
    if (key_cache.dtype is not torch.uint8
            or value_cache.dtype is not torch.uint8):
        raise KvqError(fn, KVQ_ERR_DTYPE)
    shape, strides = key_cache.shape, key_cache.stride()
    if (len(shape) != 4 or strides[3] != 1 or value_cache.shape != shape
            or value_cache.stride() != strides):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    _, B, H, full = shape
    _, sb, sh, _ = strides
    if sb == full and (sh == B * full or H == 1):
        return KVQ_LAYOUT_HND  # (with one head both layouts are the same)
    if sh == full and sb == H * full:
        return KVQ_LAYOUT_NHD
    raise KvqError(fn, KVQ_ERR_SHAPE)


def chunk_attention_workspace(device="cuda") -> torch.Tensor:
    """Workspace of kvq_chunk_attention_nvfp4 (the same for every call on a
    device; calls that may overlap each need their own)."""
    with torch.cuda.device(device):
        n = lib().kvq_chunk_attention_workspace_bytes()
    return torch.empty(n, dtype=torch.uint8, device=device)


def _rows_of(fn: str, t: torch.Tensor, dtype: torch.dtype, total: int):
    """(row stride, width) of a matrix [total, width] with contiguous rows."""
    if t.dtype is not dtype:
        raise KvqError(fn, KVQ_ERR_DTYPE)
    shape = t.shape
    if len(shape) != 2 or shape[0] != total:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    stride, step = t.stride()
    if shape[1] > 1 and step != 1 and total > 0:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    return stride if total > 1 else shape[1], shape[1]


def _record(t: torch.Tensor, here: int, stream: int | None) -> None:
    """Memory allocated here is not handed out again before `stream` is past
    it."""
    if stream is not None and stream != here:
        t.record_stream(torch.cuda.ExternalStream(
            stream, device=t.device) if stream else
            torch.cuda.default_stream(t.device))


def _attend(fn: str, query, key_cache, value_cache, block_table, cu_q_lens,
            context_lens, tensors, extra, k_scale, v_scale, scale, out,
            max_q_len, workspace, make_workspace, max_context_len, flags,
            dev_error, stream) -> None:
    """What the attentions of many query tokens per sequence share: checks
    and the call, with the arguments `extra` (of `tensors`) behind the
    contexts'."""
    # (shapes and strides are asked for once: a call of torch for each would
    # be most of a small call's time)
    dtype = _HALF_TYPES.get(query.dtype)
    if dtype is None or out.dtype is not query.dtype:
        raise KvqError(fn, KVQ_ERR_DTYPE)
    shape, strides, out_strides = query.shape, query.stride(), out.stride()
    if len(shape) != 3 or out.shape != shape:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    total, Hq, D = shape
    if (strides[2] != 1 or strides[1] != D or out_strides[2] != 1
            or out_strides[1] != D):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    layout = _page_views(fn, key_cache, value_cache)
    blocks, B, Hkv, full = key_cache.shape
    _vector(fn, torch.int32, cu_q_lens, context_lens)
    n = context_lens.numel()
    if block_table.dtype is not torch.int32:
        raise KvqError(fn, KVQ_ERR_DTYPE)
    table, table_strides = block_table.shape, block_table.stride()
    if (cu_q_lens.numel() != n + 1 or len(table) != 2 or table[0] < n
            or (table[1] > 1 and table[0] > 0 and table_strides[1] != 1)
            or full != D // 2 + D // 16):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    if (k_scale.dtype is not torch.float32
            or v_scale.dtype is not torch.float32):
        raise KvqError(fn, KVQ_ERR_DTYPE)
    _dev_error_ok(fn, dev_error)
    here = _here(fn, query, out, key_cache, value_cache, block_table,
                 cu_q_lens, context_lens, k_scale, v_scale, workspace,
                 dev_error, *tensors)
    if workspace is None:
        workspace = (make_workspace() if make_workspace is not None
                     else chunk_attention_workspace(query.device))
        _record(workspace, here, stream)
    if not workspace.is_contiguous():
        raise KvqError(fn, KVQ_ERR_SHAPE)
    st = getattr(lib(), fn)(
        query.data_ptr(), strides[0] if total > 1 else Hq * D, dtype, total,
        n, cu_q_lens.data_ptr(), int(max_q_len), Hq, Hkv, D,
        key_cache.data_ptr(), value_cache.data_ptr(), key_cache.stride(0), B,
        blocks, layout, block_table.data_ptr(),
        table_strides[0] if n > 1 else table[1], table[1],
        context_lens.data_ptr(), int(max_context_len), *extra,
        k_scale.data_ptr(), v_scale.data_ptr(), float(scale),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        out.data_ptr(), out_strides[0] if total > 1 else Hq * D, int(flags),
        _ptr(dev_error), here if stream is None else stream)
    _check(fn, st)


def kvq_chunk_attention_nvfp4(query: torch.Tensor, key_cache: torch.Tensor,
                              value_cache: torch.Tensor,
                              block_table: torch.Tensor,
                              cu_q_lens: torch.Tensor,
                              context_lens: torch.Tensor,
                              k_scale: torch.Tensor, v_scale: torch.Tensor,
                              scale: float, out: torch.Tensor,
                              max_q_len: int,
                              workspace: torch.Tensor | None = None,
                              max_context_len: int = 0, flags: int = 0,
                              dev_error: torch.Tensor | None = None,
                              stream: int | None = None) -> None:
    """Causal attention of chunks of new tokens over the NVFP4 cache (see
    ``include/kvq.h``).

    query / out: bf16 or fp16 [total_q, Hq, 128] (last two dims contiguous);
    sequence b's new tokens are rows cu_q_lens[b] .. cu_q_lens[b+1] - 1 and
    the last of its context_lens[b] cached tokens.  key_cache / value_cache:
    the store's 4-D page views; block_table int32 [num_seqs, max_blocks];
    cu_q_lens int32 [num_seqs + 1]; context_lens int32 [num_seqs];
    max_q_len: the longest chunk; max_context_len: the longest context (0:
    the block table's width).  The workspace (``chunk_attention_workspace``)
    is allocated here when it is not given."""
    _attend("kvq_chunk_attention_nvfp4", query, key_cache, value_cache,
            block_table, cu_q_lens, context_lens, (), (), k_scale, v_scale,
            scale, out, max_q_len, workspace, None, max_context_len, flags,
            dev_error, stream)


def kvq_tree_attention_nvfp4(query: torch.Tensor, key_cache: torch.Tensor,
                             value_cache: torch.Tensor,
                             block_table: torch.Tensor,
                             cu_q_lens: torch.Tensor,
                             context_lens: torch.Tensor,
                             tree_mask: torch.Tensor, k_scale: torch.Tensor,
                             v_scale: torch.Tensor, scale: float,
                             out: torch.Tensor, max_q_len: int,
                             workspace: torch.Tensor | None = None,
                             max_context_len: int = 0, flags: int = 0,
                             dev_error: torch.Tensor | None = None,
                             stream: int | None = None) -> None:
    """Attention of trees of drafted tokens over the NVFP4 cache (see
    ``include/kvq.h``): sequence b's drafts are rows cu_q_lens[b] ..
    cu_q_lens[b+1] - 1 and the last of its context_lens[b] cached tokens;
    bit j % 32 of tree_mask[r, j // 32] (int32 [total_q, words]) lets row r
    see its sequence's draft j.  Everything else as for
    ``kvq_chunk_attention_nvfp4``."""
    fn = "kvq_tree_attention_nvfp4"
    if query.dim() != 3:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    stride, words = _rows_of(fn, tree_mask, torch.int32, query.size(0))
    _attend(fn, query, key_cache, value_cache, block_table, cu_q_lens,
            context_lens, (tree_mask,),
            (tree_mask.data_ptr(), stride, words), k_scale,
            v_scale, scale, out, max_q_len, workspace, None, max_context_len,
            flags, dev_error, stream)


def kvq_quantize_indexer_q(q: torch.Tensor, weights: torch.Tensor,
                           scale: float, q_fp8: torch.Tensor,
                           weights_out: torch.Tensor, flags: int = 0,
                           stream: int | None = None) -> None:
    """The indexer's queries to fp8 (see ``include/kvq.h``): q bf16 or fp16
    [total_q, heads, head_dim] into q_fp8 (1-byte elements, the same shape,
    contiguous), weights fp32 [total_q, heads] times scale and each head's
    scale into weights_out (contiguous)."""
    fn = "kvq_quantize_indexer_q"
    dtype = _HALF_TYPES.get(q.dtype)
    if (dtype is None or q_fp8.element_size() != 1
            or weights_out.dtype is not torch.float32):
        raise KvqError(fn, KVQ_ERR_DTYPE)
    shape, strides = q.shape, q.stride()
    if len(shape) != 3 or q_fp8.shape != shape:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    total, heads, D = shape
    stride, width = _rows_of(fn, weights, torch.float32, total)
    if (strides[2] != 1 or strides[1] != D or width != heads
            or weights_out.shape != weights.shape
            or not q_fp8.is_contiguous() or not weights_out.is_contiguous()):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    here = _here(fn, q, weights, q_fp8, weights_out)
    st = lib().kvq_quantize_indexer_q(
        q.data_ptr(), strides[0] if total > 1 else heads * D, dtype,
        weights.data_ptr(), stride, float(scale), total, heads, D,
        q_fp8.data_ptr(), weights_out.data_ptr(), int(flags),
        here if stream is None else stream)
    _check(fn, st)


def kvq_score_blocks_indexer_k(q_fp8: torch.Tensor, weights: torch.Tensor,
                               kv_cache: torch.Tensor,
                               block_table: torch.Tensor,
                               cu_q_lens: torch.Tensor,
                               context_lens: torch.Tensor,
                               scores: torch.Tensor, select_block: int,
                               max_q_len: int,
                               block_size: int | None = None, flags: int = 0,
                               dev_error: torch.Tensor | None = None,
                               stream: int | None = None) -> None:
    """The indexer's score of every block of select_block tokens for every
    query row (see ``include/kvq.h``): q_fp8 e4m3 [total_q, heads, head_dim]
    and weights fp32 [total_q, heads] (``kvq_quantize_indexer_q``) against
    kv_cache uint8 [num_blocks, block_size, head_dim + 4] (or [num_blocks,
    bytes] with ``block_size`` given), into scores fp32 [total_q, columns];
    block_table, cu_q_lens, context_lens, max_q_len as for
    ``kvq_chunk_attention_nvfp4``."""
    fn = "kvq_score_blocks_indexer_k"
    if (kv_cache.element_size() != 1 or q_fp8.element_size() != 1
            or block_table.dtype is not torch.int32):
        raise KvqError(fn, KVQ_ERR_DTYPE)
    shape, strides = q_fp8.shape, q_fp8.stride()
    cache, cache_strides = kv_cache.shape, kv_cache.stride()
    if len(shape) != 3 or len(cache) not in (2, 3):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    total, heads, D = shape
    if block_size is None:
        if len(cache) != 3:
            raise KvqError(fn, KVQ_ERR_SHAPE)
        block_size = cache[1]
    # (a block's bytes lie together)
    held = cache[1] * (cache[2] if len(cache) == 3 else 1)
    if (cache_strides[-1] != 1 or held < block_size * (D + 4)
            or (len(cache) == 3 and cache_strides[1] != cache[2])):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    w_stride, width = _rows_of(fn, weights, torch.float32, total)
    s_stride, columns = _rows_of(fn, scores, torch.float32, total)
    _vector(fn, torch.int32, cu_q_lens, context_lens)
    n = context_lens.numel()
    table, table_strides = block_table.shape, block_table.stride()
    if (strides[2] != 1 or strides[1] != D or width != heads
            or cu_q_lens.numel() != n + 1 or len(table) != 2 or table[0] < n
            or (table[1] > 1 and table[0] > 0 and table_strides[1] != 1)):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    _dev_error_ok(fn, dev_error)
    here = _here(fn, q_fp8, weights, kv_cache, block_table, cu_q_lens,
                 context_lens, scores, dev_error)
    st = lib().kvq_score_blocks_indexer_k(
        q_fp8.data_ptr(), strides[0] if total > 1 else heads * D,
        weights.data_ptr(), w_stride, total, n, cu_q_lens.data_ptr(),
        int(max_q_len), heads, D, kv_cache.data_ptr(),
        cache_strides[0] if cache[0] > 1 else held, cache[0],
        int(block_size), block_table.data_ptr(),
        table_strides[0] if n > 1 else table[1], table[1],
        context_lens.data_ptr(), int(select_block), scores.data_ptr(),
        s_stride, columns, int(flags), _ptr(dev_error),
        here if stream is None else stream)
    _check(fn, st)


def kvq_select_blocks(scores: torch.Tensor, cu_q_lens: torch.Tensor,
                      context_lens: torch.Tensor, selected: torch.Tensor,
                      select_block: int, num_first: int = 0,
                      num_last: int = 0, flags: int = 0,
                      dev_error: torch.Tensor | None = None,
                      stream: int | None = None) -> None:
    """The blocks that each query row attends to (see ``include/kvq.h``): of
    scores fp32 [total_q, columns] into selected int32 [total_q,
    max_selected], rising, then -1; the first num_first and the last num_last
    blocks always."""
    fn = "kvq_select_blocks"
    if scores.dim() != 2:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    total = scores.size(0)
    s_stride, columns = _rows_of(fn, scores, torch.float32, total)
    l_stride, top = _rows_of(fn, selected, torch.int32, total)
    _vector(fn, torch.int32, cu_q_lens, context_lens)
    n = context_lens.numel()
    if cu_q_lens.numel() != n + 1:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    _dev_error_ok(fn, dev_error)
    here = _here(fn, scores, cu_q_lens, context_lens, selected, dev_error)
    st = lib().kvq_select_blocks(
        scores.data_ptr(), s_stride, columns, total, n,
        cu_q_lens.data_ptr(), context_lens.data_ptr(), int(select_block),
        int(num_first), int(num_last), selected.data_ptr(), l_stride, top,
        int(flags), _ptr(dev_error), here if stream is None else stream)
    _check(fn, st)


def sparse_attention_workspace(query: torch.Tensor, selected: torch.Tensor,
                               key_cache: torch.Tensor,
                               block_table: torch.Tensor,
                               select_block: int,
                               num_seqs: int | None = None,
                               max_context_len: int = 0) -> torch.Tensor:
    """Workspace of kvq_sparse_attention_nvfp4 for calls with these sizes, or
    with fewer rows or sequences (calls that may overlap each need their own).
    num_seqs: the sequences of a call (None: as many as the block table has
    rows); max_context_len: the longest context (0: the block table's
    width)."""
    if (query.dim() != 3 or selected.dim() != 2 or key_cache.dim() != 4
            or block_table.dim() != 2):
        raise KvqError("sparse_attention_workspace", KVQ_ERR_SHAPE)
    B, blocks = key_cache.size(1), block_table.size(1)
    if max_context_len > 0 and B > 0:
        blocks = min(blocks, -(-max_context_len // B))
    with torch.cuda.device(query.device):
        n = lib().kvq_sparse_attention_workspace_bytes(
            query.size(0),
            block_table.size(0) if num_seqs is None else num_seqs,
            query.size(1),
            key_cache.size(2), selected.size(1), int(select_block), B, blocks)
    if n < 0:
        raise KvqError("sparse_attention_workspace", KVQ_ERR_SHAPE)
    return torch.empty(n, dtype=torch.uint8, device=query.device)


def kvq_sparse_attention_nvfp4(query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor,
                               block_table: torch.Tensor,
                               cu_q_lens: torch.Tensor,
                               context_lens: torch.Tensor,
                               selected: torch.Tensor, select_block: int,
                               k_scale: torch.Tensor, v_scale: torch.Tensor,
                               scale: float, out: torch.Tensor,
                               max_q_len: int,
                               workspace: torch.Tensor | None = None,
                               max_context_len: int = 0, flags: int = 0,
                               dev_error: torch.Tensor | None = None,
                               stream: int | None = None) -> None:
    """Attention of each query row over the blocks of select_block tokens
    that selected int32 [total_q, max_selected] lists for it (see
    ``include/kvq.h``; rising, negative entries skipped:
    ``kvq_select_blocks``).  Everything else as for
    ``kvq_chunk_attention_nvfp4``; the workspace
    (``sparse_attention_workspace``) is allocated here when it is not
    given."""
    fn = "kvq_sparse_attention_nvfp4"
    if query.dim() != 3:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    stride, top = _rows_of(fn, selected, torch.int32, query.size(0))
    _attend(fn, query, key_cache, value_cache, block_table, cu_q_lens,
            context_lens, (selected,),
            (selected.data_ptr(), stride, top, int(select_block)), k_scale,
            v_scale, scale, out, max_q_len, workspace,
            lambda: sparse_attention_workspace(
                query, selected, key_cache, block_table, select_block,
                context_lens.numel(), max_context_len),
            max_context_len, flags, dev_error, stream)


def alloc_page_pool(num_blocks: int, num_rows: int, max_blocks_per_seq: int,
                    device="cuda"):
    """An empty page pool: (ref_count, block_table, seq_lens)."""
    return (torch.zeros(num_blocks, dtype=torch.int32, device=device),
            torch.full((num_rows, max_blocks_per_seq), -1,
                       dtype=torch.int32, device=device),
            torch.zeros(num_rows, dtype=torch.int32, device=device))


def _pool_args(fn: str, ref_count, block_table, seq_lens, dev_error,
               *others):
    """The state's checks; its leading C arguments, and the stream."""
    _vector(fn, torch.int32, ref_count, seq_lens)
    if block_table.dtype is not torch.int32:
        raise KvqError(fn, KVQ_ERR_DTYPE)
    if block_table.dim() != 2:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    rows, width = block_table.shape
    stride, step = block_table.stride()
    # (rows that overlap, as of an expanded table, would be written by
    # several)
    if rows != seq_lens.numel() or (rows and width and (
            (width > 1 and step != 1) or (rows > 1 and stride < width))):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    _dev_error_ok(fn, dev_error)
    here = _here(fn, ref_count, block_table, seq_lens, dev_error, *others)
    return (ref_count.data_ptr(), ref_count.numel(), block_table.data_ptr(),
            stride if rows > 1 and width else width, rows, width,
            seq_lens.data_ptr()), here


def _fill_none(stream: int | None, *slots) -> None:
    """-1 in the slots of a list without entries (the C entry launches
    nothing for one), on the call's stream."""
    for t in slots:
        if stream is None:
            t.fill_(-1)
            continue
        with torch.cuda.stream(
                torch.cuda.ExternalStream(stream, device=t.device) if stream
                else torch.cuda.default_stream(t.device)):
            t.fill_(-1)


def kvq_extend_sequences(ref_count: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, seq_ids: torch.Tensor,
                         cu_new: torch.Tensor, slot_mapping: torch.Tensor,
                         block_size: int, flags: int = 0,
                         dev_error: torch.Tensor | None = None,
                         stream: int | None = None) -> None:
    """Pages and slots for cu_new[i+1] - cu_new[i] new tokens of each row
    seq_ids[i] (see ``include/kvq.h``).  ref_count, block_table, seq_lens:
    ``alloc_page_pool``; seq_ids int32 [n]; cu_new int32 [n + 1];
    slot_mapping int64 [total], written whole."""
    fn = "kvq_extend_sequences"
    _vector(fn, torch.int32, seq_ids, cu_new)
    _vector(fn, torch.int64, slot_mapping)
    n = seq_ids.numel()
    if cu_new.numel() != n + 1:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    state, here = _pool_args(fn, ref_count, block_table, seq_lens, dev_error,
                             seq_ids, cu_new, slot_mapping)
    st = lib().kvq_extend_sequences(
        *state, int(block_size), seq_ids.data_ptr(), cu_new.data_ptr(), n,
        slot_mapping.data_ptr(), slot_mapping.numel(), int(flags),
        _ptr(dev_error), here if stream is None else stream)
    _check(fn, st)
    if n == 0:
        _fill_none(stream, slot_mapping)


def kvq_fork_sequences(ref_count: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, parent_ids: torch.Tensor,
                       child_ids: torch.Tensor, copy_src: torch.Tensor,
                       copy_dst: torch.Tensor, block_size: int,
                       flags: int = 0, dev_error: torch.Tensor | None = None,
                       stream: int | None = None) -> None:
    """Empty rows child_ids[i] become copies of rows parent_ids[i] (see
    ``include/kvq.h``); ``kvq_copy_pages(caches, copy_src, copy_dst)`` then
    copies the partly filled last pages.  All four lists int32 [n]."""
    fn = "kvq_fork_sequences"
    _vector(fn, torch.int32, parent_ids, child_ids, copy_src, copy_dst)
    n = parent_ids.numel()
    if any(t.numel() != n for t in (child_ids, copy_src, copy_dst)):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    state, here = _pool_args(fn, ref_count, block_table, seq_lens, dev_error,
                             parent_ids, child_ids, copy_src, copy_dst)
    st = lib().kvq_fork_sequences(
        *state, int(block_size), parent_ids.data_ptr(),
        child_ids.data_ptr(), n, copy_src.data_ptr(), copy_dst.data_ptr(),
        int(flags), _ptr(dev_error), here if stream is None else stream)
    _check(fn, st)


def kvq_compact_sequences(ref_count: torch.Tensor, block_table: torch.Tensor,
                          seq_lens: torch.Tensor, seq_ids: torch.Tensor,
                          keep: torch.Tensor, cu_keep: torch.Tensor,
                          src_slots: torch.Tensor, dst_slots: torch.Tensor,
                          block_size: int, flags: int = 0,
                          dev_error: torch.Tensor | None = None,
                          stream: int | None = None) -> None:
    """Rows seq_ids[i] keep the tokens at the rising positions
    keep[cu_keep[i] : cu_keep[i+1]] (see ``include/kvq.h``);
    ``kvq_move_tokens_nvfp4(caches, src_slots, dst_slots, cu_keep)`` then
    moves their bytes.  keep int32 [total]; src_slots, dst_slots int64
    [total], written whole."""
    fn = "kvq_compact_sequences"
    _vector(fn, torch.int32, seq_ids, keep, cu_keep)
    _vector(fn, torch.int64, src_slots, dst_slots)
    n = seq_ids.numel()
    if (cu_keep.numel() != n + 1 or src_slots.numel() != keep.numel()
            or dst_slots.numel() != keep.numel()):
        raise KvqError(fn, KVQ_ERR_SHAPE)
    state, here = _pool_args(fn, ref_count, block_table, seq_lens, dev_error,
                             seq_ids, keep, cu_keep, src_slots, dst_slots)
    st = lib().kvq_compact_sequences(
        *state, int(block_size), seq_ids.data_ptr(), keep.data_ptr(),
        cu_keep.data_ptr(), n, src_slots.data_ptr(), dst_slots.data_ptr(),
        keep.numel(), int(flags), _ptr(dev_error),
        here if stream is None else stream)
    _check(fn, st)
    if n == 0:
        _fill_none(stream, src_slots, dst_slots)


def kvq_free_sequences(ref_count: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, seq_ids: torch.Tensor,
                       flags: int = 0, dev_error: torch.Tensor | None = None,
                       stream: int | None = None) -> None:
    """Rows seq_ids[i] become empty, their pages are dropped (see
    ``include/kvq.h``)."""
    fn = "kvq_free_sequences"
    _vector(fn, torch.int32, seq_ids)
    state, here = _pool_args(fn, ref_count, block_table, seq_lens, dev_error,
                             seq_ids)
    st = lib().kvq_free_sequences(
        *state, seq_ids.data_ptr(), seq_ids.numel(), int(flags),
        _ptr(dev_error), here if stream is None else stream)
    _check(fn, st)


def _cache_list(fn: str, caches, dims: int):
    """(one cache's shape and strides, the addresses as a C array, how many,
    the tensors): caches is a list of uint8 tensors [num_blocks, ...] of one
    shape, or one tensor with the caches stacked in front."""
    if isinstance(caches, torch.Tensor):
        if caches.dtype is not torch.uint8:
            raise KvqError(fn, KVQ_ERR_DTYPE)
        shape, strides = caches.shape, caches.stride()
        if len(shape) < dims + 1 or shape[0] == 0:
            raise KvqError(fn, KVQ_ERR_SHAPE)
        n, step = shape[0], strides[0]
        shape, strides = shape[1:], strides[1:]
        if n > 1 and step < shape[0] * strides[0]:
            raise KvqError(fn, KVQ_ERR_SHAPE)  # caches would overlap
        base = caches.data_ptr()
        ptrs = range(base, base + n * step, step) if n > 1 else (base,)
        tensors = (caches,)
    else:
        tensors = tuple(caches)
        if not tensors:
            raise KvqError(fn, KVQ_ERR_SHAPE)
        n, shape, strides = len(tensors), tensors[0].shape, \
            tensors[0].stride()
        for t in tensors:
            if t.dtype is not torch.uint8:
                raise KvqError(fn, KVQ_ERR_DTYPE)
            if t.shape != shape or t.stride() != strides:
                raise KvqError(fn, KVQ_ERR_SHAPE)
        if len(shape) < dims:
            raise KvqError(fn, KVQ_ERR_SHAPE)
        ptrs = [t.data_ptr() for t in tensors]
        # (one cache twice: its tokens would be moved twice, at once)
        if n > 1 and shape[0] != 0 and len(set(ptrs)) < n:
            raise KvqError(fn, KVQ_ERR_SHAPE)
    # a page's bytes lie together
    page = 1
    for size, stride in zip(reversed(shape[1:]), reversed(strides[1:])):
        if size != 1 and stride != page:
            raise KvqError(fn, KVQ_ERR_SHAPE)
        page *= size
    return shape, strides, page, struct.pack(f"{n}P", *ptrs), n, tensors


def kvq_copy_pages(caches, src_pages: torch.Tensor, dst_pages: torch.Tensor,
                   flags: int = 0, dev_error: torch.Tensor | None = None,
                   stream: int | None = None) -> None:
    """Page dst_pages[i] := page src_pages[i] in every cache (see
    ``include/kvq.h``).  caches: a list of uint8 tensors [num_blocks, ...] of
    one shape, each page contiguous, or one tensor [n, num_blocks, ...];
    src_pages, dst_pages int32 [pairs], negative = skip."""
    fn = "kvq_copy_pages"
    shape, strides, page, ptrs, n, tensors = _cache_list(fn, caches, 2)
    _vector(fn, torch.int32, src_pages, dst_pages)
    if src_pages.numel() != dst_pages.numel():
        raise KvqError(fn, KVQ_ERR_SHAPE)
    _dev_error_ok(fn, dev_error)
    here = _here(fn, *tensors, src_pages, dst_pages, dev_error)
    if shape[0] == 0:
        return
    st = lib().kvq_copy_pages(
        ptrs, n, strides[0] if shape[0] > 1 else page, page, shape[0],
        src_pages.data_ptr(), dst_pages.data_ptr(), src_pages.numel(),
        int(flags), _ptr(dev_error), here if stream is None else stream)
    _check(fn, st)


def kvq_move_tokens_nvfp4(kv_caches, src_slots: torch.Tensor,
                          dst_slots: torch.Tensor, cu_moves: torch.Tensor,
                          layout: int = KVQ_LAYOUT_HND, flags: int = 0,
                          dev_error: torch.Tensor | None = None,
                          stream: int | None = None) -> None:
    """Tokens from slot to slot in every NVFP4 cache (see
    ``include/kvq.h``).  kv_caches: a list of ``alloc_nvfp4_cache``'s raw
    tensors [num_blocks, 2, H, B, D/2 + D/16] (HND; NHD has B before H), or
    one such tensor with the caches stacked in front; src_slots, dst_slots
    int64 [moves], negative = skip; cu_moves int32 [lists + 1]."""
    fn = "kvq_move_tokens_nvfp4"
    shape, strides, page, ptrs, n, tensors = _cache_list(fn, kv_caches, 5)
    if len(shape) != 5 or shape[1] != 2 or shape[4] % 9 != 0:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    if layout not in (KVQ_LAYOUT_HND, KVQ_LAYOUT_NHD):
        raise KvqError(fn, KVQ_ERR_LAYOUT)
    H, B = shape[2], shape[3]
    if layout == KVQ_LAYOUT_NHD:
        H, B = B, H
    _vector(fn, torch.int64, src_slots, dst_slots)
    _vector(fn, torch.int32, cu_moves)
    if src_slots.numel() != dst_slots.numel() or cu_moves.numel() < 1:
        raise KvqError(fn, KVQ_ERR_SHAPE)
    _dev_error_ok(fn, dev_error)
    here = _here(fn, *tensors, src_slots, dst_slots, cu_moves, dev_error)
    st = lib().kvq_move_tokens_nvfp4(
        ptrs, n, page // 2, strides[0] if shape[0] > 1 else page, shape[0],
        B, int(layout), H, shape[4] // 9 * 16, src_slots.data_ptr(),
        dst_slots.data_ptr(), src_slots.numel(), cu_moves.data_ptr(),
        cu_moves.numel() - 1, int(flags), _ptr(dev_error),
        here if stream is None else stream)
    _check(fn, st)


def alloc_nvfp4_cache(num_blocks: int, block_size: int, num_heads: int,
                      head_size: int, layout: int = KVQ_LAYOUT_HND,
                      device="cuda", fill: int | None = None):
    """Allocate an NVFP4 paged cache and return (kv_cache, key_cache,
    value_cache): kv_cache is the raw [num_blocks, 2, ...] uint8 tensor and
    key_cache / value_cache its two sides in the logical
    [num_blocks, block_size, num_heads, D/2 + D/16] order."""
    full = head_size // 2 + head_size // 16
    if layout == KVQ_LAYOUT_HND:
        kv = torch.empty(num_blocks, 2, num_heads, block_size, full,
                         dtype=torch.uint8, device=device)
        k, v = kv[:, 0].permute(0, 2, 1, 3), kv[:, 1].permute(0, 2, 1, 3)
    else:
        kv = torch.empty(num_blocks, 2, block_size, num_heads, full,
                         dtype=torch.uint8, device=device)
        k, v = kv[:, 0], kv[:, 1]
    if fill is not None:
        kv.fill_(fill)
    return kv, k, v
