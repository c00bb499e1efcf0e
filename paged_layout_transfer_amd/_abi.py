"""Constants, structures and descriptor builders of the C ABI in include/kvxfer.h.

Pure ctypes: importing this module loads nothing, so code that only builds
descriptors (or drives another build of the library) can use it without the HIP
runtime.  paged_layout_transfer_amd.kvxfer re-exports everything here.
"""
from __future__ import annotations

import ctypes
from typing import Iterable, Sequence

# ---- constants (mirror include/kvxfer.h) ---------------------------------------------
KV_OK = 0
KV_ERR_ARG = -1
KV_ERR_ALIGN = -2
KV_ERR_RANGE = -3
KV_ERR_OOM = -4
KV_ERR_RING = -5
KV_ERR_HIP = -6
KV_ERR_DEVICE = -7
KV_ERR_DUP = -8
KV_ERR_SCRATCH = -9
KV_ERR_CAPTURE = -10
KV_LAYER_FIRST = 0
KV_PAGE_FIRST = 1
KV_PAGE_TOKEN_MAJOR = 0
KV_PAGE_HEAD_MAJOR = 1
KV_GATHER = 0
KV_SCATTER = 1
KV_FLAG_VALIDATE = 0x1
KV_FLAG_DMA_STRIDED = 0x2
KV_FLAG_CACHED = 0x4
KV_FLAG_PAGE_RUNS = 0x8
KV_DEVERR_BLOCK_RANGE = 0x1
KV_RING_COHERENT = 0x0
KV_RING_NONCOHERENT = 0x1
KV_MAX_SPANS = 4096
KV_MAX_PAGE_COPIES = 65536
KV_MAX_SEQS = 4096
KV_MAX_ATTN_DIM = 256
KV_TYPE_F16 = 0
KV_TYPE_BF16 = 1
KV_TYPE_E4M3 = 2
KV_ATTN_FULL = 0x1
KV_VERSION = 300


class kv_pool_desc(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_kv", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("elem_bytes", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("page_layout", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64), ("block_stride", ctypes.c_int64),
                ("bases", ctypes.POINTER(ctypes.c_void_p))]


class kv_span(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_len", ctypes.c_int64),
                ("t_begin", ctypes.c_int64), ("t_end", ctypes.c_int64),
                ("first_chunk", ctypes.c_int64)]


class kv_chunk_spec(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("chunk_layers", ctypes.c_int32),
                ("chunk_tokens", ctypes.c_int64), ("layer_begin", ctypes.c_int32),
                ("layer_end", ctypes.c_int32), ("base", ctypes.c_void_p),
                ("slot_bytes", ctypes.c_int64), ("n_slots", ctypes.c_int64),
                ("max_workgroups", ctypes.c_int32), ("flags", ctypes.c_int32)]


class kv_transfer_info(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int64), ("chunks", ctypes.c_int64),
                ("payload_bytes", ctypes.c_int64), ("max_chunk_bytes", ctypes.c_int64)]


class kv_page_copy(ctypes.Structure):
    _fields_ = [("src", ctypes.c_int32), ("dst", ctypes.c_int32), ("n_tokens", ctypes.c_int32)]


class kv_seq(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_len", ctypes.c_int64),
                ("kv_len", ctypes.c_int64), ("q_begin", ctypes.c_int64),
                ("q_len", ctypes.c_int32), ("prefix_len", ctypes.c_int32)]


class kv_attn_desc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("q_type", ctypes.c_int32), ("kv_type", ctypes.c_int32),
                ("window", ctypes.c_int32), ("flags", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
                ("max_tokens", ctypes.c_int64)]


class kv_append_args(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("n_tokens", ctypes.c_int64), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class kv_attend_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("alibi_slopes", ctypes.c_void_p),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("n_tokens", ctypes.c_int64), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


def _addr(x) -> int:
    if x is None:
        return 0
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    return int(x)


# ---- descriptor builders ---------------------------------------------------------------

def make_pool_desc(num_layers: int, num_kv: int, num_heads: int, head_dim: int, elem_bytes: int,
                   block_size: int, num_blocks: int, block_stride: int,
                   bases: Sequence, page_layout: int = KV_PAGE_TOKEN_MAJOR) -> kv_pool_desc:
    """A kv_pool_desc; bases holds num_layers*num_kv device addresses (index l*num_kv+kv)."""
    arr = (ctypes.c_void_p * len(bases))(*[_addr(b) for b in bases])
    d = kv_pool_desc(num_layers, num_kv, num_heads, head_dim, elem_bytes, block_size, page_layout,
                     num_blocks, block_stride, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)))
    d._bases_keepalive = arr
    return d


def make_spans(spans: Iterable) -> ctypes.Array:
    """spans: (block_table, table_len, t_begin, t_end, first_chunk) tuples; block_table
    is a device address or tensor (a host address for kv_validate_targets)."""
    spans = list(spans)
    arr = (kv_span * max(1, len(spans)))()
    for i, (tbl, n, t0, t1, fc) in enumerate(spans):
        arr[i] = kv_span(_addr(tbl), int(n), int(t0), int(t1), int(fc))
    arr._n = len(spans)
    return arr


def make_chunk_spec(layout: int, chunk_layers: int, chunk_tokens: int, layer_begin: int,
                    layer_end: int, base, slot_bytes: int, n_slots: int,
                    max_workgroups: int = 0, flags: int = 0) -> kv_chunk_spec:
    return kv_chunk_spec(layout, chunk_layers, chunk_tokens, layer_begin, layer_end, _addr(base),
                         slot_bytes, n_slots, max_workgroups, flags)


def make_page_copies(copies: Iterable) -> ctypes.Array:
    """copies: (src, dst, n_tokens) triples, also for the moves of kv_remap_tables."""
    copies = list(copies)
    arr = (kv_page_copy * max(1, len(copies)))()
    for i, (src, dst, n) in enumerate(copies):
        arr[i] = kv_page_copy(int(src), int(dst), int(n))
    arr._n = len(copies)
    return arr


def make_seqs(seqs: Iterable) -> ctypes.Array:
    """seqs: (block_table, table_len, kv_len, q_begin, q_len[, prefix_len]) tuples; block_table is a device
    address or tensor."""
    seqs = list(seqs)
    arr = (kv_seq * max(1, len(seqs)))()
    for i, (tbl, n, kv_len, q_begin, q_len, *prefix) in enumerate(seqs):
        arr[i] = kv_seq(_addr(tbl), int(n), int(kv_len), int(q_begin), int(q_len), int(prefix[0]) if prefix else 0)
    arr._n = len(seqs)
    return arr


def make_attn_desc(num_q_heads: int, q_type: int, kv_type: int, max_seqs: int, max_tokens: int,
                   window: int = 0, flags: int = 0) -> kv_attn_desc:
    return kv_attn_desc(num_q_heads, q_type, kv_type, window, flags, max_seqs, max_tokens)


def _strides(x, strides):
    """(token, head) strides in elements: those given, or those of a [tokens][heads][dim] tensor,
    whose innermost dimension must be packed."""
    if strides is not None:
        return int(strides[0]), int(strides[1])
    if x.dim() != 3 or (x.shape[2] > 1 and x.stride(2) != 1):
        raise ValueError("a [tokens][heads][dim] tensor with packed dim, or its address and strides")
    return x.stride(0), x.stride(1)


def make_append_args(k, v, n_tokens: int, k_scale: float = 1.0, v_scale: float = 1.0, k_strides=None,
                     v_strides=None) -> kv_append_args:
    """k and v: [n_tokens][heads][dim] tensors, or device addresses with their (token, head) strides."""
    return kv_append_args(_addr(k), _addr(v), *_strides(k, k_strides), *_strides(v, v_strides), n_tokens, k_scale,
                          v_scale)


def make_attend_args(q, out, lse=None, *, n_tokens: int, scale: float, softcap: float = 0.0, alibi_slopes=None,
                     k_scale: float = 1.0, v_scale: float = 1.0, q_strides=None, out_strides=None) -> kv_attend_args:
    """q and out: [n_tokens][query heads][dim] tensors, or device addresses with their (token, head)
    strides; lse: [n_tokens][query heads] float32 or None."""
    return kv_attend_args(_addr(q), _addr(out), _addr(lse), _addr(alibi_slopes), *_strides(q, q_strides),
                          *_strides(out, out_strides), n_tokens, scale, softcap, k_scale, v_scale)


def _nspans(spans) -> int:
    return getattr(spans, "_n", len(spans))
