"""Python binding of libpagedkv.so: PagedAttention decode over a paged bf16 KV
cache on GB300, the cache-write and block-copy kernels, chunked prefill, and
the host block manager.

Argument marshalling only: each function reads sizes from tensor shapes,
checks device, dtype and contiguity, and calls the C entry point of the same
name on the current CUDA stream. Every computation runs in the library's
CUDA kernels; a missing library or a CPU tensor is an error.

Tensors: bf16 tensors may be torch.bfloat16 or int16/uint16 carrying bf16
bits. Pools are [num_blocks][n_kv_heads][16][head_dim]; block tables int32
[n_seqs][max_blocks]; context lengths int32 [n_seqs]; slots int64.
"""
from __future__ import annotations

import ctypes as C
from typing import List, Optional, Sequence, Tuple

from . import _capi
from ._capi import PagedKVError, check, load  # noqa: F401

__all__ = [
    "pa_decode", "pa_decode_tc", "pa_decode_workspace_bytes", "pa_decode_partition_tokens", "decode_workspace", "pa_decode_noalloc", "pa_reshape_and_cache",
    "pa_copy_blocks", "pa_prefill_paged", "pa_prefill_paged_ex", "pa_prefill_workspace_bytes",
    "prefill_workspace", "pa_reshape_and_cache_fp8", "pa_decode_fp8", "pa_decode_window",
    "pa_swap_out_blocks", "pa_swap_in_blocks", "pa_get_device_error", "pa_rope_and_cache",
    "pa_rope_and_cache_fp8_block", "pa_decode_sinks", "pa_decode_fp8_block",
    "pa_prefill_sinks", "pa_prefill_fp8_block", "pa_copy_blocks_fp8_block", "pa_decode_score_mod",
    "pa_prefill_score_mod", "pa_compact_blocks",
    "BlockManager", "load", "PagedKVError",
]


def _torch():
    import torch
    return torch


_BF16_LIKE = None


def _ptr(t, what: str, bf16: bool = False, dtype=None):
    torch = _torch()
    global _BF16_LIKE
    if _BF16_LIKE is None:
        _BF16_LIKE = {torch.bfloat16, torch.int16, getattr(torch, "uint16", torch.int16)}
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if bf16 and t.dtype not in _BF16_LIKE:
        raise TypeError(f"{what} must hold bf16 (bfloat16 or 16-bit integer bits), got {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def pa_decode_workspace_bytes(n_seqs: int, n_heads: int, head_dim: int, max_context_len: int,
                              partition_tokens: int = 0) -> int:
    return int(load().pa_decode_workspace_bytes(n_seqs, n_heads, head_dim, max_context_len,
                                                partition_tokens))


def pa_decode_partition_tokens(n_seqs: int, n_heads: int, n_kv_heads: int, head_dim: int,
                               max_context_len: int, window: int = -1, elem_bytes: int = 2) -> int:
    """The partition size the decode entry points use with partition_tokens=0."""
    st = int(load().pa_decode_partition_tokens(n_seqs, n_heads, n_kv_heads, head_dim, max_context_len,
                                               window, elem_bytes))
    check("pa_decode_partition_tokens", min(st, 0))
    return st


def decode_workspace(q, max_context_len: int, partition_tokens: int = 0):
    """A workspace tensor sized for pa_decode on this q shape and context bound."""
    torch = _torch()
    n_seqs, n_heads, head_dim = q.shape
    nbytes = pa_decode_workspace_bytes(n_seqs, n_heads, head_dim, max_context_len, partition_tokens)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)


def pa_decode(out, q, k_pool, v_pool, block_tables, context_lens, scale: float,
              max_context_len: int, workspace=None, partition_tokens: int = 0, stream=None,
              tensor_cores: bool = False) -> None:
    """out[b][h] = softmax(scale * q[b][h] . K_b^T) V_b over each sequence's
    paged K/V. q, out: [n_seqs][n_heads][head_dim]. tensor_cores=True calls
    pa_decode_tc (the warp-level MMA kernel at every group size)."""
    torch = _torch()
    n_seqs, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    if hd2 != head_dim or tuple(v_pool.shape) != tuple(k_pool.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q, out and the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != n_seqs or context_lens.numel() != n_seqs:
        raise ValueError("block_tables must be [n_seqs][max_blocks], context_lens [n_seqs]")
    ws_ptr, ws_bytes = C.c_void_p(None), 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    lib = load()
    st = (lib.pa_decode_tc if tensor_cores else lib.pa_decode_ex)(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), _ptr(k_pool, "k_pool", bf16=True),
        _ptr(v_pool, "v_pool", bf16=True), _ptr(block_tables, "block_tables", dtype=torch.int32),
        _ptr(context_lens, "context_lens", dtype=torch.int32), float(scale), n_heads, n_kv_heads,
        head_dim, block_size, n_seqs, block_tables.shape[1], int(max_context_len), num_blocks,
        int(partition_tokens), ws_ptr, ws_bytes, _stream(stream))
    check("pa_decode_tc" if tensor_cores else "pa_decode", st)


def pa_decode_tc(out, q, k_pool, v_pool, block_tables, context_lens, scale: float,
                 max_context_len: int, workspace=None, partition_tokens: int = 0, stream=None) -> None:
    """pa_decode on the tensor-core (warp-level MMA) partition kernel, any group size."""
    pa_decode(out, q, k_pool, v_pool, block_tables, context_lens, scale, max_context_len, workspace,
              partition_tokens, stream, tensor_cores=True)


def pa_decode_noalloc(out, q, k_pool, v_pool, block_tables, context_lens, scale: float,
                      max_context_len: int, stream=None) -> None:
    """pa_decode without a caller workspace, for callers that cannot allocate
    device memory: the split-K scratch is a fixed 32 MiB array inside the
    library shared by all calls on a device (calls that overlap on the GPU
    race on it). Batches needing more scratch raise (PA_ERR_WORKSPACE)."""
    torch = _torch()
    n_seqs, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    if hd2 != head_dim or tuple(v_pool.shape) != tuple(k_pool.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q, out and the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != n_seqs or context_lens.numel() != n_seqs:
        raise ValueError("block_tables must be [n_seqs][max_blocks], context_lens [n_seqs]")
    st = load().pa_decode_noalloc(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), _ptr(k_pool, "k_pool", bf16=True),
        _ptr(v_pool, "v_pool", bf16=True), _ptr(block_tables, "block_tables", dtype=torch.int32),
        _ptr(context_lens, "context_lens", dtype=torch.int32), float(scale), n_heads, n_kv_heads,
        head_dim, block_size, n_seqs, block_tables.shape[1], int(max_context_len), num_blocks,
        _stream(stream))
    check("pa_decode_noalloc", st)


def pa_reshape_and_cache(k, v, k_pool, v_pool, slot_mapping, stream=None) -> None:
    """Writes k[t], v[t] ([n_tokens][n_kv_heads][head_dim]) to slot_mapping[t]."""
    torch = _torch()
    n_tokens, n_kv_heads, head_dim = k.shape
    num_blocks, hk2, block_size, hd2 = k_pool.shape
    if (hk2, hd2) != (n_kv_heads, head_dim) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch between k/v and the pools")
    if slot_mapping.numel() != n_tokens:
        raise ValueError("slot_mapping must have n_tokens entries")
    st = load().pa_reshape_and_cache(
        _ptr(k, "k", bf16=True), _ptr(v, "v", bf16=True), _ptr(k_pool, "k_pool", bf16=True),
        _ptr(v_pool, "v_pool", bf16=True), _ptr(slot_mapping, "slot_mapping", dtype=torch.int64),
        n_tokens, n_kv_heads, head_dim, block_size, num_blocks, _stream(stream))
    check("pa_reshape_and_cache", st)


def _fp8_pool(t, what: str):
    torch = _torch()
    if t.dtype not in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        raise TypeError(f"{what} must hold E4M3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
    return _ptr(t, what)


def pa_decode_window(out, q, k_pool, v_pool, block_tables, context_lens, scale: float,
                     max_context_len: int, window: int, workspace=None, partition_tokens: int = 0,
                     stream=None) -> None:
    """Sliding-window decode: the query at position ctx-1 attends to positions
    ctx-1-window .. ctx-1; blocks wholly before that are never read."""
    torch = _torch()
    n_seqs, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    if hd2 != head_dim or tuple(v_pool.shape) != tuple(k_pool.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q, out and the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != n_seqs or context_lens.numel() != n_seqs:
        raise ValueError("block_tables must be [n_seqs][max_blocks], context_lens [n_seqs]")
    ws_ptr, ws_bytes = C.c_void_p(None), 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pa_decode_window(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), _ptr(k_pool, "k_pool", bf16=True),
        _ptr(v_pool, "v_pool", bf16=True), _ptr(block_tables, "block_tables", dtype=torch.int32),
        _ptr(context_lens, "context_lens", dtype=torch.int32), float(scale), n_heads, n_kv_heads,
        head_dim, block_size, n_seqs, block_tables.shape[1], int(max_context_len), num_blocks, int(window),
        int(partition_tokens), ws_ptr, ws_bytes, _stream(stream))
    check("pa_decode_window", st)


def _host_pinned(t, what: str):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.device.type != "cpu" or not t.is_pinned():
        raise ValueError(f"{what} must be page-locked host memory (pin_memory=True)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return C.c_void_p(t.data_ptr())


def _swap_args(k_pool, host_k, host_v, block_ids):
    torch = _torch()
    num_blocks, n_kv_heads, block_size, head_dim = k_pool.shape
    eb = k_pool.element_size()
    n = block_ids.numel()
    need = n * n_kv_heads * block_size * head_dim * eb
    for h, name in ((host_k, "host_k"), (host_v, "host_v")):
        if h.numel() * h.element_size() < need:
            raise ValueError(f"{name} holds fewer than {need} bytes")
    return (n, n_kv_heads, head_dim, block_size, eb, num_blocks,
            _ptr(block_ids, "block_ids", dtype=torch.int32) if n else C.c_void_p(None))


def pa_swap_out_blocks(k_pool, v_pool, block_ids, host_k, host_v, stream=None) -> None:
    """host_k[i], host_v[i] := pool block block_ids[i] (K and V, all heads);
    host buffers page-locked, block_ids int32 on the device. Scales per block
    stay behind: keep k_scale[block_ids] and v_scale[block_ids] beside them."""
    n, hk, d, bs, eb, nb, ids = _swap_args(k_pool, host_k, host_v, block_ids)
    st = load().pa_swap_out_blocks(_ptr(k_pool, "k_pool"), _ptr(v_pool, "v_pool"), ids, n,
                                   _host_pinned(host_k, "host_k"), _host_pinned(host_v, "host_v"), hk, d, bs,
                                   eb, nb, _stream(stream))
    check("pa_swap_out_blocks", st)


def pa_swap_in_blocks(host_k, host_v, k_pool, v_pool, block_ids, stream=None) -> None:
    """pool block block_ids[i] := host_k[i], host_v[i]. Of a cache with a scale
    per block, put the kept rows at k_scale[block_ids] and v_scale[block_ids] too."""
    n, hk, d, bs, eb, nb, ids = _swap_args(k_pool, host_k, host_v, block_ids)
    st = load().pa_swap_in_blocks(_host_pinned(host_k, "host_k"), _host_pinned(host_v, "host_v"),
                                  _ptr(k_pool, "k_pool"), _ptr(v_pool, "v_pool"), ids, n, hk, d, bs, eb, nb,
                                  _stream(stream))
    check("pa_swap_in_blocks", st)


def pa_reshape_and_cache_fp8(k, v, k_pool, v_pool, slot_mapping, k_scale, v_scale, stream=None) -> None:
    """Encodes k[t], v[t] (bf16 [n_tokens][n_kv_heads][head_dim]) as E4M3 codes
    of x / scale[head] into the uint8 pools at slot_mapping[t]."""
    torch = _torch()
    n_tokens, n_kv_heads, head_dim = k.shape
    num_blocks, hk2, block_size, hd2 = k_pool.shape
    if (hk2, hd2) != (n_kv_heads, head_dim) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch between k/v and the pools")
    if slot_mapping.numel() != n_tokens or k_scale.numel() != n_kv_heads or v_scale.numel() != n_kv_heads:
        raise ValueError("slot_mapping needs n_tokens entries, k_scale/v_scale n_kv_heads")
    st = load().pa_reshape_and_cache_fp8(
        _ptr(k, "k", bf16=True), _ptr(v, "v", bf16=True), _fp8_pool(k_pool, "k_pool"),
        _fp8_pool(v_pool, "v_pool"), _ptr(slot_mapping, "slot_mapping", dtype=torch.int64),
        _ptr(k_scale, "k_scale", dtype=torch.float32), _ptr(v_scale, "v_scale", dtype=torch.float32),
        n_tokens, n_kv_heads, head_dim, block_size, num_blocks, _stream(stream))
    check("pa_reshape_and_cache_fp8", st)


def pa_decode_fp8(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale: float,
                  max_context_len: int, workspace=None, partition_tokens: int = 0, stream=None) -> None:
    """pa_decode over an E4M3 cache: K and V are decode(code) * scale of their
    KV head. Pools uint8 [num_blocks][n_kv_heads][16][head_dim]."""
    torch = _torch()
    n_seqs, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    if hd2 != head_dim or tuple(v_pool.shape) != tuple(k_pool.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q, out and the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != n_seqs or context_lens.numel() != n_seqs:
        raise ValueError("block_tables must be [n_seqs][max_blocks], context_lens [n_seqs]")
    if k_scale.numel() != n_kv_heads or v_scale.numel() != n_kv_heads:
        raise ValueError("k_scale and v_scale need one entry per KV head")
    ws_ptr, ws_bytes = C.c_void_p(None), 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pa_decode_fp8(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), _fp8_pool(k_pool, "k_pool"),
        _fp8_pool(v_pool, "v_pool"), _ptr(k_scale, "k_scale", dtype=torch.float32),
        _ptr(v_scale, "v_scale", dtype=torch.float32), _ptr(block_tables, "block_tables", dtype=torch.int32),
        _ptr(context_lens, "context_lens", dtype=torch.int32), float(scale), n_heads, n_kv_heads,
        head_dim, block_size, n_seqs, block_tables.shape[1], int(max_context_len), num_blocks,
        int(partition_tokens), ws_ptr, ws_bytes, _stream(stream))
    check("pa_decode_fp8", st)


def _attention_args(out, q, k_pool, v_pool, k_scale, v_scale, per_block, block_tables, context_lens, n_seqs):
    """What the attention calls below check alike: (device, the addresses up to
    the scales, those of the tables and lengths, the sizes)."""
    dev = _device(q, "q")
    T = _Types
    n, n_heads, head_dim = shape = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = pool_shape = k_pool.shape
    if hd2 != head_dim or v_pool.shape != pool_shape or out.shape != shape:
        raise ValueError("shape mismatch between q, out and the pools")
    rows, max_blocks = block_tables.shape
    if rows != n_seqs or context_lens.numel() != n_seqs:
        raise ValueError("block_tables must be [n_seqs][max_blocks], context_lens [n_seqs]")
    pool_types, ks, vs = T.bf16, None, None
    if k_scale is not None and v_scale is not None:
        ns = num_blocks * n_kv_heads if per_block else n_kv_heads
        if k_scale.numel() != ns or v_scale.numel() != ns:
            raise ValueError(f"k_scale and v_scale need {ns} entries")
        ks, vs = _at(k_scale, "k_scale", T.f32, dev), _at(v_scale, "v_scale", T.f32, dev)
        pool_types = T.e4m3
    elif per_block:
        raise ValueError("k_scale and v_scale are needed")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale go together")
    data = (_at(out, "out", T.bf16, dev), _at(q, "q", T.bf16, dev), _at(k_pool, "k_pool", pool_types, dev),
            _at(v_pool, "v_pool", pool_types, dev), ks, vs)
    tables = (_at(block_tables, "block_tables", T.i32, dev), _at(context_lens, "context_lens", T.i32, dev))
    return dev, data, tables, (n_heads, n_kv_heads, head_dim, block_size, n_seqs, max_blocks), num_blocks


def _decode_call(fn: str, per_block: bool, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
                 max_context_len, window, n_sinks, workspace, partition_tokens, stream) -> None:
    dev, data, tables, sizes, num_blocks = _attention_args(out, q, k_pool, v_pool, k_scale, v_scale, per_block,
                                                           block_tables, context_lens, q.shape[0])
    longest, window, n_sinks, partition_tokens = _ints(max_context_len, window, n_sinks, partition_tokens)
    _call(fn, dev, stream, *data, *tables, float(scale), *sizes, longest, num_blocks, window, n_sinks, partition_tokens,
          *_workspace(workspace, dev))


def pa_decode_sinks(out, q, k_pool, v_pool, block_tables, context_lens, scale: float, max_context_len: int,
                    window: int, n_sinks: int, k_scale=None, v_scale=None, workspace=None, partition_tokens: int = 0,
                    stream=None) -> None:
    """Sliding-window decode whose first n_sinks positions stay visible: the
    query at i = ctx-1 attends to t <= i with t >= i-window or t < n_sinks.
    bf16 pools, or uint8 pools with k_scale and v_scale fp32 [n_kv_heads]."""
    _decode_call("pa_decode_sinks", False, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
                 max_context_len, window, n_sinks, workspace, partition_tokens, stream)


def pa_decode_fp8_block(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale: float,
                        max_context_len: int, window: int = -1, n_sinks: int = 0, workspace=None,
                        partition_tokens: int = 0, stream=None) -> None:
    """Decode over an E4M3 cache with a scale per block and head (k_scale,
    v_scale fp32 [num_blocks][n_kv_heads], see pa_rope_and_cache_fp8_block);
    window >= 0: as pa_decode_sinks."""
    _decode_call("pa_decode_fp8_block", True, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
                 max_context_len, window, n_sinks, workspace, partition_tokens, stream)


def _head_slopes(alibi_slopes, n_heads: int, dev: int):
    if alibi_slopes.numel() != n_heads:
        raise ValueError(f"alibi_slopes needs {n_heads} entries")
    return _at(alibi_slopes, "alibi_slopes", _Types.f32, dev)


def pa_decode_score_mod(out, q, k_pool, v_pool, block_tables, context_lens, scale: float, max_context_len: int,
                        softcap: float = 0.0, alibi_slopes=None, window: int = -1, n_sinks: int = 0, k_scale=None,
                        v_scale=None, workspace=None, partition_tokens: int = 0, stream=None) -> None:
    """Decode with reshaped scores: s = scale q.k becomes softcap tanh(s / softcap)
    (softcap > 0), less alibi_slopes[head] times the key's distance (fp32 [n_heads]).
    Masks as pa_decode_sinks (window -1: none). bf16 pools, or E4M3 pools with a
    scale per block and head (k_scale, v_scale fp32 [num_blocks][n_kv_heads])."""
    dev, data, tables, sizes, num_blocks = _attention_args(out, q, k_pool, v_pool, k_scale, v_scale,
                                                           k_scale is not None and v_scale is not None, block_tables,
                                                           context_lens, q.shape[0])
    longest, window, n_sinks, partition_tokens = _ints(max_context_len, window, n_sinks, partition_tokens)
    _call("pa_decode_score_mod", dev, stream, *data, *tables, float(scale), float(softcap),
          None if alibi_slopes is None else _head_slopes(alibi_slopes, sizes[0], dev), *sizes, longest, num_blocks, window,
          n_sinks, partition_tokens, *_workspace(workspace, dev))


def pa_decode_plan(context_lens, n_heads: int, n_kv_heads: int, head_dim: int, max_blocks_per_seq: int,
                   max_context_len: int, num_blocks: int, window: int = -1, elem_bytes: int = 2,
                   partition_tokens: int = 0):
    """The decode call's work items, longest partitions first, from HOST
    context lengths (a sequence of ints or an int32 array): an int32 numpy
    array [n_items][4] of (partition, kv head, sequence, 0)."""
    import numpy as np
    ctx = np.ascontiguousarray(np.asarray(context_lens, dtype=np.int32).reshape(-1))
    args = (ctx.ctypes.data_as(C.c_void_p), len(ctx), n_heads, n_kv_heads, head_dim, max_blocks_per_seq,
            int(max_context_len), num_blocks, int(window), elem_bytes, int(partition_tokens))
    n = int(load().pa_decode_plan(*args, None, 0))
    check("pa_decode_plan", min(n, 0))
    items = np.zeros((max(n, 1), 4), dtype=np.int32)
    st = int(load().pa_decode_plan(*args, items.ctypes.data_as(C.c_void_p), n))
    check("pa_decode_plan", min(st, 0))
    return items[:st]


def pa_decode_planned(out, q, k_pool, v_pool, block_tables, context_lens, scale: float, max_context_len: int,
                      items, k_scale=None, v_scale=None, window: int = -1, workspace=None,
                      partition_tokens: int = 0, stream=None) -> None:
    """pa_decode (bf16 pools), pa_decode_fp8 (uint8 pools with k_scale and
    v_scale) or, with window >= 0, pa_decode_window, run from a plan: items is
    pa_decode_plan's output for the same lengths and arguments, on the device
    (int32 [n_items][4])."""
    torch = _torch()
    n_seqs, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    if hd2 != head_dim or tuple(v_pool.shape) != tuple(k_pool.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q, out and the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != n_seqs or context_lens.numel() != n_seqs:
        raise ValueError("block_tables must be [n_seqs][max_blocks], context_lens [n_seqs]")
    if items.dim() != 2 or items.shape[1] != 4:
        raise ValueError("items must be int32 [n_items][4]")
    fp8 = k_pool.dtype == torch.uint8
    if fp8 != (k_scale is not None) or (k_scale is None) != (v_scale is None):
        raise ValueError("an fp8 (uint8) pool needs k_scale and v_scale, a bf16 pool neither")
    ws_ptr, ws_bytes = C.c_void_p(None), 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    if fp8:
        kp, vp_ = _fp8_pool(k_pool, "k_pool"), _fp8_pool(v_pool, "v_pool")
        ks = _ptr(k_scale, "k_scale", dtype=torch.float32)
        vs = _ptr(v_scale, "v_scale", dtype=torch.float32)
    else:
        kp, vp_ = _ptr(k_pool, "k_pool", bf16=True), _ptr(v_pool, "v_pool", bf16=True)
        ks = vs = C.c_void_p(None)
    st = load().pa_decode_planned(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), kp, vp_, ks, vs,
        _ptr(block_tables, "block_tables", dtype=torch.int32), _ptr(context_lens, "context_lens", dtype=torch.int32),
        float(scale), n_heads, n_kv_heads, head_dim, block_size, n_seqs, block_tables.shape[1],
        int(max_context_len), num_blocks, int(window), int(partition_tokens),
        _ptr(items, "items", dtype=torch.int32), items.shape[0], ws_ptr, ws_bytes, _stream(stream))
    check("pa_decode_planned", st)


class _Types:
    """dtypes an argument may have, and the per-device stream lookup; filled on
    first use, as torch is imported lazily."""
    ready = False

    @classmethod
    def fill(cls):
        torch = _torch()
        cls.bf16 = (torch.bfloat16, torch.int16, getattr(torch, "uint16", torch.int16))
        cls.e4m3 = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))
        cls.movable = cls.bf16 + cls.e4m3
        cls.f32, cls.i32, cls.i64 = (torch.float32,), (torch.int32,), (torch.int64,)
        # torch.cuda.current_device() checks each time whether CUDA is initialised, 0.2 us (a CUDA tensor is at hand);
        # torch.cuda.current_stream() takes 3 us to build its object; a small launch takes 2
        device = getattr(torch._C, "_cuda_getDevice", None)
        cls.current_device = staticmethod(device or torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.raw_stream = staticmethod(raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
        cls.ready = True


def _device(t, what: str) -> int:
    """The CUDA device index of the call's first tensor."""
    if not _Types.ready:
        _Types.fill()
    dev = t.get_device() if isinstance(t, _torch().Tensor) else -1
    if dev < 0:
        _refuse(t, what, None, 0)
    return dev


def _at(t, what: str, dtypes, dev: int, strided: bool = False) -> int:
    """The address of an argument on device `dev`, contiguous (or not, if
    strided), of one of `dtypes` (None: any)."""
    try:
        if t.get_device() == dev and (dtypes is None or t.dtype in dtypes) and (strided or t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, what, dtypes, dev)


def _refuse(t, what: str, dtypes, dev: int):
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (the library has no CPU path)")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, the other tensors on cuda:{dev}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dict.fromkeys(dtypes))}, got {t.dtype}")
    raise ValueError(f"{what} must be contiguous")


def _call(fn: str, dev: int, stream, *args) -> None:
    """Calls the C entry point with device `dev` current, on `stream` or that
    device's current stream."""
    if dev != _Types.current_device():
        with _torch().cuda.device(dev):
            return _call(fn, dev, stream, *args)
    st = getattr(_capi._lib or load(), fn)(*args, _Types.raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        check(fn, st)


def _ints(a, b, c, d):
    """The values as C ints (a larger one would be cut to its low 32 bits)."""
    a, b, c, d = int(a), int(b), int(c), int(d)
    if (a <= 0x7fffffff and b <= 0x7fffffff and c <= 0x7fffffff and d <= 0x7fffffff and
            a >= -0x80000000 and b >= -0x80000000 and c >= -0x80000000 and d >= -0x80000000):
        return a, b, c, d
    raise ValueError(f"a size, window or count does not fit 32 bits: {(a, b, c, d)}")


def _workspace(t, dev: int):
    return (None, 0) if t is None else (_at(t, "workspace", None, dev), t.numel() * t.element_size())


def _token_stride(t, what: str, n: int, heads: int, dim: int) -> int:
    """Elements between the tokens of [n][heads][dim], whose heads must be
    contiguous (a view of a packed projection will do)."""
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != dim and heads > 1):
        raise ValueError(f"{what} must have contiguous heads")
    return s0 if n > 1 else heads * dim


def _rope(fn: str, per_block: bool, q_out, q, k, v, k_pool, v_pool, k_scale, v_scale, cos_sin, positions, slot_mapping,
          interleaved, stream) -> None:
    dev = _device(k, "k")
    T = _Types
    n_tokens, n_kv_heads, head_dim = shape = k.shape
    num_blocks, hk2, block_size, hd2 = pool_shape = k_pool.shape
    if hk2 != n_kv_heads or hd2 != head_dim or v.shape != shape or v_pool.shape != pool_shape:
        raise ValueError("shape mismatch between k/v and the pools")
    n_heads = rot = max_position = qo_stride = q_stride = 0
    q_at = qo_at = cs_at = pos_at = ks_at = vs_at = None
    if q is not None and q_out is not None:
        nq, n_heads, dq = q.shape
        if nq != n_tokens or dq != head_dim or q_out.shape != q.shape:
            raise ValueError("q and q_out must be [n_tokens][n_heads][head_dim]")
        q_at, qo_at = _at(q, "q", T.bf16, dev, True), _at(q_out, "q_out", T.bf16, dev, True)
        q_stride = _token_stride(q, "q", n_tokens, n_heads, head_dim)
        qo_stride = _token_stride(q_out, "q_out", n_tokens, n_heads, head_dim)
    elif q is not None or q_out is not None:
        raise ValueError("q and q_out go together")
    if slot_mapping.numel() != n_tokens:
        raise ValueError("slot_mapping must have n_tokens entries")
    if cos_sin is not None:
        if cos_sin.dim() != 2 or positions is None or positions.numel() != n_tokens:
            raise ValueError("cos_sin must be [max_position][rot_dim], positions [n_tokens]")
        max_position, rot = cos_sin.shape
        cs_at, pos_at = _at(cos_sin, "cos_sin", T.f32, dev), _at(positions, "positions", T.i64, dev)
    pool_types = T.bf16
    if k_scale is not None and v_scale is not None:
        n = num_blocks * n_kv_heads if per_block else n_kv_heads
        if k_scale.numel() != n or v_scale.numel() != n:
            raise ValueError(f"k_scale and v_scale need {n} entries")
        ks_at, vs_at = _at(k_scale, "k_scale", T.f32, dev), _at(v_scale, "v_scale", T.f32, dev)
        pool_types = T.e4m3
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale go together")
    rest = (cs_at, pos_at, _at(slot_mapping, "slot_mapping", T.i64, dev))
    _call(fn, dev, stream, qo_at, q_at, _at(k, "k", T.bf16, dev, True), _at(v, "v", T.bf16, dev, True),
          _at(k_pool, "k_pool", pool_types, dev), _at(v_pool, "v_pool", pool_types, dev),
          *((ks_at, vs_at) + rest if per_block else rest + (ks_at, vs_at)), qo_stride, q_stride,
          _token_stride(k, "k", n_tokens, n_kv_heads, head_dim), _token_stride(v, "v", n_tokens, n_kv_heads, head_dim),
          n_tokens, n_heads, n_kv_heads, head_dim, rot, max_position, 1 if interleaved else 0, block_size, num_blocks)


def pa_rope_and_cache(q_out, q, k, v, k_pool, v_pool, cos_sin, positions, slot_mapping, interleaved: bool = False,
                      k_scale=None, v_scale=None, stream=None) -> None:
    """Rotates q and k by their tokens' positions and writes k and v to
    slot_mapping[t], in one launch. q, k, v: [n_tokens][heads][head_dim], bf16,
    views of a packed projection allowed (contiguous heads); q_out may be q.
    cos_sin fp32 [max_position][rot_dim] (cosines, then sines), positions int64;
    cos_sin None: no rotation; q and q_out None: only k and v. bf16 pools, or
    uint8 pools with k_scale and v_scale fp32 [n_kv_heads]."""
    _rope("pa_rope_and_cache", False, q_out, q, k, v, k_pool, v_pool, k_scale, v_scale, cos_sin, positions, slot_mapping,
          interleaved, stream)


def pa_rope_and_cache_fp8_block(q_out, q, k, v, k_pool, v_pool, k_scale, v_scale, cos_sin, positions, slot_mapping,
                                interleaved: bool = False, stream=None) -> None:
    """pa_rope_and_cache into E4M3 pools with a scale per block and head:
    k_scale, v_scale fp32 [num_blocks][n_kv_heads], set and raised by the call.
    A call's tokens of one block must lie within 16 consecutive entries of slot_mapping."""
    if k_scale is None or v_scale is None:
        raise ValueError("k_scale and v_scale are needed")
    _rope("pa_rope_and_cache_fp8_block", True, q_out, q, k, v, k_pool, v_pool, k_scale, v_scale, cos_sin, positions,
          slot_mapping, interleaved, stream)


def pa_copy_blocks(k_pool, v_pool, block_mapping, stream=None) -> None:
    """block_mapping int64 [n][2] (src, dst) on the device: dst block := src block.
    The pools may be bf16 or fp8 (uint8 E4M3 codes); the element size is read
    from k_pool."""
    torch = _torch()
    num_blocks, n_kv_heads, block_size, head_dim = k_pool.shape
    n_pairs = block_mapping.shape[0] if block_mapping.numel() else 0
    if k_pool.dtype == torch.uint8:
        kp, vp_, eb = _fp8_pool(k_pool, "k_pool"), _fp8_pool(v_pool, "v_pool"), 1
    else:
        kp, vp_, eb = _ptr(k_pool, "k_pool", bf16=True), _ptr(v_pool, "v_pool", bf16=True), 2
    if v_pool.dtype != k_pool.dtype or tuple(v_pool.shape) != tuple(k_pool.shape):
        raise ValueError("k_pool and v_pool must have the same shape and dtype")
    st = load().pa_copy_blocks_ex(
        kp, vp_, _ptr(block_mapping, "block_mapping", dtype=torch.int64) if n_pairs else C.c_void_p(None),
        n_pairs, n_kv_heads, head_dim, block_size, eb, num_blocks, _stream(stream))
    check("pa_copy_blocks_ex", st)


def pa_prefill_paged(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc,
                     scale: float, max_chunk_len: int, stream=None) -> None:
    """Causal attention of each sequence's chunk rows over its paged cache."""
    torch = _torch()
    n_rows, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    n_seqs = context_lens.numel()
    if hd2 != head_dim or tuple(out.shape) != tuple(q.shape) or q_start_loc.numel() != n_seqs + 1:
        raise ValueError("shape mismatch in pa_prefill_paged arguments")
    st = load().pa_prefill_paged(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), _ptr(k_pool, "k_pool", bf16=True),
        _ptr(v_pool, "v_pool", bf16=True), _ptr(block_tables, "block_tables", dtype=torch.int32),
        _ptr(context_lens, "context_lens", dtype=torch.int32),
        _ptr(q_start_loc, "q_start_loc", dtype=torch.int32), float(scale), n_heads, n_kv_heads,
        head_dim, block_size, n_seqs, block_tables.shape[1], int(max_chunk_len), num_blocks,
        _stream(stream))
    check("pa_prefill_paged", st)


def pa_prefill_workspace_bytes(n_seqs: int, n_heads: int, n_kv_heads: int, max_chunk_len: int,
                               splits: int = 0) -> int:
    return int(load().pa_prefill_workspace_bytes(n_seqs, n_heads, n_kv_heads, max_chunk_len, splits))


def prefill_workspace(q, n_seqs: int, n_kv_heads: int, max_chunk_len: int, splits: int = 0):
    """A workspace tensor for pa_prefill_paged_ex (None when no split is needed)."""
    torch = _torch()
    nbytes = pa_prefill_workspace_bytes(n_seqs, q.shape[1], n_kv_heads, max_chunk_len, splits)
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None


def pa_prefill_paged_ex(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale: float,
                        max_chunk_len: int, splits: int = 0, workspace=None, stream=None) -> None:
    """pa_prefill_paged with each query-tile pair's key range split into pieces
    (splits = 0: chosen from the grid and the SM count) merged afterwards."""
    torch = _torch()
    n_rows, n_heads, head_dim = q.shape
    num_blocks, n_kv_heads, block_size, hd2 = k_pool.shape
    n_seqs = context_lens.numel()
    if hd2 != head_dim or tuple(out.shape) != tuple(q.shape) or q_start_loc.numel() != n_seqs + 1:
        raise ValueError("shape mismatch in pa_prefill_paged_ex arguments")
    ws_ptr, ws_bytes = C.c_void_p(None), 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pa_prefill_paged_ex(
        _ptr(out, "out", bf16=True), _ptr(q, "q", bf16=True), _ptr(k_pool, "k_pool", bf16=True),
        _ptr(v_pool, "v_pool", bf16=True), _ptr(block_tables, "block_tables", dtype=torch.int32),
        _ptr(context_lens, "context_lens", dtype=torch.int32),
        _ptr(q_start_loc, "q_start_loc", dtype=torch.int32), float(scale), n_heads, n_kv_heads,
        head_dim, block_size, n_seqs, block_tables.shape[1], int(max_chunk_len), num_blocks, int(splits),
        ws_ptr, ws_bytes, _stream(stream))
    check("pa_prefill_paged_ex", st)


def _prefill_call(fn: str, per_block: bool, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                  q_start_loc, scale, max_chunk_len, window, n_sinks, splits, workspace, stream) -> None:
    n_seqs = context_lens.numel()
    if q_start_loc.numel() != n_seqs + 1:
        raise ValueError("q_start_loc must have n_seqs + 1 entries")
    dev, data, tables, sizes, num_blocks = _attention_args(out, q, k_pool, v_pool, k_scale, v_scale, per_block,
                                                           block_tables, context_lens, n_seqs)
    longest, window, n_sinks, splits = _ints(max_chunk_len, window, n_sinks, splits)
    _call(fn, dev, stream, *(data if per_block else data[:4]), *tables, _at(q_start_loc, "q_start_loc", _Types.i32, dev),
          float(scale), *sizes, longest, num_blocks, window, n_sinks, splits, *_workspace(workspace, dev))


def pa_prefill_sinks(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale: float, max_chunk_len: int,
                     window: int, n_sinks: int, splits: int = 0, workspace=None, stream=None) -> None:
    """pa_prefill_paged_ex under a sliding window whose first n_sinks positions
    stay visible: a row at position p attends to t <= p with t >= p-window or
    t < n_sinks. Workspace: prefill_workspace."""
    _prefill_call("pa_prefill_sinks", False, out, q, k_pool, v_pool, None, None, block_tables, context_lens, q_start_loc,
                  scale, max_chunk_len, window, n_sinks, splits, workspace, stream)


def pa_prefill_fp8_block(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, q_start_loc, scale: float,
                         max_chunk_len: int, window: int = -1, n_sinks: int = 0, splits: int = 0, workspace=None,
                         stream=None) -> None:
    """pa_prefill_paged_ex (or, with window >= 0, pa_prefill_sinks) over an E4M3
    cache with a scale per block and head."""
    _prefill_call("pa_prefill_fp8_block", True, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                  q_start_loc, scale, max_chunk_len, window, n_sinks, splits, workspace, stream)


def pa_prefill_score_mod(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale: float,
                         max_chunk_len: int, softcap: float = 0.0, alibi_slopes=None, prefix_lens=None, window: int = -1,
                         n_sinks: int = 0, k_scale=None, v_scale=None, splits: int = 0, workspace=None,
                         stream=None) -> None:
    """Chunked prefill with the reshaped scores of pa_decode_score_mod. prefix_lens
    (int32 [n_seqs]): keys before it are visible to earlier rows of the sequence
    too. Caches as pa_decode_score_mod; workspace: prefill_workspace."""
    n_seqs = context_lens.numel()
    if q_start_loc.numel() != n_seqs + 1:
        raise ValueError("q_start_loc must have n_seqs + 1 entries")
    dev, data, tables, sizes, num_blocks = _attention_args(out, q, k_pool, v_pool, k_scale, v_scale,
                                                           k_scale is not None and v_scale is not None, block_tables,
                                                           context_lens, n_seqs)
    prefix = None
    if prefix_lens is not None:
        if prefix_lens.numel() != n_seqs:
            raise ValueError("prefix_lens must have n_seqs entries")
        prefix = _at(prefix_lens, "prefix_lens", _Types.i32, dev)
    longest, window, n_sinks, splits = _ints(max_chunk_len, window, n_sinks, splits)
    _call("pa_prefill_score_mod", dev, stream, *data, *tables, _at(q_start_loc, "q_start_loc", _Types.i32, dev),
          float(scale), float(softcap), None if alibi_slopes is None else _head_slopes(alibi_slopes, sizes[0], dev), prefix,
          *sizes, longest, num_blocks, window, n_sinks, splits, *_workspace(workspace, dev))


def pa_compact_blocks(k_pool, v_pool, block_tables, keep, keep_start_loc, k_scale=None, v_scale=None, stream=None) -> None:
    """Moves the tokens of each sequence that stay to its first positions, in
    place: position j becomes what position keep[keep_start_loc[s] + j] was.
    keep: int32 [n_kept], ascending in each sequence, or [n_kv_heads][n_kept];
    keep_start_loc: int32 [n_seqs + 1]. bf16 or E4M3 pools; k_scale and v_scale
    (fp32 [num_blocks][n_kv_heads]) when E4M3 pools have a scale per block and
    head. BlockManager.compact_batch gives the tables and frees the blocks."""
    dev = _device(k_pool, "k_pool")
    T = _Types
    num_blocks, n_kv_heads, block_size, head_dim = pool_shape = k_pool.shape
    n_seqs, max_blocks = block_tables.shape
    bits = k_pool.element_size()
    if v_pool.shape != pool_shape or v_pool.element_size() != bits:
        raise ValueError("k_pool and v_pool must have one shape and element size")
    lists = keep.shape
    if len(lists) != 1 and (len(lists) != 2 or lists[0] != n_kv_heads):
        raise ValueError("keep must be [n_kept] or [n_kv_heads][n_kept]")
    if keep_start_loc.numel() != n_seqs + 1:
        raise ValueError("keep_start_loc must have n_seqs + 1 entries")
    ks = vs = None
    if k_scale is not None and v_scale is not None:
        ns = num_blocks * n_kv_heads
        if k_scale.numel() != ns or v_scale.numel() != ns:
            raise ValueError(f"k_scale and v_scale need {ns} entries")
        ks, vs = _at(k_scale, "k_scale", T.f32, dev), _at(v_scale, "v_scale", T.f32, dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale go together")
    kinds = T.e4m3 if ks is not None else T.movable
    _call("pa_compact_blocks", dev, stream, _at(k_pool, "k_pool", kinds, dev), _at(v_pool, "v_pool", kinds, dev), ks, vs,
          _at(block_tables, "block_tables", T.i32, dev), _at(keep, "keep", T.i32, dev) if lists[-1] else None,
          _at(keep_start_loc, "keep_start_loc", T.i32, dev), n_kv_heads if len(lists) == 2 else 1, lists[-1], n_kv_heads,
          head_dim, block_size, bits, n_seqs, max_blocks, num_blocks)


def pa_copy_blocks_fp8_block(k_pool, v_pool, k_scale, v_scale, block_mapping, stream=None) -> None:
    """pa_copy_blocks of an E4M3 cache with a scale per block and head: the
    blocks' rows of k_scale and v_scale [num_blocks][n_kv_heads] are copied too."""
    dev = _device(k_pool, "k_pool")
    T = _Types
    num_blocks, n_kv_heads, block_size, head_dim = k_pool.shape
    if v_pool.shape != k_pool.shape or k_scale.numel() != num_blocks * n_kv_heads or v_scale.numel() != k_scale.numel():
        raise ValueError("k_pool and v_pool must have one shape, the scales num_blocks * n_kv_heads entries")
    n_pairs = block_mapping.shape[0] if block_mapping.numel() else 0
    _call("pa_copy_blocks_fp8_block", dev, stream, _at(k_pool, "k_pool", T.e4m3, dev), _at(v_pool, "v_pool", T.e4m3, dev),
          _at(k_scale, "k_scale", T.f32, dev), _at(v_scale, "v_scale", T.f32, dev),
          _at(block_mapping, "block_mapping", T.i64, dev) if n_pairs else None, n_pairs, n_kv_heads, head_dim,
          block_size, num_blocks)


def pa_get_device_error() -> int:
    """Reads and clears the device error word (a PA_DEVERR_* mask)."""
    v = C.c_int(0)
    check("pa_get_device_error", load().pa_get_device_error(C.byref(v)))
    return v.value


class BlockManager:
    """Host block manager (free list, refcounts, fork, copy-on-write) in the
    library; builds block tables, slots and copy pairs."""

    def __init__(self, num_blocks: int, block_size: int = 16):
        self._lib = load()
        self._h = self._lib.pa_bm_create(num_blocks, block_size)
        if not self._h:
            raise ValueError("pa_bm_create failed")
        self.num_blocks = num_blocks
        self.block_size = block_size

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._lib.pa_bm_destroy(h)
            self._h = None

    def add_seq(self, seq_id: int) -> None:
        check("pa_bm_add_seq", self._lib.pa_bm_add_seq(self._h, seq_id))

    def append_tokens(self, seq_id: int, n: int) -> Tuple[List[int], List[Tuple[int, int]]]:
        slots = (C.c_int64 * max(n, 1))()
        pairs = (C.c_int64 * 2)()
        ncow = C.c_int(0)
        check("pa_bm_append_tokens", self._lib.pa_bm_append_tokens(
            self._h, seq_id, n, slots, pairs, 1, C.byref(ncow)))
        cow = [(pairs[0], pairs[1])] if ncow.value else []
        return list(slots)[:n], cow

    def make_private(self, seq_id: int, logical_block: int) -> List[Tuple[int, int]]:
        pair = (C.c_int64 * 2)()
        n = C.c_int(0)
        check("pa_bm_make_private", self._lib.pa_bm_make_private(
            self._h, seq_id, logical_block, pair, C.byref(n)))
        return [(pair[0], pair[1])] if n.value else []

    def fork(self, parent: int, child: int) -> None:
        check("pa_bm_fork", self._lib.pa_bm_fork(self._h, parent, child))

    def free_seq(self, seq_id: int) -> None:
        check("pa_bm_free_seq", self._lib.pa_bm_free_seq(self._h, seq_id))

    def _swap(self, fn: str, seq_id: int) -> List[int]:
        n = C.c_int(0)
        st = getattr(self._lib, fn)(self._h, seq_id, None, 0, C.byref(n))
        if st == _capi.PA_OK:
            return []
        if st != _capi.PA_ERR_CAPACITY:
            check(fn, st)
        buf = (C.c_int32 * n.value)()
        check(fn, getattr(self._lib, fn)(self._h, seq_id, buf, n.value, C.byref(n)))
        return list(buf)[:n.value]

    def swap_out(self, seq_id: int) -> List[int]:
        """Releases the sequence's private tail; returns its block ids (copy
        their contents to host memory before anything reuses them)."""
        return self._swap("pa_bm_swap_out", seq_id)

    def swap_in(self, seq_id: int) -> List[int]:
        """Re-allocates a swapped sequence's tail; returns the new block ids
        (copy the contents back into them)."""
        return self._swap("pa_bm_swap_in", seq_id)

    def cache_blocks(self, seq_id: int, tokens: Sequence[int]) -> int:
        """Registers the sequence's full blocks in the prefix cache; returns
        how many entries were added."""
        arr = (C.c_int32 * max(len(tokens), 1))(*tokens)
        n = C.c_int(0)
        check("pa_bm_cache_blocks", self._lib.pa_bm_cache_blocks(self._h, seq_id, arr, len(tokens), C.byref(n)))
        return n.value

    def add_seq_cached(self, seq_id: int, tokens: Sequence[int]) -> int:
        """Starts a sequence on the longest cached prefix of tokens; returns
        the number of tokens it already holds."""
        arr = (C.c_int32 * max(len(tokens), 1))(*tokens)
        n = C.c_int64(0)
        check("pa_bm_add_seq_cached", self._lib.pa_bm_add_seq_cached(self._h, seq_id, arr, len(tokens),
                                                                      C.byref(n)))
        return n.value

    def num_cached(self) -> int:
        return self._lib.pa_bm_num_cached(self._h)

    def release_before(self, seq_id: int, first_pos: int) -> int:
        """Drops the blocks wholly before logical position first_pos (sliding
        window); their table entries become -1. Returns how many were dropped."""
        n = C.c_int(0)
        check("pa_bm_release_before", self._lib.pa_bm_release_before(self._h, seq_id, first_pos, C.byref(n)))
        return n.value

    def release_between(self, seq_id: int, from_pos: int, to_pos: int) -> int:
        """Drops the blocks that lie wholly in [from_pos, to_pos), as
        release_before does (a window whose sinks, positions below from_pos,
        stay). Returns how many were dropped."""
        n = C.c_int(0)
        check("pa_bm_release_between", self._lib.pa_bm_release_between(self._h, seq_id, from_pos, to_pos, C.byref(n)))
        return n.value

    def compact(self, seq_id: int, n_tokens: int, first_moved: int = 0) -> Tuple[List[int], List[Tuple[int, int]]]:
        """Shortens the sequence to n_tokens, for pa_compact_blocks: returns the
        block table that call needs (the old one, with shared blocks that it
        writes replaced by private ones) and the copy pairs of those blocks
        (pa_copy_blocks first). Positions below first_moved stay where they are;
        the blocks behind the kept tokens are released: launch the copies and the
        compaction before anything that writes blocks handed out later, the next
        compact's copies among them (compact_batch: several sequences at once)."""
        n_pairs, n_table = C.c_int(0), C.c_int(0)
        st = self._lib.pa_bm_compact(self._h, seq_id, n_tokens, first_moved, None, 0, C.byref(n_pairs), None, 0,
                                     C.byref(n_table))
        if st == _capi.PA_OK:
            return [], []
        if st != _capi.PA_ERR_CAPACITY:
            check("pa_bm_compact", st)
        pairs = (C.c_int64 * (2 * max(n_pairs.value, 1)))()
        table = (C.c_int32 * max(n_table.value, 1))()
        check("pa_bm_compact", self._lib.pa_bm_compact(self._h, seq_id, n_tokens, first_moved, pairs, n_pairs.value,
                                                       C.byref(n_pairs), table, n_table.value, C.byref(n_table)))
        return list(table)[:n_table.value], [(pairs[2 * i], pairs[2 * i + 1]) for i in range(n_pairs.value)]

    def compact_batch(self, seq_ids: Sequence[int], n_tokens: Sequence[int], first_moved: Optional[Sequence[int]] = None):
        """compact for sequences that one pa_compact_blocks moves together: (tables
        int32 [n][longest] as a numpy array, -1 behind a sequence's blocks, and the
        copy pairs of all of them, for one pa_copy_blocks)."""
        import numpy as np
        n = len(seq_ids)
        if len(n_tokens) != n or (first_moved is not None and len(first_moved) != n):
            raise ValueError("seq_ids, n_tokens and first_moved must have one length")
        p64 = C.POINTER(C.c_int64)
        ids, lens, firsts = (np.array(x, dtype=np.int64) for x in (seq_ids, n_tokens, [0] * n if first_moved is None else first_moved))
        n_pairs, n_blocks = C.c_int(0), C.c_int(0)

        def call(pairs, tables):
            return self._lib.pa_bm_compact_batch(
                self._h, ids.ctypes.data_as(p64), lens.ctypes.data_as(p64), firsts.ctypes.data_as(p64), n,
                pairs.ctypes.data_as(p64), len(pairs), C.byref(n_pairs), tables.ctypes.data_as(C.POINTER(C.c_int32)),
                tables.shape[1], C.byref(n_blocks))

        pairs, tables = np.empty((0, 2), np.int64), np.empty((n, 0), np.int32)
        st = call(pairs, tables)
        if st == _capi.PA_ERR_CAPACITY:
            pairs, tables = np.empty((n_pairs.value, 2), np.int64), np.empty((n, n_blocks.value), np.int32)
            st = call(pairs, tables)
        check("pa_bm_compact_batch", st)
        return tables, [(int(a), int(b)) for a, b in pairs]

    def block_table(self, seq_id: int) -> List[int]:
        n = C.c_int(0)
        st = self._lib.pa_bm_block_table(self._h, seq_id, None, 0, C.byref(n))
        if st not in (_capi.PA_OK, _capi.PA_ERR_CAPACITY):
            check("pa_bm_block_table", st)
        buf = (C.c_int32 * max(n.value, 1))()
        check("pa_bm_block_table", self._lib.pa_bm_block_table(self._h, seq_id, buf, n.value,
                                                               C.byref(n)))
        return list(buf)[:n.value]

    def seq_len(self, seq_id: int) -> int:
        v = self._lib.pa_bm_seq_len(self._h, seq_id)
        if v < 0:
            check("pa_bm_seq_len", int(v))
        return int(v)

    def num_free(self) -> int:
        return int(self._lib.pa_bm_num_free(self._h))

    def refcount(self, block_id: int) -> int:
        v = self._lib.pa_bm_refcount(self._h, block_id)
        if v < 0:
            check("pa_bm_refcount", v)
        return int(v)

    def build_batch(self, seq_ids: Sequence[int], max_blocks: int):
        """(tables int32 [n][max_blocks], context_lens int32 [n]) as numpy arrays."""
        import numpy as np
        n = len(seq_ids)
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        tabs = np.empty((n, max_blocks), dtype=np.int32)
        lens = np.empty((n,), dtype=np.int32)
        check("pa_bm_build_batch", self._lib.pa_bm_build_batch(
            self._h, ids.ctypes.data_as(C.POINTER(C.c_int64)), n, max_blocks,
            tabs.ctypes.data_as(C.POINTER(C.c_int32)), lens.ctypes.data_as(C.POINTER(C.c_int32))))
        return tabs, lens
