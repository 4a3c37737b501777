"""Attention under a sliding window with sinks, fp64, over any of the caches.

The query at position p attends to t <= p with t >= p - window, or t < n_sinks
(window < 0: every t <= p). "KV Cache Explained Like You're an LLM Engineer",
section "Sliding Window Attention" gives the window; the sinks are the
sequence's first tokens, kept visible besides.
"""
from __future__ import annotations

import numpy as np

from .bf16 import bf16_bits_to_f64
from .fp8 import e4m3_to_f64

BS = 16


def dense_kv(pool, scale, table_row, n):
    """fp64 [n][n_kv_heads][D] of a sequence's first n tokens. scale: None (bf16
    bits), [n_kv_heads], or [num_blocks][n_kv_heads]. Table entries of -1 give
    NaN rows."""
    blocks = np.asarray(table_row)[:(n + BS - 1) // BS]
    ids = np.maximum(blocks, 0)
    tile = np.asarray(pool)[ids]                                    # [nb][Hk][16][D]
    x = bf16_bits_to_f64(tile) if scale is None else e4m3_to_f64(tile)
    if scale is not None:
        s = np.asarray(scale, np.float64)
        x = x * (s[None, :, None, None] if s.ndim == 1 else s[ids][:, :, None, None])
    x[blocks < 0] = np.nan
    return np.moveaxis(x, 1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def attend_rows(q, positions, k, v, scale, window=-1, n_sinks=0):
    """q bf16 bits [L][H][D] at `positions`; k, v fp64 [n][Hk][D]. fp64 [L][H][D]."""
    q = bf16_bits_to_f64(q)
    L, H, D = q.shape
    g = H // k.shape[1]
    out = np.zeros((L, H, D))
    t = np.arange(len(k))
    for i in range(L):
        p = int(positions[i])
        see = t <= p
        if window >= 0:
            see &= (t >= p - window) | (t < n_sinks)
        kk, vv = k[see], v[see]
        for h in range(k.shape[1]):
            s = q[i, h * g:(h + 1) * g] @ kk[:, h].T * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            out[i, h * g:(h + 1) * g] = (w @ vv[:, h]) / w.sum(-1, keepdims=True)
    return out


def paged_decode(q, k_pool, v_pool, tables, ctx, scale, window=-1, n_sinks=0, k_scale=None, v_scale=None):
    out = np.zeros(np.asarray(q).shape)
    for b, n in enumerate(ctx):
        n = int(n)
        if n > 0:
            k, v = dense_kv(k_pool, k_scale, tables[b], n), dense_kv(v_pool, v_scale, tables[b], n)
            out[b] = attend_rows(np.asarray(q)[b:b + 1], [n - 1], k, v, scale, window, n_sinks)[0]
    return out


def paged_prefill(q, k_pool, v_pool, tables, ctx, q_start_loc, scale, window=-1, n_sinks=0, k_scale=None, v_scale=None):
    out = np.zeros(np.asarray(q).shape)
    for b, n in enumerate(ctx):
        a, e = int(q_start_loc[b]), int(q_start_loc[b + 1])
        if e > a:
            n = int(n)
            k, v = dense_kv(k_pool, k_scale, tables[b], n), dense_kv(v_pool, v_scale, tables[b], n)
            out[a:e] = attend_rows(np.asarray(q)[a:e], np.arange(n - (e - a), n), k, v, scale, window, n_sinks)
    return out
