"""Attention with reshaped scores over any of the caches, and the compaction of a
cache, in fp64.

With s = scale * (q . k), the score of key t for a query at position p is
    z = cap * tanh(s / cap) - slope[head] * |p - t|        (cap 0: s; no slopes: no bias)
and the query attends to t <= p and to t < prefix, of those, under a window >= 0,
to t >= p - window or t < n_sinks. Compaction: new position j of a sequence holds
what its position keep[j] held; in an E4M3 cache with a scale per block a block's
new scale is the largest of its new tokens' scales.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_to_f64, f64_to_e4m3
from .bf16 import bf16_bits_to_f64
from .sinks import dense_kv

BS = 16


def reshape_scores(s, cap=0.0, slopes=None, distance=None):
    """s [heads][...][keys]; distance broadcasts against s[0]."""
    z = cap * np.tanh(s / cap) if cap > 0 else np.array(s, np.float64)
    if slopes is not None:
        z = z - np.asarray(slopes, np.float64).reshape((-1,) + (1,) * (s.ndim - 1)) * distance
    return z


def visible(p, t, prefix=0, window=-1, n_sinks=0):
    """Whether a query at position p sees key t (arrays broadcast)."""
    see = (t <= p) | (t < prefix)
    if window >= 0:
        see = see & ((t >= p - window) | (t < n_sinks))
    return see


def attend(q, positions, k, v, scale, cap=0.0, slopes=None, prefix=0, window=-1, n_sinks=0):
    """q bf16 bits [L][H][D] at `positions`; k, v fp64 [n][Hk][D]. fp64 [L][H][D]."""
    q = bf16_bits_to_f64(q)
    L, H, D = q.shape
    Hk = k.shape[1]
    g = H // Hk
    p, t = np.asarray(positions)[:, None], np.arange(len(k))[None]
    see = visible(p, t, prefix, window, n_sinks)
    read = see.any(0)
    out = np.zeros((L, H, D))
    for h in range(Hk):
        kk, vv = np.where(read[:, None], k[:, h], 0.0), np.where(read[:, None], v[:, h], 0.0)
        heads = slice(h * g, (h + 1) * g)
        s = np.einsum("lgd,td->glt", q[:, heads], kk) * scale
        z = reshape_scores(s, cap, None if slopes is None else np.asarray(slopes)[heads], np.abs(p - t))
        z = np.where(see[None], z, -np.inf)
        w = np.exp(z - z.max(-1, keepdims=True))
        out[:, heads] = np.einsum("glt,td->lgd", w, vv) / w.sum(-1).T[..., None]
    return out


def paged_decode(q, k_pool, v_pool, tables, ctx, scale, cap=0.0, slopes=None, window=-1, n_sinks=0, k_scale=None,
                 v_scale=None):
    out = np.zeros(np.asarray(q).shape)
    for b, n in enumerate(ctx):
        n = int(n)
        if n > 0:
            k, v = dense_kv(k_pool, k_scale, tables[b], n), dense_kv(v_pool, v_scale, tables[b], n)
            out[b] = attend(np.asarray(q)[b:b + 1], [n - 1], k, v, scale, cap, slopes, 0, window, n_sinks)[0]
    return out


def paged_prefill(q, k_pool, v_pool, tables, ctx, q_start_loc, scale, cap=0.0, slopes=None, prefix=None, window=-1,
                  n_sinks=0, k_scale=None, v_scale=None):
    out = np.zeros(np.asarray(q).shape)
    for b, n in enumerate(ctx):
        a, e = int(q_start_loc[b]), int(q_start_loc[b + 1])
        if e > a:
            n = int(n)
            k, v = dense_kv(k_pool, k_scale, tables[b], n), dense_kv(v_pool, v_scale, tables[b], n)
            out[a:e] = attend(np.asarray(q)[a:e], np.arange(n - (e - a), n), k, v, scale, cap, slopes,
                              0 if prefix is None else int(prefix[b]), window, n_sinks)
    return out


def compact(pool, tables, keep, starts, scale=None):
    """(pool, scale) after compaction, one KV head and one sequence after the other.
    keep [n] or [Hk][n]."""
    pool = np.array(pool)
    new_scale = None if scale is None else np.array(scale, np.float32)
    keep = np.asarray(keep)
    for b in range(len(starts) - 1):
        a, e = int(starts[b]), int(starts[b + 1])
        for h in range(pool.shape[1]):
            kept = [int(x) for x in (keep[h] if keep.ndim == 2 else keep)[a:e]]
            first = next((j for j, x in enumerate(kept) if x != j), len(kept)) // BS * BS
            rows = {}
            for j in range(first, len(kept)):
                blk = int(tables[b][kept[j] // BS])
                rows[j] = (pool[blk, h, kept[j] % BS].copy(), None if scale is None else np.float32(scale[blk, h]))
            if all(x == j for j, x in enumerate(kept)):
                continue
            for j0 in range(first, len(kept), BS):
                blk = int(tables[b][j0 // BS])
                js = range(j0, min(j0 + BS, len(kept)))
                if scale is not None:
                    new = max(rows[j][1] for j in js)
                    new_scale[blk, h] = new
                for j in js:
                    x, old = rows[j]
                    if scale is not None and old != new:
                        x = f64_to_e4m3(e4m3_to_f64(x) * (np.float64(old) / np.float64(new)))
                    pool[blk, h, j % BS] = x
    return pool, new_scale
