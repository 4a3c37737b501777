"""Rotary rotation and block-scaled E4M3 cache write, oracle side.

* Rotation: each pair (x, y) of dims turns by its token's angle,
  x' = x cos - y sin, y' = y cos + x sin; pairs are (i, i + r/2), or
  (2i, 2i + 1) when interleaved, i < r/2. ``rotate_f64`` is the definition;
  ``rotate_f32`` takes the same steps in fp32, each product and sum rounded to
  nearest, which is what the library promises bit for bit.
* Block-scaled E4M3 cache ("Inference serving: the KV-cache machine", section
  "What insiders know": fp8 KV with scale factors per head "or finer"): one
  scale per (block, KV head), the smallest power of two 2^e, -32 <= e <= 32,
  with max |x| <= 448 * 2^e over the block's tokens, never lowered while the
  block fills; when it grows, the codes already there are encoded again.
"""
from __future__ import annotations

import numpy as np

from .bf16 import bf16_bits_to_f64
from .fp8 import e4m3_to_f64, f64_to_e4m3

BS = 16


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _rotate(x, cos_sin, positions, interleaved, dtype):
    """x [T][heads][D] of `dtype`; cos_sin [max_position][rot]."""
    rot = cos_sin.shape[1]
    a, b = _pairs(rot, interleaved)
    row = cos_sin[np.asarray(positions)].astype(dtype)
    c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
    y = x.astype(dtype).copy()
    xa, xb = x[..., a].astype(dtype), x[..., b].astype(dtype)
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


def rotate_f64(bits, cos_sin, positions, interleaved=False):
    return _rotate(bf16_bits_to_f64(bits), cos_sin, positions, interleaved, np.float64)


def rotate_f32(bits, cos_sin, positions, interleaved=False):
    return _rotate(bf16_bits_to_f64(bits).astype(np.float32), cos_sin, positions, interleaved, np.float32)


def power_scale(amax: float) -> float:
    """The smallest 2^e, -32 <= e <= 32, with amax <= 448 * 2^e."""
    e = -32
    while e < 32 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def block_scaled_write(x, pool8, scales, slots):
    """x fp32 [T][Hk][D] (K already rotated); pool8 uint8 [nb][Hk][16][D],
    scales fp32 [nb][Hk]. Tokens with slot < 0 are skipped. The tokens of one
    block are next to each other in slots. Returns new (pool8, scales)."""
    pool, sc = np.array(pool8), np.array(scales)
    slots = np.asarray(slots)
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] % BS != 0:
            n += 1
        blk, off = int(slots[t]) // BS, int(slots[t]) % BS
        for h in range(pool.shape[1]):
            a = np.abs(x[t:t + n, h].astype(np.float64))
            a = a[np.isfinite(a)]
            need = power_scale(float(a.max()) if a.size else 0.0)
            old = float(sc[blk, h])
            new = need if off == 0 else max(old, need)
            if off != 0 and new != old:
                keep = np.ones(BS, bool)
                keep[off:off + n] = False
                pool[blk, h, keep] = f64_to_e4m3(e4m3_to_f64(pool[blk, h, keep]) * (old / new))
            pool[blk, h, off:off + n] = f64_to_e4m3(x[t:t + n, h].astype(np.float64) / new)
            sc[blk, h] = np.float32(new)
        t += n
    return pool, sc
