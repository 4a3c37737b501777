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


def read_scale(s: float) -> float:
    """A block's scale as the attention calls read it: in [2^-32, 2^32], NaN as 2^-32."""
    return 2.0 ** -32 if s != s else min(max(float(s), 2.0 ** -32), 2.0 ** 32)


def block_scaled_write(x, pool8, scales, slots):
    """x fp32 [T][Hk][D] (K already rotated); pool8 uint8 [nb][Hk][16][D],
    scales fp32 [nb][Hk]. Tokens with slot < 0 are skipped. The tokens of one
    block lie within 16 consecutive entries of slots, in any order; they share
    one new scale. A block whose first slot is among them gets it anew, any
    other keeps at least its own. Returns new (pool8, scales)."""
    pool, sc = np.array(pool8), np.array(scales)
    slots = np.asarray(slots)
    block = np.where(slots < 0, -1, slots // BS)
    for t in range(len(slots)):
        blk = int(block[t])
        if blk < 0 or (block[max(0, t - BS + 1):t] == blk).any():
            continue  # skipped, or written with an earlier token of its block
        rows = t + np.nonzero(block[t:t + BS] == blk)[0]
        off = slots[rows] % BS
        for h in range(pool.shape[1]):
            a = np.abs(x[rows, h].astype(np.float64))
            a = a[np.isfinite(a)]
            need = power_scale(float(a.max()) if a.size else 0.0)
            old = read_scale(sc[blk, h])
            least = 2.0 ** np.ceil(np.log2(old))  # of a scale from elsewhere: the next power of two
            new = np.float32(need if (off == 0).any() else max(least, need))
            if not (off == 0).any() and new != old:
                keep = np.ones(BS, bool)
                keep[off] = False
                moved = e4m3_to_f64(pool[blk, h, keep]).astype(np.float32) * (np.float32(old) / new)
                pool[blk, h, keep] = f64_to_e4m3(moved.astype(np.float64))
            pool[blk, h, off] = f64_to_e4m3((x[rows, h].astype(np.float32) / new).astype(np.float64))
            sc[blk, h] = new
    return pool, sc
