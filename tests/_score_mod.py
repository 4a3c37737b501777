"""Inputs and tolerances shared by the tests of reshaped scores (not a test module)."""
import numpy as np

from oracle.bf16 import bf16_bits_to_f64
from oracle.sinks import dense_kv
from tests._serving import assert_close
from workloads import f32_to_bf16_bits


def slopes_of(H):
    return np.exp2(-8.0 * np.arange(1, H + 1) / H).astype(np.float32)


def queries(seed, n, H, D, spread=4.0):
    return f32_to_bf16_bits((np.random.default_rng(seed).standard_normal((n, H, D)) * spread).astype(np.float32))


def weight_error(D, largest, cap, rounding):
    """Relative error of a softmax weight. `largest`: of sum_i |q_i k_i| * scale.
    D products are accumulated in fp32 in any order: a score is off by D 2^-24 of
    that at most. tanh is off by a few 2^-23 of the cap (2^-20 taken). The score in
    base 2, its scale, bias and reference cost four roundings of values up to
    1.45 * (largest + 40) (a key 40 below the maximum has no weight left). One of e
    in the score moves a weight by e (1 + e). `rounding`: of the weight itself."""
    e = D * 2.0 ** -24 * largest + cap * 2.0 ** -20 + 4 * 2.0 ** -24 * 1.45 * (largest + 40)
    return rounding + e * (1 + e)


def largest_sum(q, c, rows, D, scale):
    """The largest sum_i |q_i k_i| * |scale| of a query and a key of its sequence.
    rows[b]: the sequence's rows of q."""
    qa, most = np.abs(bf16_bits_to_f64(q)), 0.0
    for b, n in enumerate(c.ctx):
        if n > 0 and rows[b].stop > rows[b].start:
            k = np.abs(dense_kv(c.k, c.k_scale, c.tables[b], int(n)))
            for h in range(k.shape[1]):
                g = qa.shape[1] // k.shape[1]
                s = qa[rows[b], h * g:(h + 1) * g].reshape(-1, D) @ np.nan_to_num(k[:, h]).T
                most = max(most, float(s.max()))
    return most * abs(scale)


def compare(got, ref, q, c, rows, D, scale, cap, rounding, floor=0.0, what=""):
    """`floor`: an absolute error of V's elements."""
    vmax = max([np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[b], int(n))))
                for b, n in enumerate(c.ctx) if n > 0 and rows[b].stop > rows[b].start], default=1.0)
    weight = weight_error(D, largest_sum(q, c, rows, D, scale), cap, rounding)
    assert_close(got, ref, weight + floor / vmax, vmax, what)
