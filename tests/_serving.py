"""Caches and tolerances shared by the tests of attention under windows with
sinks and over block-scaled E4M3 caches (not a test module)."""
import numpy as np

from oracle.fp8 import f64_to_e4m3
from workloads import f32_to_bf16_bits

BS = 16


def blocks_seen(n, first_query, window, n_sinks):
    """Logical blocks of n tokens that hold a position some query from
    first_query on sees."""
    t = np.arange(n)
    lo = max(0, first_query - window) if window >= 0 else 0
    see = (t >= lo) | (t < n_sinks)
    return np.unique(t[see] // BS)


class Cache:
    """Paged K and V of sequences of the given lengths, kind "bf16", "head" or
    "block" (E4M3 with scales per head, per block and head). Everything that no
    query sees is NaN, its table entries -1."""

    def __init__(self, seed, kind, ctx, Hk, D, window=-1, n_sinks=0, chunk=None, spread=1.0, kmag=1.0):
        rng = np.random.default_rng(seed)
        self.kind, self.ctx, self.window, self.n_sinks = kind, np.asarray(ctx, np.int32), window, n_sinks
        chunk = chunk if chunk is not None else [1] * len(ctx)
        seen = [blocks_seen(n, n - c, window, n_sinks) if n > 0 else np.zeros(0, int) for n, c in zip(ctx, chunk)]
        nb = max(2, int(sum(len(s) for s in seen) * 1.25) + 1)
        ids = rng.permutation(nb)
        self.tables = np.full((len(ctx), max(1, max((n + BS - 1) // BS for n in ctx))), -1, np.int32)
        self.nb = nb
        shape = (nb, Hk, BS, D)
        k = rng.standard_normal(shape).astype(np.float32) * kmag
        v = rng.standard_normal(shape).astype(np.float32)
        self.k_scale = self.v_scale = None
        if kind == "bf16":
            self.k, self.v, nan = f32_to_bf16_bits(k), f32_to_bf16_bits(v), 0x7FC0
        else:
            nan = 0x7F
            if kind == "head":
                self.k_scale, self.v_scale = (np.exp2(rng.uniform(-8, -6, Hk)).astype(np.float32) for _ in range(2))
                sk, sv = self.k_scale[None, :, None, None], self.v_scale[None, :, None, None]
            else:  # powers of two, as the cache write makes them; V's magnitudes differ from block to block
                e = rng.uniform(-spread, spread, (2, nb, Hk, 1, 1))
                v = (v * np.exp2(e[1])).astype(np.float32)
                sk, sv = (np.exp2(np.ceil(np.log2(np.abs(x).max((2, 3), keepdims=True) / 448))).astype(np.float32)
                          for x in (k, v))
                self.k_scale, self.v_scale = sk[:, :, 0, 0].copy(), sv[:, :, 0, 0].copy()
            self.k, self.v = f64_to_e4m3(k / sk), f64_to_e4m3(v / sv)
        used = np.zeros((nb, BS), bool)
        at = 0
        for b, s in enumerate(seen):
            self.tables[b, s] = ids[at:at + len(s)]
            lo = max(0, ctx[b] - chunk[b] - window) if window >= 0 else 0
            for logical, phys in zip(s, ids[at:at + len(s)]):
                pos = logical * BS + np.arange(BS)
                used[phys] = (pos < ctx[b]) & ((pos >= lo) | (pos < n_sinks))
            at += len(s)
        self.k[np.broadcast_to(~used[:, None, :, None], shape)] = nan
        self.v[np.broadcast_to(~used[:, None, :, None], shape)] = nan
        if kind == "block":  # scales of blocks that nothing reads
            free = ~used.any(1)
            self.k_scale[free] = self.v_scale[free] = np.nan

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)


def assert_close(got_bits, ref, weight, vmax, what=""):
    """Against fp64. `weight` bounds the relative error of a softmax weight,
    vmax the magnitude of V: an output is a mean of V, so a relative error e of
    every weight moves it by at most 2 e vmax; the output's own rounding to bf16
    is 2^-8 |ref|."""
    got = (np.asarray(got_bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + 2 * weight * vmax
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} out of tolerance, worst {(err / np.maximum(bound, 1e-30)).max()}"
