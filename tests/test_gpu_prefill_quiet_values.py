"""Windowed prefill of a bf16 cache whose values are small, or differ from block
to block, against fp64.

Tolerance: a weight as in the other tests of this call (2^-11 + 2^-12); V is
staged as fp16, scaled by a power of two for every 32 keys so that it is off by
at most 2^-17 of their largest magnitude (down to magnitudes of 2^-64). The
bound is in units of each sequence's largest |V|, not of 1.
"""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.sinks import dense_kv, paged_prefill
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._serving import Cache, assert_close
from tests.test_gpu_sinks_prefill import WEIGHT, pk, run, start_loc  # noqa: F401 (pk: a fixture)
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

CTX = [1, 17, 130, 300, 700]
CHUNK = [1, 3, 130, 65, 40]


def scale_values(c, factor):
    """V times `factor` (fp32, broadcast over [nb][Hk][16][D])."""
    v = bf16_bits_to_f64(c.v).astype(np.float32) * np.broadcast_to(np.asarray(factor, np.float32), c.v.shape)
    bits = f32_to_bf16_bits(v)
    c.v = np.where((c.v & 0x7FFF) > 0x7F80, c.v, bits).astype(np.uint16)


def check(pk, c, H, D, splits, weight=WEIGHT + 2.0 ** -17):
    c.scale = D ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(H + D).standard_normal((sum(CHUNK), H, D)).astype(np.float32))
    loc = start_loc(CHUNK)
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, loc, c.scale, c.window, c.n_sinks)
    got = run(pk, c, q, CHUNK, splits)
    for b, n in enumerate(CTX):
        vm = np.nanmax(np.abs(dense_kv(c.v, None, c.tables[b], n)))
        assert_close(got[loc[b]:loc[b + 1]], ref[loc[b]:loc[b + 1]], weight, vm, f"sequence {b}, |V| up to {vm}")
    check_device_error(0)


@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("window,sinks", [(127, 5), (2 ** 30, 0)])
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("e", [-6, -12, -20, -60, 12])
def test_values_of_any_magnitude(pk, D, H, Hk, window, sinks, splits, e):
    c = Cache(D + e, "bf16", CTX, Hk, D, window if window < 2 ** 30 else -1, sinks, CHUNK)
    c.window = window
    scale_values(c, 2.0 ** e)
    check(pk, c, H, D, splits)


@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 8, 1)])
@pytest.mark.parametrize("splits", [0, 1])
def test_sequences_and_blocks_of_different_magnitudes(pk, D, H, Hk, splits):
    """Every sequence another magnitude, and every block up to 2^10 apart from the next."""
    c = Cache(D, "bf16", CTX, Hk, D, 100, 20, CHUNK)
    f = np.exp2(np.random.default_rng(1).integers(-10, 1, (c.nb, Hk, 1, 1)).astype(np.float64))
    for b, e in enumerate([-30, 3, -12, -18, -5]):
        f[c.tables[b][c.tables[b] >= 0]] *= 2.0 ** e
    scale_values(c, f)
    check(pk, c, H, D, splits)


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_a_quiet_value_with_all_the_weight(pk, splits):
    """One key, 2^-14 of the others' magnitude, takes nearly all of the softmax: the output is its
    value, to its own rounding, in a block of its kind and besides to 2^-17 of the 32 keys'."""
    D, H, Hk = 128, 4, 1
    c = Cache(1, "bf16", CTX, Hk, D, 100, 16, CHUNK)
    f = np.ones((c.nb, 1, 1, 1))
    for b, n in enumerate(CTX):
        f[c.tables[b, 0]] = 2.0 ** -14
        c.k[c.tables[b, 0], :, 0] = f32_to_bf16_bits(np.full((Hk, D), 4.0, np.float32))
    scale_values(c, f)
    c.scale = D ** -0.5
    q = f32_to_bf16_bits(np.abs(np.random.default_rng(3).standard_normal((sum(CHUNK), H, D))).astype(np.float32) + 1)
    loc = start_loc(CHUNK)
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, loc, c.scale, 100, 16)
    # scores of about 80 against about +-20: the other weights are below 2^-60
    vm = max(float(np.abs(dense_kv(c.v, None, c.tables[b], 1)).max()) for b in range(len(CTX)))
    most = max(float(np.nanmax(np.abs(dense_kv(c.v, None, c.tables[b], n)))) for b, n in enumerate(CTX))
    got = bf16_bits_to_f64(run(pk, c, q, CHUNK, splits))
    assert np.isfinite(got).all() and (np.abs(ref) <= vm).all()
    assert (np.abs(got - ref) <= 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(ref) + 2 * WEIGHT * vm + 2.0 ** -17 * most).all()
    check_device_error(0)


@pytest.mark.parametrize("splits", [0, 1])
def test_zero_values(pk, splits):
    """Whole blocks of zeros beside others; and nothing but zeros."""
    for share in (0.5, 1.0):
        c = Cache(2, "bf16", CTX, 2, 64, 90, 7, CHUNK)
        scale_values(c, (np.random.default_rng(4).random((c.nb, 2, 1, 1)) >= share) * 2.0 ** -9)
        c.scale = 0.125
        q = f32_to_bf16_bits(np.random.default_rng(5).standard_normal((sum(CHUNK), 4, 64)).astype(np.float32))
        ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, start_loc(CHUNK), c.scale, 90, 7)
        vm = np.nanmax(np.abs(ref)) if share < 1 else 0.0
        assert_close(run(pk, c, q, CHUNK, splits), ref, WEIGHT + 2.0 ** -17, 4 * 2.0 ** -9 + vm if share < 1 else 0.0)
        check_device_error(0)


def test_prefill_and_decode_agree_on_quiet_values(pk):
    """The last row of a chunk and the decode at the same position, V of magnitude 2^-14."""
    torch = torch_cuda()
    c = Cache(6, "bf16", CTX, 2, 128, 60, 4, CHUNK)
    scale_values(c, 2.0 ** -14)
    c.scale = 128 ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(7).standard_normal((sum(CHUNK), 8, 128)).astype(np.float32))
    last = start_loc(CHUNK)[1:] - 1
    a = bf16_bits_to_f64(run(pk, c, q, CHUNK, 0)[last])
    qd = dev(q[last])
    out = torch.zeros_like(qd)
    pk.pa_decode_sinks(out, qd, dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), c.scale, max(CTX), 60, 4,
                       workspace=pk.decode_workspace(qd, max(CTX)))
    b = bf16_bits_to_f64(host_bits(out))
    vm = 2.0 ** -14 * 5
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) * (1 + 2.0 ** -7) + 4 * (WEIGHT + 2.0 ** -17) * vm).all()
    check_device_error(0)
