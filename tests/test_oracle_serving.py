"""Pins for the oracles of the rotated, block-scaled cache write and of windows
with sinks (CPU)."""
import numpy as np
import pytest

from oracle.attention import paged_decode as full_decode
from oracle.attention import paged_decode_window
from oracle.bf16 import bf16_bits_to_f64
from oracle.fp8 import e4m3_to_f64
from oracle.rope_cache import block_scaled_write, power_scale, rotate_f32, rotate_f64
from oracle.sinks import paged_decode, paged_prefill
from tests._serving import Cache
from workloads import f32_to_bf16_bits, make_decode_case, make_decode_case_window

torch = pytest.importorskip("torch")


def test_sinks_oracle_against_the_older_ones():
    wl = make_decode_case(1, [1, 16, 33, 100], 4, 2, 64, n_new=0)
    a = full_decode(wl.q, wl.k_pool, wl.v_pool, wl.dec_tables, wl.dec_ctx, wl.scale)
    for window, sinks in [(-1, 0), (200, 0), (0, 200), (50, 50)]:
        b = paged_decode(wl.q, wl.k_pool, wl.v_pool, wl.dec_tables, wl.dec_ctx, wl.scale, window, sinks)
        np.testing.assert_allclose(a, b, rtol=1e-11, atol=1e-12)
    wl = make_decode_case_window(2, [1, 16, 33, 100], 4, 2, 64, 20, n_new=0)
    a = paged_decode_window(wl.q, wl.k_pool, wl.v_pool, wl.dec_tables, wl.dec_ctx, wl.scale, 20)
    b = paged_decode(wl.q, wl.k_pool, wl.v_pool, wl.dec_tables, wl.dec_ctx, wl.scale, 20, 0)
    np.testing.assert_allclose(a, b, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("kind", ["bf16", "head", "block"])
def test_sinks_oracle_against_a_dense_mask(kind):
    c = Cache(3, kind, [37, 90], 2, 64, 11, 5, chunk=[9, 20])
    q = f32_to_bf16_bits(np.random.default_rng(0).standard_normal((29, 4, 64)).astype(np.float32))
    got = paged_prefill(q, c.k, c.v, c.tables, c.ctx, [0, 9, 29], 0.125, 11, 5, **c.scales())
    from oracle.sinks import dense_kv
    for a, e, b in [(0, 9, 0), (9, 29, 1)]:
        n = int(c.ctx[b])
        k, v = (torch.from_numpy(np.nan_to_num(dense_kv(p, s, c.tables[b], n))) for p, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
        i, t = torch.arange(n - (e - a), n)[:, None], torch.arange(n)[None]
        mask = (t <= i) & ((i - t <= 11) | (t < 5))
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(bf16_bits_to_f64(q[a:e])).transpose(0, 1), k.transpose(0, 1).repeat_interleave(2, 0),
            v.transpose(0, 1).repeat_interleave(2, 0), attn_mask=mask, scale=0.125).transpose(0, 1)
        np.testing.assert_allclose(got[a:e], ref.numpy(), rtol=1e-10, atol=1e-12)


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x = f32_to_bf16_bits(rng.standard_normal((5, 3, 64)).astype(np.float32))
    ang = rng.uniform(0, 6, (9, 16))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = np.array([0, 8, 3, 3, 1])
    for il in (False, True):
        y, v = rotate_f64(x, cs, pos, il), bf16_bits_to_f64(x)
        a, b = (slice(0, 32, 2), slice(1, 32, 2)) if il else (slice(0, 16), slice(16, 32))
        z = (v[..., a] + 1j * v[..., b]) * np.exp(1j * ang[pos])[:, None]
        np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-12)
        assert np.array_equal(y[..., 32:], v[..., 32:])
        np.testing.assert_allclose(rotate_f32(x, cs.astype(np.float32), pos, il), y, atol=1e-5)


def test_block_scaled_write_against_the_definition():
    assert [power_scale(a) for a in (0.0, 448.0, 448.0001, 224.0, 3e38, 1e-30)] == [2.0 ** -32, 1, 2, 0.5, 2.0 ** 32, 2.0 ** -32]
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((20, 2, 64)) * np.exp2(rng.integers(-4, 5, (20, 1, 1)))).astype(np.float32)
    pool, sc = np.full((4, 2, 16, 64), 0x7F, np.uint8), np.ones((4, 2), np.float32)
    slots = np.r_[np.arange(32, 48), -1, np.arange(16, 19)]
    p1, s1 = block_scaled_write(x, pool, sc, slots)
    assert (p1[[0, 3]] == 0x7F).all() and (s1[[0, 3]] == 1).all() and (p1[1, :, 3:] == 0x7F).all()
    for blk, rows in ((2, x[:16]), (1, x[17:])):
        want = np.moveaxis(rows.astype(np.float64), 0, 1)
        for h in range(2):
            s = float(s1[blk, h])
            assert 224 * s < np.abs(want[h]).max() <= 448 * s
            got = e4m3_to_f64(p1[blk, h, :rows.shape[0]]) * s
            assert (np.abs(got - want[h]) <= np.maximum(2.0 ** -4 * np.abs(want[h]), 2.0 ** -10 * s)).all()
    # louder tokens in a partly filled block: the others keep their values to half a subnormal step
    for gain in (64, 2 ** 14):
        p2, s2 = block_scaled_write(x[:1] * gain, p1, s1, [19])
        for h in range(2):
            was, now = (e4m3_to_f64(p[1, h, :3]) * float(s[1, h]) for p, s in ((p1, s1), (p2, s2)))
            assert s2[1, h] >= s1[1, h] and (np.abs(was - now) <= 2.0 ** -10 * s2[1, h]).all()
    assert (s2[1] > s1[1]).all()
