"""The fp64 definitions of reshaped scores and of compaction, on the CPU: against
loops over single keys, and the limits they must have."""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.fp8 import e4m3_to_f64, f64_to_e4m3
from oracle.score_mod import attend, compact, paged_decode, paged_prefill, reshape_scores, visible
from oracle.sinks import attend_rows
from tests._score_mod import queries, slopes_of


def kv(seed, n, Hk, D):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, Hk, D)), r.standard_normal((n, Hk, D))


@pytest.mark.parametrize("cap,alibi,prefix,window,sinks", [(0.0, False, 0, -1, 0), (5.0, False, 0, -1, 0),
                                                            (0.0, True, 0, -1, 0), (3.0, True, 9, -1, 0),
                                                            (2.0, True, 11, 3, 2), (0.0, False, 20, 0, 1)])
def test_attend_is_the_formula_key_by_key(cap, alibi, prefix, window, sinks):
    H, Hk, D, n, L = 4, 2, 16, 14, 6
    q = queries(1, L, H, D)
    k, v = kv(2, n, Hk, D)
    slopes = slopes_of(H) if alibi else None
    out = attend(q, np.arange(n - L, n), k, v, 0.25, cap, slopes, prefix, window, sinks)
    for i in range(L):
        p = n - L + i
        for h in range(H):
            total, acc = 0.0, np.zeros(D)
            for t in range(n):
                if not (t <= p or t < prefix) or (window >= 0 and t < p - window and t >= sinks):
                    continue
                s = 0.25 * float(bf16_bits_to_f64(q[i, h]) @ k[t, h // 2])
                if cap:
                    s = cap * (1 - 2 / (1 + np.exp(2 * s / cap)))
                if alibi:
                    s -= float(slopes[h]) * abs(p - t)
                total += np.exp(s)
                acc += np.exp(s) * v[t, h // 2]
            assert np.allclose(out[i, h], acc / total, rtol=1e-12, atol=1e-13)


def test_without_reshaping_it_is_the_windowed_attention():
    q = queries(3, 5, 4, 32)
    k, v = kv(4, 40, 2, 32)
    pos = np.arange(35, 40)
    for window, sinks in ((-1, 0), (7, 0), (7, 3)):
        assert np.allclose(attend(q, pos, k, v, 0.2, window=window, n_sinks=sinks), attend_rows(q, pos, k, v, 0.2, window, sinks),
                           rtol=1e-13, atol=1e-14)
    assert np.allclose(attend(q, pos, k, v, 0.2, cap=1e9), attend(q, pos, k, v, 0.2), rtol=1e-7)


def test_a_cap_bounds_scores_and_a_prefix_shows_later_keys():
    s = np.linspace(-1e4, 1e4, 101)[None]
    z = reshape_scores(s, 50.0)
    assert np.abs(z).max() <= 50.0 and (np.diff(z[0]) >= 0).all()
    t = np.arange(8)
    assert list(visible(2, t, prefix=5)) == [True] * 5 + [False] * 3
    assert list(visible(6, t, prefix=5)) == [True] * 7 + [False]
    assert list(visible(3, t, prefix=6, window=1)) == [False, False, True, True, True, True, False, False]


def test_paged_forms_gather_through_the_tables():
    rng = np.random.default_rng(5)
    from workloads import f32_to_bf16_bits
    pool = [f32_to_bf16_bits(rng.standard_normal((9, 2, 16, 16)).astype(np.float32)) for _ in range(2)]
    tables = np.array([[7, 2, 5], [1, 0, -1]], np.int32)
    ctx = np.array([37, 20], np.int32)
    dense = [[np.concatenate([bf16_bits_to_f64(p[i]) for i in row if i >= 0], 1).transpose(1, 0, 2)[:n]
              for p in pool] for row, n in zip(tables, ctx)]
    q = queries(6, 5, 4, 16)
    starts = [0, 3, 5]
    got = paged_prefill(q, *pool, tables, ctx, starts, 0.3, 20.0, slopes_of(4), [30, 0], 9, 1)
    for b in range(2):
        a, e = starts[b:b + 2]
        want = attend(q[a:e], np.arange(ctx[b] - (e - a), ctx[b]), *dense[b], 0.3, 20.0, slopes_of(4), [30, 0][b], 9, 1)
        assert np.allclose(got[a:e], want)
    last = paged_decode(q[[2, 4]], *pool, tables, ctx, 0.3, 20.0, slopes_of(4), 9, 1)
    assert np.allclose(last, got[[2, 4]])


def test_compaction_moves_what_positions_held():
    rng = np.random.default_rng(7)
    pool = rng.integers(0, 1 << 16, (8, 3, 16, 4)).astype(np.uint16)
    tables = np.array([[4, 1, 6], [0, 3, -1]], np.int32)
    keep = np.concatenate([np.sort(rng.choice(45, 20, replace=False)), np.arange(18)])
    got, _ = compact(pool, tables, keep, [0, 20, 38])
    flat = np.concatenate([pool[i] for i in tables[0]], 1)
    after = np.concatenate([got[i] for i in tables[0]], 1)
    assert np.array_equal(after[:, :20], flat[:, keep[:20]]) and np.array_equal(after[:, 20:32], flat[:, 20:32])
    for i in (0, 3, 2, 5, 7, 6):
        assert np.array_equal(got[i], pool[i])  # all of the second sequence stays


def test_compaction_takes_the_largest_scale():
    codes = np.zeros((3, 1, 16, 2), np.uint8)
    codes[0, 0, :, 0] = f64_to_e4m3(np.arange(16.0))
    codes[1, 0, :, 0] = f64_to_e4m3(np.arange(16.0) * 2)
    scale = np.array([[0.25], [4.0], [1.0]], np.float32)
    got, s = compact(codes, np.array([[0, 1]]), [0, 3, 5, 17, 18], [0, 5], scale)
    assert s[0, 0] == 4.0 and s[1, 0] == 4.0
    assert np.array_equal(e4m3_to_f64(got[0, 0, :5, 0]) * 4, [0, 0.75, 1.25, 8, 16])
    assert np.array_equal(got[1], codes[1]) and np.array_equal(got[0, 0, 5:], codes[0, 0, 5:])
