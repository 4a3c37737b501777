"""Chunked prefill under a sliding window with sinks (bf16) and over a
block-scaled E4M3 cache, against fp64.

What no row of a chunk sees is NaN (K, V, the scales of unread blocks) or has
table entry -1. Tolerance as for the decode: a weight is off by its score's
error (at most 2.2e-4 < 2^-12 of it for unit normals: fp32 accumulation over D
terms) and by the fp16 rounding, 2^-11; V is exact in fp16 for an E4M3 cache,
and for bf16 too above 2^-6, below which it is off by at most 2^-17 absolute.
"""
import numpy as np
import pytest

from oracle.sinks import dense_kv, paged_prefill
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._serving import Cache, assert_close
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -11 + 2.0 ** -12


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def start_loc(chunk):
    return np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)


def call(pk, c, qd, chunk, splits, out, ws, tensors, max_chunk=None):
    max_chunk = max(chunk) if max_chunk is None else max_chunk
    k, v, ks, vs, tab, ctx, loc = tensors
    if c.kind == "block":
        pk.pa_prefill_fp8_block(out, qd, k, v, ks, vs, tab, ctx, loc, c.scale, max_chunk, window=c.window,
                                n_sinks=c.n_sinks, splits=splits, workspace=ws)
    else:
        pk.pa_prefill_sinks(out, qd, k, v, tab, ctx, loc, c.scale, max_chunk, c.window, c.n_sinks, splits=splits,
                            workspace=ws)


def tensors_of(c, chunk):
    sc = [None if s is None else dev(s) for s in (c.k_scale, c.v_scale)]
    return [dev(c.k), dev(c.v), *sc, dev(c.tables), dev(c.ctx), dev(start_loc(chunk))]


def run(pk, c, q, chunk, splits, max_chunk=None):
    torch = torch_cuda()
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    hk = c.k.shape[1]
    ws = pk.prefill_workspace(qd, len(chunk), hk, max(chunk) if max_chunk is None else max_chunk, splits)
    call(pk, c, qd, chunk, splits, out, ws, tensors_of(c, chunk), max_chunk)
    torch.cuda.synchronize()
    return host_bits(out)


def check(pk, c, H, D, chunk, splits, what="", scale=None):
    c.scale = D ** -0.5 if scale is None else scale
    q = f32_to_bf16_bits(np.random.default_rng(H + D).standard_normal((sum(chunk), H, D)).astype(np.float32))
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, start_loc(chunk), c.scale, c.window, c.n_sinks, **c.scales())
    vm = max(np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[b], int(n)))) for b, n in enumerate(c.ctx) if chunk[b] > 0)
    assert_close(run(pk, c, q, chunk, splits), ref, WEIGHT + 2.0 ** -16 / vm, vm, what)
    check_device_error(0)


CTX = [1, 17, 130, 300, 513, 900, 64, 0]
CHUNK = [1, 3, 130, 65, 200, 33, 0, 0]


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 8, 8), (128, 8, 1), (64, 6, 3), (128, 2, 2), (64, 8, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (5, 4), (127, 16), (128, 129), (100, 5), (400, 300), (5000, 4)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_window_with_sinks(pk, kind, D, H, Hk, window, sinks, splits):
    c = Cache(window + sinks + D + H, kind, CTX, Hk, D, window, sinks, CHUNK)
    check(pk, c, H, D, CHUNK, splits, f"{kind} D={D} H={H} window={window} sinks={sinks} splits={splits}")


@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 8, 8), (128, 8, 1), (64, 2, 1), (128, 3, 3)])
@pytest.mark.parametrize("splits", [0, 1, 2, 7])
@pytest.mark.parametrize("spread", [0.0, 4.0])
def test_block_scaled_full_context(pk, D, H, Hk, splits, spread):
    c = Cache(D + H, "block", CTX, Hk, D, chunk=CHUNK, spread=spread)
    check(pk, c, H, D, CHUNK, splits, f"D={D} H={H} splits={splits}")


def test_many_segments_per_cta(pk):
    """More query-tile pairs than SMs: the persistent CTAs run several segments,
    barrier phases going on from one to the next."""
    chunk = [129, 257, 64, 300, 1, 500]
    for kind, window, sinks in (("bf16", 200, 4), ("block", -1, 0), ("block", 77, 130)):
        c = Cache(3, kind, [700, 257, 900, 400, 1000, 650], 16, 64, window, sinks, chunk)
        check(pk, c, 16, 64, chunk, 0, f"{kind}")


@pytest.mark.parametrize("scale", [0.0, -0.0884])
def test_zero_and_negative_softmax_scales(pk, scale):
    for kind, D in (("bf16", 128), ("block", 128), ("bf16", 64), ("block", 64)):
        c = Cache(4, kind, [300, 90], 2, D, 100, 5, [70, 90])
        check(pk, c, 4, D, [70, 90], 0, kind, scale)


def test_extreme_block_scales(pk):
    """K scales that dominate or erase a block's scores, V scales 2^-20 to 2^20
    apart; the bound is in units of the loudest V."""
    chunk = [40, 7]
    for D, H, Hk in [(128, 4, 2), (64, 4, 4)]:
        c = Cache(9, "block", [400, 33], Hk, D, chunk=chunk)
        rng = np.random.default_rng(1)
        c.v_scale = np.exp2(rng.integers(-20, 21, (c.nb, Hk))).astype(np.float32)
        c.k_scale = (c.k_scale * np.exp2(rng.integers(-12, 1, (c.nb, Hk)))).astype(np.float32)
        check(pk, c, H, D, chunk, 0)


def test_rows_as_wide_windows_equal_full_prefill(pk):
    """A window past the context is no window: the same bits as pa_prefill_paged_ex,
    unsplit (splits = 0 cuts the key ranges at other places, and where a row's
    partial sums are joined decides their fp32 roundings)."""
    torch = torch_cuda()
    chunk = [100, 33]
    c = Cache(5, "bf16", [300, 33], 2, 128, chunk=chunk)
    c.window, c.n_sinks, c.scale = 2 ** 31 - 1, 2 ** 31 - 1, 128 ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(2).standard_normal((133, 8, 128)).astype(np.float32))
    got = run(pk, c, q, chunk, 1)
    qd = dev(q)
    out = torch.zeros_like(qd)
    t = tensors_of(c, chunk)
    pk.pa_prefill_paged_ex(out, qd, t[0], t[1], t[4], t[5], t[6], c.scale, 100, splits=1)
    assert np.array_equal(got, host_bits(out))
    check_device_error(0)


def test_a_long_window(pk):
    """A 257-token chunk behind 20,000 tokens, window 4,096, 4 sinks, both caches;
    rows sampled."""
    n, L, D, H, Hk = 20257, 257, 128, 8, 2
    for kind in ("bf16", "block"):
        c = Cache(6, kind, [n], Hk, D, 4096, 4, [L])
        c.scale = D ** -0.5
        q = f32_to_bf16_bits(np.random.default_rng(8).standard_normal((L, H, D)).astype(np.float32))
        from oracle.sinks import attend_rows
        k, v = dense_kv(c.k, c.k_scale, c.tables[0], n), dense_kv(c.v, c.v_scale, c.tables[0], n)
        rows = [0, 1, 63, 64, 100, 255, 256]
        ref = attend_rows(q[rows], [n - L + r for r in rows], k, v, c.scale, 4096, 4)
        vm = float(np.nanmax(np.abs(v)))
        for splits in (0, 1, 5):
            assert_close(run(pk, c, q, [L], splits)[rows], ref, WEIGHT + 2.0 ** -16 / vm, vm, f"{kind} {splits}")
    check_device_error(0)


@pytest.mark.parametrize("D,H,Hk", [(128, 4, 1), (64, 2, 2), (128, 8, 1), (64, 1, 1)])
def test_short_chunks_behind_long_contexts(pk, D, H, Hk):
    """One to forty rows behind up to 9,000 tokens: many pieces of few rows, joined
    by row, and of many, joined by column; twice, with the same bits."""
    for chunk, ctx in (([1], [9000]), ([3, 1], [5000, 200]), ([40], [9000]), ([1, 17], [3000, 6001])):
        for kind, window, sinks in (("bf16", 2 ** 30, 0), ("block", -1, 0), ("bf16", 4000, 5)):
            c = Cache(9, kind, ctx, Hk, D, window if window < 2 ** 30 else -1, sinks, chunk)
            c.window = window
            check(pk, c, H, D, chunk, 0, f"{kind} {chunk}")
            q = f32_to_bf16_bits(np.random.default_rng(1).standard_normal((sum(chunk), H, D)).astype(np.float32))
            assert np.array_equal(run(pk, c, q, chunk, 0), run(pk, c, q, chunk, 0))


def test_rows_behind_the_last_chunk_and_a_loose_bound(pk):
    """q and out longer than the chunks, max_chunk_len above every chunk: the
    rows behind the last one stay as they were."""
    torch = torch_cuda()
    for kind in ("bf16", "block"):
        chunk = [20, 5]
        c = Cache(7, kind, [100, 40], 2, 64, 30, 3, chunk)
        c.scale = 0.125
        q = f32_to_bf16_bits(np.random.default_rng(3).standard_normal((60, 4, 64)).astype(np.float32))
        for splits in (0, 1, 4):
            got = run(pk, c, q, chunk, splits, max_chunk=300)
            assert (got[25:] == 0x7FC0).all()
            ref = paged_prefill(q[:25], c.k, c.v, c.tables, c.ctx, start_loc(chunk), c.scale, 30, 3, **c.scales())
            assert_close(got[:25], ref, WEIGHT + 2.0 ** -16, 8.0)
    check_device_error(0)


def test_flags(pk):
    torch = torch_cuda()
    chunk = [20, 5]
    c = Cache(8, "block", [100, 40], 2, 64, 30, 3, chunk)
    c.scale = 0.125
    q = f32_to_bf16_bits(np.random.default_rng(3).standard_normal((25, 4, 64)).astype(np.float32))
    good = c.tables.copy()
    c.tables[0, 6] = c.nb            # past the pool, in the window of every row
    run(pk, c, q, chunk, 0)
    check_device_error(1)
    c.tables = good
    c.ctx[1] = 4                     # a chunk longer than its context: that sequence is left out
    got = run(pk, c, q, chunk, 0)
    check_device_error(16)
    assert (got[20:] == 0x7FC0).all() and (got[:20] != 0x7FC0).any()


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_sequences_beyond_the_calls_bounds_are_left_out(pk, kind, splits):
    """A context that its table does not hold, a chunk beyond max_chunk_len:
    flagged, its rows left as they were, the others' unchanged."""
    chunk = [20, 5, 70]
    c = Cache(8, kind, [300, 40, 100], 2, 64, 120, 3, chunk)
    c.scale = 0.125
    q = f32_to_bf16_bits(np.random.default_rng(3).standard_normal((95, 16, 64)).astype(np.float32))
    want = run(pk, c, q, chunk, splits)
    check_device_error(0)
    tables, c.tables = c.tables, c.tables[:, :18].copy()  # of 19 blocks
    got = run(pk, c, q, chunk, splits)
    check_device_error(16)
    assert (got[:20] == 0x7FC0).all() and np.array_equal(got[20:], want[20:])
    c.tables = tables
    got = run(pk, c, q, chunk, splits, max_chunk=64)  # pairs of 32 rows: the third chunk has 70
    check_device_error(16)
    assert (got[25:] == 0x7FC0).all() and np.array_equal(got[:25], want[:25])


def test_captured_and_replayed_and_two_streams(pk):
    torch = torch_cuda()
    chunk = [90, 200, 33]
    for kind in ("bf16", "block"):
        c = Cache(16, kind, [700, 200, 1300], 4, 128, 200, 5, chunk)
        c.scale = 128 ** -0.5
        q = f32_to_bf16_bits(np.random.default_rng(4).standard_normal((323, 16, 128)).astype(np.float32))
        want = run(pk, c, q, chunk, 0)
        qd, t = dev(q), tensors_of(c, chunk)
        outs = [torch.zeros_like(qd) for _ in range(2)]
        spaces = [pk.prefill_workspace(qd, 3, 4, 200) for _ in range(2)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(pk, c, qd, chunk, 0, outs[0], spaces[0], t)
        for _ in range(2):
            outs[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(host_bits(outs[0]), want)
        outs[0].zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(10):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    call(pk, c, qd, chunk, 0, outs[i], spaces[i], t)
        torch.cuda.synchronize()
        assert all(np.array_equal(host_bits(o), want) for o in outs)
    check_device_error(0)


def test_numbers_beyond_32_bits_are_refused(pk):
    torch = torch_cuda()
    chunk = [4]
    c = Cache(17, "block", [100], 2, 128, chunk=chunk)
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    k, v, ks, vs, tab, ctx, loc = tensors_of(c, chunk)
    one = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (2 ** 32, 2 ** 31, -2 ** 31 - 1, 2 ** 32 + 5):
        for over in (dict(window=bad), dict(window=5, n_sinks=bad), dict(splits=bad)):
            with pytest.raises(ValueError):
                pk.pa_prefill_fp8_block(out, q, k, v, ks, vs, tab, ctx, loc, 0.1, 4, **{"splits": 1, **over})
        for over in (dict(window=bad), dict(window=5, n_sinks=bad), dict(partition_tokens=bad)):
            with pytest.raises(ValueError):
                pk.pa_decode_fp8_block(torch.empty_like(one), one, k, v, ks, vs, tab, ctx, 0.1, 100, **over)
    check_device_error(0)


def test_refusals(pk):
    torch = torch_cuda()
    chunk = [4]
    c = Cache(17, "block", [100], 2, 128, chunk=chunk)
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    k, v, ks, vs, tab, ctx, loc = tensors_of(c, chunk)
    with pytest.raises(ValueError):
        pk.pa_prefill_fp8_block(out, q, k, v, ks[:1], vs[:1], tab, ctx, loc, 0.1, 4, splits=1)
    with pytest.raises(ValueError):
        pk.pa_prefill_fp8_block(out, q, k, v, None, vs, tab, ctx, loc, 0.1, 4, splits=1)
    with pytest.raises(ValueError):
        pk.pa_prefill_sinks(out, q, k, v, tab, ctx, loc[:1], 0.1, 4, 5, 1, splits=1)
    with pytest.raises(TypeError):
        pk.pa_prefill_sinks(out, q, k, v, tab, ctx, loc, 0.1, 4, 5, 1, splits=1)
    with pytest.raises(pk.PagedKVError):
        pk.pa_prefill_fp8_block(out, q, k, v, ks, vs, tab, ctx, loc, 0.1, 4, window=-2, splits=1)
    with pytest.raises(pk.PagedKVError):   # the balanced mode needs its workspace
        pk.pa_prefill_fp8_block(out, q, k, v, ks, vs, tab, ctx, loc, 0.1, 4)
