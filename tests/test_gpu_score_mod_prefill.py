"""Chunked prefill with capped scores, distance biases and prefixes, bf16 and
block-scaled E4M3, against fp64. What no row of a chunk sees is NaN or has table
entry -1. Tolerance: tests/_score_mod.py, a weight rounded to fp16 (2^-11); V of a bf16
cache is staged within 2^-17 of the largest of its rows."""
import numpy as np
import pytest

from oracle.score_mod import paged_prefill
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._score_mod import compare, queries, slopes_of
from tests._serving import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def start_loc(chunk):
    return np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)


def run(pk, c, q, chunk, scale, cap=0.0, slopes=None, prefix=None, splits=0, max_chunk=None, stream=None, out=None):
    torch = torch_cuda()
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0) if out is None else out
    max_chunk = max(chunk) if max_chunk is None else max_chunk
    ws = pk.prefill_workspace(qd, len(chunk), c.k.shape[1], max_chunk, splits)
    sc = dict(k_scale=dev(c.k_scale), v_scale=dev(c.v_scale)) if c.kind == "block" else {}
    pk.pa_prefill_score_mod(out, qd, dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), dev(start_loc(chunk)), scale, max_chunk,
                            softcap=cap, alibi_slopes=None if slopes is None else dev(slopes),
                            prefix_lens=None if prefix is None else dev(np.asarray(prefix, np.int32)), window=c.window,
                            n_sinks=c.n_sinks, splits=splits, workspace=ws, stream=stream, **sc)
    torch.cuda.synchronize()
    return host_bits(out)


def check(pk, c, H, D, chunk, cap=0.0, alibi=False, prefix=None, splits=0, spread=4.0, scale=None, slopes=None):
    scale = D ** -0.5 if scale is None else scale
    q = queries(H + D, sum(chunk), H, D, spread)
    slopes = slopes_of(H) if alibi and slopes is None else slopes
    loc = start_loc(chunk)
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, loc, scale, cap, slopes, prefix, c.window, c.n_sinks, c.k_scale,
                        c.v_scale)
    got = run(pk, c, q, chunk, scale, cap, slopes, prefix, splits)
    rows = [slice(int(a), int(b)) for a, b in zip(loc[:-1], loc[1:])]
    floor = 2.0 ** -17 * 8 if c.kind == "bf16" else 0.0  # normal V: no magnitude above 8
    compare(got, ref, q, c, rows, D, scale, min(cap, 400.0), 2.0 ** -11, floor,
            f"{c.kind} D={D} H={H} cap={cap} alibi={alibi} splits={splits}")
    check_device_error(0)


CTX = [1, 17, 130, 300, 513, 900, 64, 0]
CHUNK = [1, 3, 130, 65, 200, 33, 0, 0]
SHAPES = [(128, 8, 2), (64, 8, 8), (128, 8, 1), (64, 6, 3)]


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", SHAPES)
@pytest.mark.parametrize("cap,alibi", [(50.0, False), (0.0, True), (5.0, True), (0.0, False), (1000.0, False)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_scores(pk, kind, D, H, Hk, cap, alibi, splits):
    c = Cache(D + H, kind, CTX, Hk, D, chunk=CHUNK)
    check(pk, c, H, D, CHUNK, cap, alibi, splits=splits)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", SHAPES)
@pytest.mark.parametrize("cap,alibi,window,sinks,prefix", [(30.0, False, -1, 0, None), (0.0, True, 130, 5, None),
                                                            (10.0, True, -1, 0, [1, 17, 130, 300, 400, 10 ** 6, 0, 0]),
                                                            (300.0, False, 60, 0, [0, 0, 64, 250, 513, 880, 0, 0])])
def test_wide_tables_are_planned(pk, kind, D, H, Hk, cap, alibi, window, sinks, prefix):
    """Tables that could hold long contexts: pairs are listed and cut by the plan
    (short ones run as the grid gives them, in the other tests)."""
    c = Cache(D + H, kind, CTX, Hk, D, window, sinks, CHUNK)
    c.tables = np.pad(c.tables, ((0, 0), (0, 100)), constant_values=-1)
    check(pk, c, H, D, CHUNK, cap, alibi, prefix, 0)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (5, 4), (127, 16), (128, 129), (100, 5), (400, 300), (5000, 4)])
def test_under_windows_with_sinks(pk, kind, D, H, Hk, window, sinks):
    c = Cache(window + sinks + D + H, kind, CTX, Hk, D, window, sinks, CHUNK)
    check(pk, c, H, D, CHUNK, 20.0, True)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", SHAPES)
@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 0), (60, 5), (300, 0)])
@pytest.mark.parametrize("splits", [0, 2])
def test_prefixes(pk, kind, D, H, Hk, window, sinks, splits):
    """Prefixes of none, inside the chunk, as long as the context, longer, negative,
    and before the chunk."""
    ctx, chunk = [300, 300, 129, 257, 40, 500], [300, 200, 129, 256, 40, 33]
    prefix = [0, 271, 129, 10 ** 6, -3, 400]
    c = Cache(window + D + H, kind, ctx, Hk, D, window, sinks, chunk)
    check(pk, c, H, D, chunk, 30.0, splits == 2, prefix, splits)


@pytest.mark.parametrize("kind,D,H,Hk", [("bf16", 128, 4, 2), ("block", 128, 4, 1), ("block", 64, 2, 2)])
@pytest.mark.parametrize("cap", [0.01, 1.0, 128.0, 129.0, 1e4, 1e30])
@pytest.mark.parametrize("spread", [0.01, 30.0])
def test_caps_far_below_and_above_the_scores(pk, kind, D, H, Hk, cap, spread):
    check(pk, Cache(3, kind, [200, 31], Hk, D, chunk=[150, 31]), H, D, [150, 31], cap, spread=spread)


@pytest.mark.parametrize("kind,D,H,Hk", [("bf16", 64, 4, 4), ("bf16", 128, 8, 1), ("block", 128, 4, 1)])
def test_steep_zero_and_negative_slopes(pk, kind, D, H, Hk):
    c = Cache(4, kind, [700, 90], Hk, D, chunk=[140, 90])
    for slopes in ([8.0] * H, [0.0] * H, [-0.5] * H, list(np.linspace(-1, 3, H))):
        check(pk, c, H, D, [140, 90], slopes=np.array(slopes, np.float32), spread=1.0, prefix=[650, 0])


@pytest.mark.parametrize("scale", [0.0, -0.0884])
def test_zero_and_negative_softmax_scales(pk, scale):
    for kind, D in (("bf16", 128), ("block", 128), ("bf16", 64), ("block", 64)):
        check(pk, Cache(4, kind, [300, 90], 2, D, 100, 5, [70, 90]), 4, D, [70, 90], 30.0, True, scale=scale)


def test_many_segments_per_cta(pk):
    """More query-tile pairs than SMs: the persistent CTAs run several segments."""
    chunk = [129, 257, 64, 300, 1, 500]
    for kind, window, sinks, prefix in (("bf16", 200, 4, None), ("block", -1, 0, [0, 200, 900, 0, 5, 640]), ("bf16", -1, 0, None)):
        c = Cache(3, kind, [700, 257, 900, 400, 1000, 650], 16, 64, window, sinks, chunk)
        check(pk, c, 16, 64, chunk, 40.0, kind == "bf16", prefix)


def test_rows_behind_the_last_sequence_are_left(pk):
    torch = torch_cuda()
    c = Cache(7, "bf16", [64, 20], 2, 128, chunk=[30, 20])
    q = queries(1, 90, 4, 128)
    out = torch.full((90, 4, 128), 0x1234, dtype=torch.int16, device="cuda")
    got = run(pk, c, q, [30, 20], 0.1, 20.0, out=out)
    assert (got[50:] == 0x1234).all() and not (got[:50] == 0x1234).all()
    check_device_error(0)


def test_bounds_are_flagged_and_the_sequence_left_out(pk):
    torch = torch_cuda()
    for kind in ("bf16", "block"):
        c = Cache(8, kind, [300, 40], 2, 128, chunk=[280, 40])
        q = queries(2, 320, 16, 128)
        out = torch.full((320, 16, 128), 0x1234, dtype=torch.int16, device="cuda")
        got = run(pk, c, q, [280, 40], 0.1, 20.0, max_chunk=64, out=out)     # the first chunk is longer
        assert (got[:280] == 0x1234).all() and not (got[280:] == 0x1234).any(axis=(1, 2)).all()
        check_device_error(16)
        c.ctx = np.array([300, 39], np.int32)                                # the second one's is not in the cache
        got = run(pk, c, q, [280, 40], 0.1, 20.0, out=out.fill_(0x1234))
        assert (got[280:] == 0x1234).all()
        check_device_error(16)


def test_another_stream_and_a_captured_graph(pk):
    torch = torch_cuda()
    chunk = [200, 33]
    for kind in ("bf16", "block"):
        c = Cache(11, kind, [300, 50], 2, 128, chunk=chunk)
        q = queries(4, 233, 8, 128)
        want = run(pk, c, q, chunk, 0.1, 20.0, slopes_of(8), [250, 0])
        side = torch.cuda.Stream()
        assert np.array_equal(run(pk, c, q, chunk, 0.1, 20.0, slopes_of(8), [250, 0], stream=side), want)
        qd = dev(q)
        out = torch.zeros_like(qd)
        ws = pk.prefill_workspace(qd, 2, 2, 200)
        t = [dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), dev(start_loc(chunk))]
        more = dict(alibi_slopes=dev(slopes_of(8)), prefix_lens=dev(np.array([250, 0], np.int32)), workspace=ws)
        if kind == "block":
            more.update(k_scale=dev(c.k_scale), v_scale=dev(c.v_scale))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pk.pa_prefill_score_mod(out, qd, *t, 0.1, 200, softcap=20.0, **more)
        for _ in range(2):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(host_bits(out), want)
    check_device_error(0)


def test_a_long_capped_window(pk):
    """257 rows behind 20,000 tokens, window 4,096, no sinks; and all of 9,000 under
    biases. Rows sampled by a chunk of its own."""
    for kind, window, n in (("bf16", 4096, 20000), ("block", -1, 9000), ("bf16", -1, 9000)):
        c = Cache(13, kind, [n], 1, 128, window, 0, [257])
        check(pk, c, 4, 128, [257], 30.0, window < 0)


@pytest.mark.parametrize("scale,cap", [(1e8, 1.0), (1e-8, 100.0), (1e30, 50.0)])
def test_scales_far_from_the_cap(pk, scale, cap):
    """Scores of zero, whatever multiplies them: a row is the mean of V up to it."""
    for kind, D in (("bf16", 128), ("block", 128), ("bf16", 64)):
        c = Cache(14, kind, [200], 2, D, chunk=[150])
        q = np.zeros((150, 4, D), np.uint16)
        ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, start_loc([150]), 1.0, 0.0, None, None, -1, 0, c.k_scale, c.v_scale)
        compare(run(pk, c, q, [150], scale, cap), ref, q, c, [slice(0, 150)], D, 0.0, cap, 2.0 ** -11, 2.0 ** -17 * 8)
    check_device_error(0)


def test_refusals(pk):
    torch = torch_cuda()
    c = Cache(12, "block", [40], 2, 64, chunk=[20])
    q = dev(queries(5, 20, 4, 64))
    out = torch.zeros_like(q)
    k, v, ks, vs, tab, ctx, loc = (dev(x) for x in (c.k, c.v, c.k_scale, c.v_scale, c.tables, c.ctx, start_loc([20])))
    ws = pk.prefill_workspace(q, 1, 2, 20)

    def call(**over):
        a = dict(softcap=10.0, k_scale=ks, v_scale=vs, workspace=ws)
        a.update(over)
        pk.pa_prefill_score_mod(out, q, k, v, tab, ctx, loc, 0.1, 20, **a)

    call()
    s, p = dev(slopes_of(4)), dev(np.zeros(1, np.int32))
    for over, kind in ((dict(alibi_slopes=s[:3]), ValueError), (dict(alibi_slopes=s.double()), TypeError),
                       (dict(prefix_lens=p.long()), TypeError), (dict(prefix_lens=p.expand(2)), ValueError),
                       (dict(prefix_lens=p.cpu()), ValueError), (dict(v_scale=None), ValueError),
                       (dict(softcap=-1.0), pk.PagedKVError), (dict(workspace=None), pk.PagedKVError),
                       (dict(window=-2), pk.PagedKVError), (dict(splits=65), pk.PagedKVError),
                       (dict(k_scale=None, v_scale=None), TypeError)):
        with pytest.raises(kind):
            call(**over)
    check_device_error(0)
