"""Decode with capped scores and distance biases, bf16 and block-scaled E4M3, against
fp64. What the query does not see is NaN or has table entry -1.

Tolerance (tests/_score_mod.py): a weight's rounding is 2^-11 where it enters the P.V
product as fp16 (E4M3 at head_dim 128), 2^-16 where it is two bf16 terms or fp32."""
import numpy as np
import pytest

from oracle.score_mod import paged_decode
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


def run(pk, c, q, scale, cap=0.0, slopes=None, partition_tokens=0, max_ctx=None, stream=None):
    torch = torch_cuda()
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    max_ctx = max(1, int(max(c.ctx))) if max_ctx is None else max_ctx
    ws = pk.decode_workspace(qd, max_ctx, partition_tokens)
    sc = dict(k_scale=dev(c.k_scale), v_scale=dev(c.v_scale)) if c.kind == "block" else {}
    tables = np.pad(c.tables, ((0, 0), (0, max(0, (max_ctx + 15) // 16 - c.tables.shape[1]))), constant_values=-1)
    pk.pa_decode_score_mod(out, qd, dev(c.k), dev(c.v), dev(tables), dev(c.ctx), scale, max_ctx, softcap=cap,
                           alibi_slopes=None if slopes is None else dev(slopes), window=c.window, n_sinks=c.n_sinks,
                           workspace=ws, partition_tokens=partition_tokens, stream=stream, **sc)
    torch.cuda.synchronize()
    return host_bits(out)


def check(pk, c, H, D, cap=0.0, alibi=False, partition_tokens=0, spread=4.0, scale=None, slopes=None, max_ctx=None):
    scale = D ** -0.5 if scale is None else scale
    q = queries(H + D, len(c.ctx), H, D, spread)
    slopes = slopes_of(H) if alibi and slopes is None else slopes
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, scale, cap, slopes, c.window, c.n_sinks, c.k_scale, c.v_scale)
    got = run(pk, c, q, scale, cap, slopes, partition_tokens, max_ctx)
    rounding = 2.0 ** -11 if c.kind == "block" and D == 128 else 2.0 ** -16
    compare(got, ref, q, c, [slice(b, b + 1) for b in range(len(c.ctx))], D, scale, cap, rounding,
            what=f"{c.kind} D={D} H={H} cap={cap} alibi={alibi}")
    check_device_error(0)


CTX = [1, 17, 130, 300, 513, 0, 16, 64]


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 8, 8), (128, 8, 1), (64, 6, 3), (128, 2, 2), (64, 8, 1), (64, 4, 1), (128, 6, 3)])
@pytest.mark.parametrize("cap,alibi", [(50.0, False), (0.0, True), (5.0, True), (0.0, False)])
@pytest.mark.parametrize("partition_tokens", [0, 64])
def test_scores(pk, kind, D, H, Hk, cap, alibi, partition_tokens):
    c = Cache(D + H, kind, CTX, Hk, D)
    check(pk, c, H, D, cap, alibi, partition_tokens)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 8, 4), (128, 8, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (5, 4), (127, 16), (100, 33), (5000, 4)])
def test_under_windows_with_sinks(pk, kind, D, H, Hk, window, sinks):
    c = Cache(window + sinks, kind, CTX, Hk, D, window, sinks)
    check(pk, c, H, D, 20.0, True, 64)


@pytest.mark.parametrize("kind,D,H,Hk", [("bf16", 128, 4, 2), ("bf16", 128, 8, 1), ("block", 128, 4, 1), ("block", 64, 2, 2)])
@pytest.mark.parametrize("cap", [0.01, 1.0, 30.0, 1e4, 1e30])
@pytest.mark.parametrize("spread", [0.01, 30.0])
def test_caps_far_below_and_above_the_scores(pk, kind, D, H, Hk, cap, spread):
    """A cap of 0.01 levels all scores, one of 1e30 leaves them."""
    c = Cache(3, kind, [200, 31], Hk, D)
    scale = D ** -0.5
    q = queries(1, 2, H, D, spread)
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, scale, cap, None, k_scale=c.k_scale, v_scale=c.v_scale)
    # tanh is exact relative to the score, too: a few 2^-23 of min(cap, score)
    compare(run(pk, c, q, scale, cap), ref, q, c, [slice(0, 1), slice(1, 2)], D, scale, min(cap, 400.0),
            2.0 ** -11 if kind == "block" and D == 128 else 2.0 ** -16, what=f"cap {cap} spread {spread}")
    check_device_error(0)


@pytest.mark.parametrize("kind,D,H,Hk", [("bf16", 64, 4, 4), ("bf16", 128, 8, 1), ("block", 128, 4, 1)])
def test_steep_zero_and_negative_slopes(pk, kind, D, H, Hk):
    c = Cache(4, kind, [700, 90], Hk, D)
    for slopes in ([8.0] * H, [0.0] * H, [-0.5] * H, list(np.linspace(-1, 3, H))):
        check(pk, c, H, D, 0.0, slopes=np.array(slopes, np.float32), partition_tokens=128, spread=1.0)


@pytest.mark.parametrize("scale", [0.0, -0.0884])
def test_zero_and_negative_softmax_scales(pk, scale):
    for kind, D in (("bf16", 128), ("block", 128), ("block", 64)):
        check(pk, Cache(4, kind, [300, 90], 2, D), 4, D, 30.0, True, scale=scale)


def test_long_contexts_are_split_and_joined(pk):
    for kind, D, H, Hk in (("bf16", 128, 4, 1), ("block", 128, 8, 1), ("bf16", 64, 8, 8)):
        c = Cache(6, kind, [20000, 9000, 1], Hk, D)
        check(pk, c, H, D, 30.0, D == 64)


def test_plain_scores_equal_the_plain_decode(pk):
    """No cap and no slopes: the attention of pa_decode_sinks, up to the order in
    which blocks are taken."""
    torch = torch_cuda()
    c = Cache(8, "bf16", CTX, 2, 128, 100, 5)
    check(pk, c, 8, 128)
    c = Cache(8, "block", [300, 17], 2, 128)
    check(pk, c, 8, 128)
    assert torch is not None


def test_a_context_beyond_its_bound_is_flagged(pk):
    for kind in ("bf16", "block"):
        c = Cache(9, kind, [100, 40], 2, 128)
        q = queries(2, 2, 4, 128)
        sc = dict(k_scale=c.k_scale, v_scale=c.v_scale)
        ref = paged_decode(q, c.k, c.v, c.tables, [64, 40], 0.1, 10.0, slopes_of(4), **sc)
        got = run(pk, c, q, 0.1, 10.0, slopes_of(4), max_ctx=64)
        compare(got, ref, q, c, [slice(0, 1), slice(1, 2)], 128, 0.1, 10.0, 2.0 ** -11)
        check_device_error(16)


def test_a_bad_block_is_skipped_and_flagged(pk):
    for kind in ("bf16", "block"):
        c = Cache(10, kind, [100], 2, 128)
        c.tables[0, 2] = c.nb
        q = queries(3, 1, 4, 128)
        got = run(pk, c, q, 0.1, 10.0)
        check_device_error(1)
        assert np.isfinite((got.astype(np.uint32) << 16).view(np.float32)).all()


def test_another_stream_and_a_captured_graph(pk):
    torch = torch_cuda()
    c = Cache(11, "bf16", [300, 50], 2, 128)
    q = queries(4, 2, 8, 128)
    want = run(pk, c, q, 0.1, 20.0, slopes_of(8), 64)
    side = torch.cuda.Stream()
    assert np.array_equal(run(pk, c, q, 0.1, 20.0, slopes_of(8), 64, stream=side), want)
    qd, out = dev(q), None
    out = torch.zeros_like(qd)
    ws = pk.decode_workspace(qd, 300, 64)
    t = [dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), dev(slopes_of(8))]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_decode_score_mod(out, qd, *t[:4], 0.1, 300, softcap=20.0, alibi_slopes=t[4], workspace=ws, partition_tokens=64)
    qd.zero_()
    g.replay()
    torch.cuda.synchronize()
    first = host_bits(out)
    qd.copy_(dev(q))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out), want) and not np.array_equal(first, want)
    check_device_error(0)


@pytest.mark.parametrize("scale,cap", [(1e8, 1.0), (1e-8, 100.0), (1e30, 50.0)])
def test_scales_far_from_the_cap(pk, scale, cap):
    """Scores of zero, whatever multiplies them: the mean of V."""
    for kind, D, H in (("bf16", 128, 4), ("block", 128, 4), ("bf16", 64, 2), ("bf16", 128, 2)):
        c = Cache(14, kind, [200], 2, D)
        q = np.zeros((1, H, D), np.uint16)
        ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, 1.0, 0.0, None, -1, 0, c.k_scale, c.v_scale)
        compare(run(pk, c, q, scale, cap), ref, q, c, [slice(0, 1)], D, 0.0, cap, 2.0 ** -11)
    check_device_error(0)


def test_refusals(pk):
    torch = torch_cuda()
    c = Cache(12, "block", [40], 2, 64)
    q = dev(queries(5, 1, 4, 64))
    out = torch.zeros_like(q)
    k, v, ks, vs, tab, ctx = dev(c.k), dev(c.v), dev(c.k_scale), dev(c.v_scale), dev(c.tables), dev(c.ctx)
    ok = dict(softcap=10.0, k_scale=ks, v_scale=vs)

    def call(**over):
        a = dict(ok, **over)
        pk.pa_decode_score_mod(out, q, k, v, tab, ctx, 0.1, 40, **a)

    call()
    s = dev(slopes_of(4))
    for over, kind in ((dict(alibi_slopes=s[:3]), ValueError), (dict(alibi_slopes=s.double()), TypeError),
                       (dict(alibi_slopes=s.cpu()), ValueError), (dict(v_scale=None), ValueError),
                       (dict(k_scale=ks[:1]), ValueError), (dict(softcap=-1.0), pk.PagedKVError),
                       (dict(softcap=float("nan")), pk.PagedKVError), (dict(window=-2), pk.PagedKVError),
                       (dict(window=2 ** 31), ValueError), (dict(k_scale=None, v_scale=None), TypeError)):
        with pytest.raises(kind):
            call(**over)
    check_device_error(0)
