"""Decode under a sliding window with sinks (bf16, E4M3 per head, E4M3 per
block) and decode over a block-scaled cache, against fp64.

Positions that no query sees hold NaN (in K and V, and in the scales of unread
blocks) and blocks without a visible position have table entry -1, so a read of
one shows as a flag or a NaN.

Tolerance (``assert_close``): a weight's relative error is that of its score,
ln 2 times at most D 2^-23 scale sum |q k| (fp32 accumulation, a truncating
tensor core counted as 2^-23 an add): 128 * 2^-23 * 0.0884 * 160 = 2.2e-4 <
2^-12 for the sums of |q k| (about 82, below 160) of unit normals, 2^-22 for
exp2, and with an E4M3 cache at head_dim 128 2^-11 for the fp16 weight.
"""
import numpy as np
import pytest

from oracle.sinks import dense_kv, paged_decode
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._serving import Cache, assert_close
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

CTX = [1, 2, 16, 17, 40, 129, 300, 513, 1000, 0]


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def weight(kind):
    return 2.0 ** -12 + (0 if kind == "bf16" else 2.0 ** -11)


def vmax(c):
    return max(np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[b], int(n)))) for b, n in enumerate(c.ctx) if n > 0)


def run(pk, c, q, pt=0, stream=None):
    torch = torch_cuda()
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    max_ctx = int(c.ctx.max())
    ws = pk.decode_workspace(qd, max_ctx, pt)
    sc = [None if s is None else dev(s) for s in (c.k_scale, c.v_scale)]
    a = (out, qd, dev(c.k), dev(c.v))
    b = (dev(c.tables), dev(c.ctx), c.scale, max_ctx)
    if c.kind == "block":
        pk.pa_decode_fp8_block(*a, *sc, *b, window=c.window, n_sinks=c.n_sinks, workspace=ws, partition_tokens=pt)
    else:
        pk.pa_decode_sinks(*a, *b, c.window, c.n_sinks, *sc, workspace=ws, partition_tokens=pt)
    torch.cuda.synchronize()
    return host_bits(out)


def check(pk, c, H, D, seed, pt=0, what="", scale=None):
    c.scale = D ** -0.5 if scale is None else scale
    q = f32_to_bf16_bits(np.random.default_rng(seed).standard_normal((len(c.ctx), H, D)).astype(np.float32))
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, c.scale, c.window, c.n_sinks, **c.scales())
    got = run(pk, c, q, pt)
    assert_close(got, ref, weight(c.kind), vmax(c), what)
    check_device_error(0)
    return got


@pytest.mark.parametrize("kind", ["bf16", "head", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 32, 8), (64, 8, 8), (128, 16, 2), (64, 6, 3), (128, 2, 1), (64, 8, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (1, 4), (15, 16), (16, 17), (100, 4), (30, 150), (600, 33),
                                          (250, 600), (5000, 4)])
@pytest.mark.parametrize("pt", [0, 64])
def test_window_with_sinks(pk, kind, D, H, Hk, window, sinks, pt):
    c = Cache(window + sinks + D + H, kind, CTX, Hk, D, window, sinks)
    check(pk, c, H, D, 3, pt, f"{kind} D={D} H={H} window={window} sinks={sinks}")


@pytest.mark.parametrize("D,H,Hk", [(128, 32, 8), (64, 8, 8), (128, 16, 2), (64, 6, 3), (128, 3, 3), (64, 8, 1)])
@pytest.mark.parametrize("pt", [0, 64, 192])
@pytest.mark.parametrize("spread", [0.0, 4.0])
def test_block_scaled_full_context(pk, D, H, Hk, pt, spread):
    c = Cache(D + H + pt, "block", CTX + [2500], Hk, D, spread=spread)
    check(pk, c, H, D, 5, pt, f"D={D} H={H} pt={pt} spread={spread}")


@pytest.mark.parametrize("D,H,Hk", [(128, 8, 8), (64, 8, 8), (128, 8, 1)])
def test_extreme_block_scales(pk, D, H, Hk):
    """K scales that dominate or erase a block's scores and V scales 2^-20 to
    2^20 apart. The quiet blocks' values vanish beside the loud ones', so the
    bound is in units of the loudest V, as derived."""
    c = Cache(9, "block", [400, 33], Hk, D)
    rng = np.random.default_rng(1)
    nb = c.nb
    c.v_scale = np.exp2(rng.integers(-20, 21, (nb, Hk))).astype(np.float32)
    c.k_scale = (c.k_scale * np.exp2(rng.integers(-12, 1, (nb, Hk)))).astype(np.float32)
    check(pk, c, H, D, 6)


@pytest.mark.parametrize("scale", [0.0, -0.0884])
def test_zero_and_negative_softmax_scales(pk, scale):
    for kind in ("bf16", "head", "block"):
        for D, H, Hk in [(128, 8, 2), (64, 8, 8), (128, 8, 1)]:
            check(pk, Cache(4, kind, [300, 90, 1], Hk, D, 100, 5), H, D, 8, 64, kind, scale)


def test_float8_pools_are_taken_as_they_are(pk):
    torch = torch_cuda()
    c = Cache(18, "block", [100, 700], 2, 128)
    c.scale = 128 ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(2).standard_normal((2, 8, 128)).astype(np.float32))
    want = run(pk, c, q)
    k, v = (dev(x).view(torch.float8_e4m3fn) for x in (c.k, c.v))
    qd = dev(q).view(torch.bfloat16)
    out = torch.empty_like(qd)
    pk.pa_decode_fp8_block(out, qd, k, v, dev(c.k_scale), dev(c.v_scale), dev(c.tables), dev(c.ctx), c.scale, 700,
                           workspace=pk.decode_workspace(qd, 700))
    assert np.array_equal(host_bits(out), want)


def test_uniform_scales_equal_head_scales_bit_for_bit(pk):
    """With one K scale per head and V scales of 1 the block-scaled kernel makes
    the per-head kernel's steps: a multiply-add with e = 0 is its multiply."""
    for D, H, Hk in [(128, 8, 2), (64, 8, 8)]:
        c = Cache(11, "head", [5, 300, 1500], Hk, D)
        c.k_scale[:] = 2.0 ** -7
        c.v_scale[:] = 1.0
        c.scale = D ** -0.5
        c.window, c.n_sinks = 5000, 0
        q = f32_to_bf16_bits(np.random.default_rng(2).standard_normal((3, H, D)).astype(np.float32))
        a = run(pk, c, q)
        c.kind, c.window = "block", -1
        c.k_scale, c.v_scale = (np.tile(s, (c.nb, 1)) for s in (c.k_scale, c.v_scale))
        assert np.array_equal(a, run(pk, c, q))
    check_device_error(0)


def test_scales_outside_the_range_are_clamped(pk):
    c = Cache(12, "block", [200], 2, 128)
    c.scale, c.window = 128 ** -0.5, -1
    q = f32_to_bf16_bits(np.random.default_rng(2).standard_normal((1, 8, 128)).astype(np.float32))
    c.v_scale[:] = 2.0 ** 40
    a = run(pk, c, q)
    c.v_scale[:] = 2.0 ** 32
    assert np.array_equal(a, run(pk, c, q))
    c.k_scale[:] = 0.0
    a = run(pk, c, q)
    c.k_scale[:] = 2.0 ** -32
    assert np.array_equal(a, run(pk, c, q))
    check_device_error(0)


def test_no_sinks_equals_window_decode_bit_for_bit(pk):
    torch = torch_cuda()
    for D, H, Hk in [(128, 32, 8), (64, 8, 8), (128, 16, 2)]:
        c = Cache(13, "bf16", CTX, Hk, D, 100, 0)
        c.scale = D ** -0.5
        q = f32_to_bf16_bits(np.random.default_rng(2).standard_normal((len(CTX), H, D)).astype(np.float32))
        a = run(pk, c, q)
        qd = dev(q)
        out = torch.empty_like(qd)
        pk.pa_decode_window(out, qd, dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), c.scale, 1000, 100,
                            workspace=pk.decode_workspace(qd, 1000))
        assert np.array_equal(a, host_bits(out))
    check_device_error(0)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40])
def test_the_largest_windows_and_sinks(pk, window):
    c = Cache(14, "bf16", [1, 300, 1000], 8, 128)
    c.window, c.n_sinks = window, 2 ** 31 - 1
    check(pk, c, 8, 128, 7)
    c = Cache(14, "block", [1, 300, 1000], 8, 64)
    c.window, c.n_sinks = window, 2 ** 31 - 1
    check(pk, c, 8, 64, 7)


def test_long_context_and_blocks_past_2_31_elements(pk):
    """131,072 tokens in the last blocks of an E4M3 pool of more than 2^31
    elements, one query group of 8 and one head per KV head."""
    torch = torch_cuda()
    Hk, D, n = 8, 128, 131072
    nb = (1 << 31) // (Hk * 16 * D) + n // 16
    g = torch.Generator(device="cuda").manual_seed(3)
    kp, vp = (torch.randint(0, 126, (nb, Hk, 16, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    for p in (kp, vp):
        p |= torch.randint(0, 2, (nb, 1, 1, D), generator=g, device="cuda", dtype=torch.uint8) << 7
    ks = torch.full((nb, Hk), 2.0 ** -9, device="cuda")
    vs = torch.exp2(torch.randint(-12, -6, (nb, Hk), generator=g, device="cuda").float())
    tab = (nb - 1 - torch.arange(n // 16, device="cuda", dtype=torch.int32))[None].contiguous()
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    for H in (8, 64):
        q = torch.randn((1, H, D), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        out = torch.zeros_like(q)
        pk.pa_decode_fp8_block(out, q, kp, vp, ks, vs, tab, ctx, D ** -0.5, n, workspace=pk.decode_workspace(q, n))
        ids = tab[0].long()
        for h in (0, 5):
            k = (kp[ids, h].view(torch.float8_e4m3fn).double() * ks[ids, h, None, None]).view(n, D)
            v = (vp[ids, h].view(torch.float8_e4m3fn).double() * vs[ids, h, None, None]).view(n, D)
            heads = slice(h * (H // 8), (h + 1) * (H // 8))
            w = torch.softmax(q[0, heads].double() @ k.T * D ** -0.5, -1)
            ref = (w @ v).cpu().numpy()
            # sums of |q k| reach 128 * 0.875 * 1.7 * 3: the score term of the tolerance grows with them
            score = float((q[0, heads].double().abs() @ k.abs().T).max()) * D ** -0.5 * 128 * 2.0 ** -23
            assert_close(host_bits(out[0, heads]), ref, weight("block") + score, float(v.abs().max()))
    check_device_error(0)


def test_a_bad_block_id_is_flagged(pk):
    c = Cache(15, "block", [100, 200], 2, 128)
    c.scale = 128 ** -0.5
    most = vmax(c)
    c.tables[1, 3] = c.nb
    q = f32_to_bf16_bits(np.random.default_rng(2).standard_normal((2, 8, 128)).astype(np.float32))
    ref = paged_decode(q[:1], c.k, c.v, c.tables[:1], c.ctx[:1], c.scale, **c.scales())
    got = run(pk, c, q)
    check_device_error(1)
    assert_close(got[:1], ref, weight("block"), most)


def test_captured_and_replayed_and_two_streams(pk):
    torch = torch_cuda()
    c = Cache(16, "block", [700, 90, 1300], 8, 128, 200, 5)
    c.scale = 128 ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(4).standard_normal((3, 32, 128)).astype(np.float32))
    want = run(pk, c, q, 64)
    a = [dev(x) for x in (q, c.k, c.v, c.k_scale, c.v_scale, c.tables, c.ctx)]
    outs, spaces = [torch.zeros_like(a[0]) for _ in range(2)], [pk.decode_workspace(a[0], 1300, 64) for _ in range(2)]
    torch.cuda.synchronize()

    def call(i):
        pk.pa_decode_fp8_block(outs[i], *a, c.scale, 1300, window=200, n_sinks=5, workspace=spaces[i], partition_tokens=64)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(outs[0]), want)
    outs[0].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(i)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(outs[0]), want) and np.array_equal(host_bits(outs[1]), want)
    check_device_error(0)


def test_refusals(pk):
    torch = torch_cuda()
    c = Cache(17, "block", [100], 2, 128)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    k, v, ks, vs, tab, ctx = (dev(x) for x in (c.k, c.v, c.k_scale, c.v_scale, c.tables, c.ctx))
    with pytest.raises(ValueError):
        pk.pa_decode_fp8_block(out, q, k, v, None, None, tab, ctx, 0.1, 100)
    with pytest.raises(ValueError):      # per-head scales are no block scales
        pk.pa_decode_fp8_block(out, q, k, v, ks[0].contiguous(), vs[0].contiguous(), tab, ctx, 0.1, 100)
    with pytest.raises(TypeError):       # an E4M3 pool is no bf16 pool
        pk.pa_decode_sinks(out, q, k, v, tab, ctx, 0.1, 100, 10, 4)
    with pytest.raises(ValueError):
        pk.pa_decode_sinks(out, q, k, v, tab, ctx, 0.1, 100, 10, 4, k_scale=ks[0].contiguous())
    with pytest.raises(ValueError):
        pk.pa_decode_fp8_block(out.cpu(), q, k, v, ks, vs, tab, ctx, 0.1, 100)
    with pytest.raises(pk.PagedKVError):
        pk.pa_decode_fp8_block(out, q, k, v, ks, vs, tab, ctx, 0.1, 100, window=-2)
    with pytest.raises(pk.PagedKVError):
        pk.pa_decode_fp8_block(out, q, k, v, ks, vs, tab, ctx, 0.1, 100, window=5, n_sinks=-1)
