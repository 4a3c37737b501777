"""GPU tests of the rotated cache write (bf16, E4M3 per head, E4M3 per block).

The library promises fp32 products and sums rounded one by one and one rounding
to the stored type, so outputs are compared bit for bit with numpy doing the
same steps (``oracle.rope_cache.rotate_f32``). Against the fp64 definition an
output y = a c - b s is off by at most 2^-24 (|a c| + |b s| + |y|) from the
three fp32 roundings (2^-24 each; the factor 1.001 covers their products), and
by 2^-8 |y| from the bf16 one.
"""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.fp8 import e4m3_to_f64, f64_to_e4m3
from oracle.rope_cache import block_scaled_write, rotate_f32, rotate_f64
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

SLOT, POSITION = 2, 256


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def table(max_pos, rot):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(max_pos)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Case:
    """Packed q, k, v of runs of tokens [(first slot, count)], with pools of
    known content; slots in `skip` become -1."""

    def __init__(self, seed, runs, H, Hk, D, rot, num_blocks, max_pos=1000, mag=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.Hk, self.D, self.rot, self.nb = H, Hk, D, rot, num_blocks
        self.slots = np.concatenate([np.arange(s, s + n) for s, n in runs]).astype(np.int64)
        T = len(self.slots)
        self.pos = rng.integers(0, max_pos, T).astype(np.int64)
        x = rng.standard_normal((T, (H + 2 * Hk) * D)).astype(np.float32)
        x *= np.exp2(rng.integers(-3, 4, (T, 1))).astype(np.float32) * mag
        self.qkv = f32_to_bf16_bits(x)
        self.cs = table(max_pos, rot) if rot else None
        self.rng = rng

    def parts(self):
        T, H, Hk, D = len(self.slots), self.H, self.Hk, self.D
        return (self.qkv[:, :H * D].reshape(T, H, D), self.qkv[:, H * D:(H + Hk) * D].reshape(T, Hk, D),
                self.qkv[:, (H + Hk) * D:].reshape(T, Hk, D))

    def dev_parts(self):
        T, H, Hk, D = len(self.slots), self.H, self.Hk, self.D
        x = dev(self.qkv)
        return (x[:, :H * D].view(T, H, D), x[:, H * D:(H + Hk) * D].view(T, Hk, D),
                x[:, (H + Hk) * D:].view(T, Hk, D))

    def rotated(self, x, il):
        return bf16_bits_to_f64(x).astype(np.float32) if self.cs is None else \
            rotate_f32(x, self.cs, np.clip(self.pos, 0, len(self.cs) - 1), il)


RUNS = [(5, 3), (64, 16), (80, 7), (163, 1), (176, 16), (192, 16), (208, 1)]
SHAPES = [(8, 2, 128, 128, False), (8, 2, 128, 128, True), (4, 4, 64, 64, False), (3, 1, 64, 32, True),
          (16, 2, 128, 48, False), (8, 8, 128, 16, False), (8, 2, 128, 80, True), (2, 1, 64, 0, False)]


def bf16_pools(c):
    shape = (c.nb, c.Hk, 16, c.D)
    return c.rng.integers(0, 1 << 16, shape).astype(np.uint16), c.rng.integers(0, 1 << 16, shape).astype(np.uint16)


def scatter(pool, rows, slots):
    pool = pool.copy()
    for t, s in enumerate(slots):
        if s >= 0:
            pool[s // 16, :, s % 16] = rows[t]
    return pool


def args(c):
    return (None, None) if c.cs is None else (dev(c.cs), dev(c.pos))


@pytest.mark.parametrize("H,Hk,D,rot,il", SHAPES)
@pytest.mark.parametrize("many", [False, True])
def test_bf16_bit_exact(pk, H, Hk, D, rot, il, many):
    torch = torch_cuda()
    runs = RUNS + ([(320, 16 * 200 + 9)] if many else [])
    c = Case(7 + D + rot, runs, H, Hk, D, rot, 240)
    if c.cs is not None:
        c.pos[1] = -1   # skipped: nothing of the token is written
    c.slots[4] = -1     # padding: q only
    kp0, vp0 = bf16_pools(c)
    kp, vp = dev(kp0), dev(vp0)
    q, k, v = c.dev_parts()
    out = torch.full((len(c.slots), H, D), 0x1234, dtype=torch.int16, device="cuda")
    cs, pos = args(c)
    pk.pa_rope_and_cache(out, q, k, v, kp, vp, cs, pos, dev(c.slots), interleaved=il)
    hq, hk, hv = c.parts()
    want_q = f32_to_bf16_bits(c.rotated(hq, il))
    want_k = f32_to_bf16_bits(c.rotated(hk, il))
    slots = c.slots.copy()
    if c.cs is not None:
        want_q[1] = 0x1234
        slots[1] = -1
    assert np.array_equal(host_bits(out), want_q)
    assert np.array_equal(host_bits(kp), scatter(kp0, want_k, slots))
    assert np.array_equal(host_bits(vp), scatter(vp0, hv, slots))
    check_device_error(0)


def test_against_the_definition_in_64_bits(pk):
    torch = torch_cuda()
    c = Case(3, RUNS, 8, 2, 128, 128, 16, max_pos=131072)
    q, k, v = c.dev_parts()
    kp, vp = (dev(p) for p in bf16_pools(c))
    out = torch.empty((len(c.slots), 8, 128), dtype=torch.int16, device="cuda")
    pk.pa_rope_and_cache(out, q, k, v, kp, vp, dev(c.cs), dev(c.pos), dev(c.slots))
    hq = c.parts()[0]
    ref = rotate_f64(hq, c.cs, c.pos)
    x = np.abs(bf16_bits_to_f64(hq))
    row = np.abs(c.cs[c.pos].astype(np.float64))[:, None]
    terms = np.concatenate([x[..., :64] * row[..., :64] + x[..., 64:] * row[..., 64:],
                            x[..., 64:] * row[..., :64] + x[..., :64] * row[..., 64:]], -1)
    bound = 1.001 * 2.0 ** -24 * (terms + np.abs(ref)) + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -20)
    # the bf16 rounding is of the fp32 value, itself off by the first term
    assert (np.abs(bf16_bits_to_f64(host_bits(out)) - ref) <= bound * 1.01).all()


@pytest.mark.parametrize("H,Hk,D,rot,il", SHAPES)
def test_head_scaled_bit_exact(pk, H, Hk, D, rot, il):
    c = Case(21 + D + rot, RUNS, H, Hk, D, rot, 16)
    c.slots[0] = -1
    shape = (c.nb, Hk, 16, D)
    kp0, vp0 = (c.rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
    ks, vs = (np.exp2(c.rng.uniform(-9, -3, Hk)).astype(np.float32) for _ in range(2))
    kp, vp = dev(kp0), dev(vp0)
    _, k, v = c.dev_parts()
    cs, pos = args(c)
    pk.pa_rope_and_cache(None, None, k, v, kp, vp, cs, pos, dev(c.slots), interleaved=il, k_scale=dev(ks), v_scale=dev(vs))
    _, hk, hv = c.parts()
    rk, rv = c.rotated(hk, il), bf16_bits_to_f64(hv).astype(np.float32)
    want_k = f64_to_e4m3((rk / ks[:, None]).astype(np.float64))
    want_v = f64_to_e4m3((rv / vs[:, None]).astype(np.float64))
    assert np.array_equal(kp.cpu().numpy(), scatter(kp0, want_k, c.slots))
    assert np.array_equal(vp.cpu().numpy(), scatter(vp0, want_v, c.slots))
    check_device_error(0)


def block_pools(c):
    shape = (c.nb, c.Hk, 16, c.D)
    finite = np.array([x for x in range(256) if x & 0x7F != 0x7F], np.uint8)
    pools = [finite[c.rng.integers(0, 254, shape)] for _ in range(2)]
    return pools + [np.exp2(c.rng.integers(-10, 2, shape[:2])).astype(np.float32) for _ in range(2)]


def same_codes(got, want):
    """E4M3 codes, the two NaN codes and the two zeros of a re-encoded subnormal each alike."""
    nan = (got & 0x7F == 0x7F) & (want & 0x7F == 0x7F)
    return bool(((got == want) | nan).all())


@pytest.mark.parametrize("H,Hk,D,rot,il", SHAPES)
@pytest.mark.parametrize("many", [False, True])
def test_block_scaled_bit_exact(pk, H, Hk, D, rot, il, many):
    torch = torch_cuda()
    runs = RUNS + ([(320, 16 * 400 + 9), (6784 + 15, 18)] + [(6848 + 16 * i + i % 16, 1) for i in range(500)]
                   if many else [])
    c = Case(31 + D + rot, runs, H, Hk, D, rot, 960)
    kp0, vp0, ks0, vs0 = block_pools(c)
    hq, hk, hv = c.parts()
    slots = c.slots.copy()
    c.slots[2] = -1       # padding at a run's end
    slots[2] = -1
    if c.cs is not None:
        c.pos[26] = -1    # a skipped token: a run's only one
        slots[26] = -1
    kp, vp, ks, vs = (dev(x) for x in (kp0, vp0, ks0, vs0))
    q, k, v = c.dev_parts()
    out = torch.zeros((len(c.slots), H, D), dtype=torch.int16, device="cuda")
    cs, pos = args(c)
    pk.pa_rope_and_cache_fp8_block(out, q, k, v, kp, vp, ks, vs, cs, pos, dev(c.slots), interleaved=il)
    want_q = f32_to_bf16_bits(c.rotated(hq, il))
    if c.cs is not None:
        want_q[26] = 0
    assert np.array_equal(host_bits(out), want_q)
    wk, wks = block_scaled_write(c.rotated(hk, il), kp0, ks0, slots)
    wv, wvs = block_scaled_write(bf16_bits_to_f64(hv).astype(np.float32), vp0, vs0, slots)
    assert np.array_equal(ks.cpu().numpy(), wks) and np.array_equal(vs.cpu().numpy(), wvs)
    assert same_codes(kp.cpu().numpy(), wk) and same_codes(vp.cpu().numpy(), wv)
    check_device_error(0)


def test_block_scale_grows_token_by_token(pk):
    """A block filled one token per call, each four times louder than the one
    before. A value is rounded to E4M3 once (2^-4 of it), and at each of at most
    15 raises of the scale it is exact or, where it has become a subnormal, off
    by half a subnormal step of the new scale: 2^-10 * s_i, the s_i growing to
    the last s: sum <= 2^-10 s (1 + 1/4 + ...) < 2^-9 s; + 2^-10 s for the
    first rounding of a value that starts as a subnormal."""
    Hk, D = 2, 128
    rng = np.random.default_rng(5)
    x = rng.standard_normal((16, Hk, D)).astype(np.float32) * np.exp2(2.0 * np.arange(16) - 14)[:, None, None].astype(np.float32)
    bits = f32_to_bf16_bits(x)
    kp, vp = dev(np.full((3, Hk, 16, D), 0x7F, np.uint8)), dev(np.full((3, Hk, 16, D), 0x7F, np.uint8))
    ks, vs = dev(np.full((3, Hk), np.nan, np.float32)), dev(np.full((3, Hk), np.inf, np.float32))
    for t in range(16):
        row = dev(bits[t:t + 1])
        pk.pa_rope_and_cache_fp8_block(None, None, row, row, kp, vp, ks, vs, None, None, dev(np.array([16 + t], np.int64)))
    for pool, scale in ((kp, ks), (vp, vs)):
        s = scale.cpu().numpy()[1].astype(np.float64)
        got = e4m3_to_f64(pool.cpu().numpy()[1]) * s[:, None, None]          # [Hk][16][D]
        want = np.moveaxis(bf16_bits_to_f64(bits), 0, 1)
        assert (np.abs(want).max((1, 2)) <= 448 * s).all() and (np.abs(want).max((1, 2)) > 224 * s).all()
        assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 3 * 2.0 ** -10 * s[:, None, None]).all()
        assert (pool.cpu().numpy()[[0, 2]] == 0x7F).all() and not np.isfinite(scale.cpu().numpy()[[0, 2]]).any()
    check_device_error(0)


def test_extremes_of_the_block_scale(pk):
    """Zeros, values beyond 448 * 2^32, below 2^-41 and non-finite ones."""
    Hk, D = 1, 64
    x = np.zeros((48, Hk, D), np.float32)
    x[16:32] = 1e38
    x[16, 0, 0] = -1e38
    x[32:] = 2.0 ** -60
    x[40, 0, 1], x[40, 0, 2], x[40, 0, 3] = np.inf, -np.inf, np.nan
    bits = f32_to_bf16_bits(x)
    kp, vp = dev(np.full((3, Hk, 16, D), 9, np.uint8)), dev(np.full((3, Hk, 16, D), 9, np.uint8))
    ks, vs = dev(np.full((3, Hk), 1.0, np.float32)), dev(np.full((3, Hk), 1.0, np.float32))
    pk.pa_rope_and_cache_fp8_block(None, None, dev(bits), dev(bits), kp, vp, ks, vs, None, None, dev(np.arange(48)))
    assert ks.cpu().numpy()[:, 0].tolist() == [2.0 ** -32, 2.0 ** 32, 2.0 ** -32]
    got = e4m3_to_f64(kp.cpu().numpy())
    assert (got[0] == 0).all() and (np.abs(got[1]) == 448).all() and got[1, 0, 0, 0] == -448
    assert got[2, 0, 8, 1] == 448 and got[2, 0, 8, 2] == -448 and np.isnan(got[2, 0, 8, 3])
    assert np.isnan(got[2]).sum() == 1 and (got[2, 0, 0] == 0).all()
    check_device_error(0)


def test_bad_slots_and_positions_are_flagged_and_skipped(pk):
    torch = torch_cuda()
    for block in (False, True):
        c = Case(9, [(0, 5), (32, 4)], 4, 2, 128, 128, 4, max_pos=50)
        c.slots[2], c.pos[6] = 64, 50       # one past the pool, one past the table
        slots = c.slots.copy()
        slots[2] = slots[6] = -1
        kp0, vp0, ks0, vs0 = block_pools(c)
        q, k, v = c.dev_parts()
        out = torch.zeros((9, 4, 128), dtype=torch.int16, device="cuda")
        hq, hk, hv = c.parts()
        rk, rv = c.rotated(hk, False), bf16_bits_to_f64(hv).astype(np.float32)
        if block:
            kp, vp, ks, vs = (dev(x) for x in (kp0, vp0, ks0, vs0))
            pk.pa_rope_and_cache_fp8_block(out, q, k, v, kp, vp, ks, vs, dev(c.cs), dev(c.pos), dev(c.slots))
            # both skips split their block's tokens in two runs of one warp or of two: the block's
            # scale is not defined, the others' are, and nothing past the pool is written
            assert (ks.cpu().numpy()[[1, 3]] == ks0[[1, 3]]).all() and (kp.cpu().numpy()[[1, 3]] == kp0[[1, 3]]).all()
        else:
            kb, vb = bf16_pools(c)
            kp, vp = dev(kb), dev(vb)
            pk.pa_rope_and_cache(out, q, k, v, kp, vp, dev(c.cs), dev(c.pos), dev(c.slots))
            assert np.array_equal(host_bits(kp), scatter(kb, f32_to_bf16_bits(rk), slots))
            assert np.array_equal(host_bits(vp), scatter(vb, hv, slots))
        want = f32_to_bf16_bits(c.rotated(hq, False))
        want[6] = 0
        assert np.array_equal(host_bits(out), want)
        check_device_error(SLOT | POSITION)


def test_in_place_q_another_stream_and_graph(pk):
    torch = torch_cuda()
    c = Case(17, RUNS, 8, 2, 128, 64, 16)
    kp0, vp0, ks0, vs0 = block_pools(c)
    hq, hk, hv = c.parts()
    want = f32_to_bf16_bits(c.rotated(hq, False))
    wk, wks = block_scaled_write(c.rotated(hk, False), kp0, ks0, c.slots)
    kp, vp, ks, vs = (dev(x) for x in (kp0, vp0, ks0, vs0))
    q, k, v = c.dev_parts()
    cs, pos, slots = dev(c.cs), dev(c.pos), dev(c.slots)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pk.pa_rope_and_cache_fp8_block(q, q, k, v, kp, vp, ks, vs, cs, pos, slots)
    s.synchronize()
    assert np.array_equal(host_bits(q.contiguous()), want) and same_codes(kp.cpu().numpy(), wk)
    out = torch.zeros((len(c.slots), 8, 128), dtype=torch.int16, device="cuda")
    q, k, v = c.dev_parts()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_rope_and_cache_fp8_block(out, q, k, v, kp, vp, ks, vs, cs, pos, slots)
    kp.copy_(dev(kp0)), ks.copy_(dev(ks0))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out), want) and same_codes(kp.cpu().numpy(), wk)
    assert np.array_equal(ks.cpu().numpy(), wks)
    check_device_error(0)


def test_slots_past_2_31_elements(pk):
    """The last blocks of an E4M3 pool of more than 2^31 elements."""
    torch = torch_cuda()
    Hk, D, nb = 8, 128, (1 << 31) // (8 * 16 * 128) + 3
    kp, vp = (torch.zeros((nb, Hk, 16, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, Hk), dtype=torch.float32, device="cuda") for _ in range(2))
    c = Case(2, [((nb - 1) * 16, 16), ((nb - 3) * 16 + 1, 2)], 8, Hk, D, 128, nb)
    _, k, v = c.dev_parts()
    pk.pa_rope_and_cache_fp8_block(None, None, k, v, kp, vp, ks, vs, dev(c.cs), dev(c.pos), dev(c.slots))
    wk, wks = block_scaled_write(c.rotated(c.parts()[1], False), np.zeros((3, Hk, 16, D), np.uint8),
                                 np.zeros((3, Hk), np.float32), c.slots - (nb - 3) * 16)
    assert same_codes(kp[nb - 3:].cpu().numpy(), wk) and np.array_equal(ks[nb - 3:].cpu().numpy(), wks)
    assert int(kp[:nb - 3].max()) == 0
    check_device_error(0)


def test_empty_and_refused(pk):
    torch = torch_cuda()
    c = Case(1, [(0, 3)], 4, 2, 64, 64, 4)
    kp, vp = (dev(p) for p in bf16_pools(c))
    q, k, v = c.dev_parts()
    cs, pos, slots = dev(c.cs), dev(c.pos), dev(c.slots)
    out = torch.empty((3, 4, 64), dtype=torch.int16, device="cuda")
    pk.pa_rope_and_cache(out[:0], q[:0], k[:0], v[:0], kp, vp, cs, pos[:0], slots[:0])
    ok = dict(q_out=out, q=q, k=k, v=v, k_pool=kp, v_pool=vp, cos_sin=cs, positions=pos, slot_mapping=slots)
    for bad, err in [(dict(q=None), ValueError), (dict(slot_mapping=slots[:2]), ValueError),
                     (dict(positions=pos[:2]), ValueError), (dict(positions=None), ValueError),
                     (dict(positions=pos.int()), TypeError), (dict(cos_sin=cs.double()), TypeError),
                     (dict(k=k.cpu()), ValueError), (dict(k=k.float()), TypeError),
                     (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                     (dict(v=v[:, :1]), ValueError), (dict(k_scale=torch.ones(2, device="cuda")), ValueError),
                     (dict(cos_sin=cs[:, :24].contiguous()), pk.PagedKVError),
                     (dict(cos_sin=torch.zeros((5, 80), device="cuda")), pk.PagedKVError)]:
        with pytest.raises(err):
            pk.pa_rope_and_cache(**{**ok, **bad})
    with pytest.raises(TypeError):   # bf16 pools are no E4M3 pools
        pk.pa_rope_and_cache_fp8_block(out, q, k, v, kp, vp, torch.ones((4, 2), device="cuda"),
                                       torch.ones((4, 2), device="cuda"), cs, pos, slots)
    check_device_error(0)
