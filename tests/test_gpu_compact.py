"""Compaction of paged sequences in place, bit for bit against a plain one."""
import numpy as np
import pytest

from oracle.score_mod import compact
from tests._gpu import check_device_error, dev, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def cache(rng, kind, nb, Hk, D):
    shape = (nb, Hk, 16, D)
    if kind == "bf16":
        return [rng.integers(0, 1 << 16, shape).astype(np.uint16) for _ in range(2)], None  # bits, NaN among them
    codes = [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
    if kind == "head":
        return codes, None
    codes = [np.where((c & 0x7F) == 0x7F, 0, c).astype(np.uint8) for c in codes]
    return codes, [np.exp2(rng.integers(-14, 3, (nb, Hk))).astype(np.float32) for _ in range(2)]


def tables_of(rng, ctx, nb):
    need = [(n + 15) // 16 for n in ctx]
    assert sum(need) <= nb
    ids, at = rng.permutation(nb), 0
    tables = np.full((len(ctx), max(1, max(need))), -1, np.int32)
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    return tables


def lists(rng, ctx, kept, heads, lead=0):
    out = []
    for n, m in zip(ctx, kept):
        rows = []
        for _ in range(heads):
            a = min(lead, m)
            rest = np.sort(rng.choice(np.arange(a, n), m - a, replace=False)) if m > a else np.zeros(0, int)
            rows.append(np.concatenate([np.arange(a), rest]))
        out.append(np.array(rows, np.int32).reshape(heads, m))
    return np.concatenate(out, 1), np.concatenate([[0], np.cumsum(kept)]).astype(np.int32)


def run(pk, pools, scales, tables, keep, starts, stream=None):
    torch = torch_cuda()
    p = [dev(x) for x in pools]
    s = [None, None] if scales is None else [dev(x) for x in scales]
    pk.pa_compact_blocks(*p, dev(tables), dev(keep), dev(starts), k_scale=s[0], v_scale=s[1], stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy().view(pools[0].dtype) for x in p], None if scales is None else [x.cpu().numpy() for x in s]


def check(pk, rng, kind, Hk, D, ctx, kept, per_head, lead=0):
    nb = sum((n + 15) // 16 for n in ctx) + 3
    pools, scales = cache(rng, kind, nb, Hk, D)
    tables = tables_of(rng, ctx, nb)
    keep, starts = lists(rng, ctx, kept, Hk if per_head else 1, lead)
    keep = keep if per_head else keep[0]
    got, got_scales = run(pk, pools, scales, tables, keep, starts)
    for i in range(2):
        want, want_scale = compact(pools[i], tables, keep, starts, None if scales is None else scales[i])
        if scales is not None:
            assert np.array_equal(got_scales[i], want_scale)
            # -0 and 0 are one value
            same = (got[i] == want) | ((got[i] | want) & 0x7F == 0)
            assert same.all(), (kind, D, np.argwhere(~same)[:5])
        else:
            assert np.array_equal(got[i], want), (kind, D, np.argwhere(got[i] != want)[:5])
    check_device_error(0)


@pytest.mark.parametrize("kind", ["bf16", "head", "block"])
@pytest.mark.parametrize("Hk,D", [(1, 64), (1, 128), (3, 64), (8, 128), (40, 64)])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("lead", [0, 4, 21, 290])
def test_ragged_sequences(pk, kind, Hk, D, per_head, lead):
    rng = np.random.default_rng(lead + D + Hk)
    check(pk, rng, kind, Hk, D, [300, 1, 17, 0, 64, 700, 33], [100, 1, 3, 0, 64, 699, 0], per_head, lead)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("n,m", [(2, 1), (16, 15), (17, 16), (128, 127), (513, 512), (1025, 1024), (2000, 1999), (5000, 4800), (9000, 40)])
def test_lengths(pk, kind, n, m):
    rng = np.random.default_rng(n)
    for Hk, D, lead in ((2, 128, 0), (2, 64, 0), (1, 128, m - 1), (1, 64, m // 2)):
        check(pk, rng, kind, Hk, D, [n], [m], False, lead)


@pytest.mark.parametrize("kind", ["bf16", "head", "block"])
def test_many_sequences(pk, kind):
    """Enough for whole rows (no column slices), and a shift by one token: sources and
    destinations overlap everywhere."""
    rng = np.random.default_rng(5)
    ctx = [int(x) for x in rng.integers(1, 700, 60)]
    check(pk, rng, kind, 4, 128, ctx, [int(rng.integers(0, n + 1)) for n in ctx], True)
    check(pk, rng, kind, 4, 64, ctx, [n - 1 for n in ctx], False)


def test_a_long_document(pk):
    rng = np.random.default_rng(6)
    for kind in ("bf16", "block"):
        check(pk, rng, kind, 2, 64, [70001], [69000], False)
        check(pk, rng, kind, 1, 128, [40000], [13000], True, 5)


def test_clusters_of_odd_sizes(pk):
    """Few units of long lists: 9 to 16 CTAs take a step together."""
    rng = np.random.default_rng(14)
    for kind, Hk, D, ctx in (("bf16", 8, 128, [12000]), ("block", 8, 128, [12000]), ("bf16", 5, 64, [9000, 8000]),
                             ("block", 3, 128, [9000, 100, 6000]), ("head", 7, 128, [15000])):
        check(pk, rng, kind, Hk, D, ctx, [n * 9 // 10 for n in ctx], True)


def test_scales_far_apart_and_out_of_range(pk):
    """Codes that vanish, subnormal ones, scales that are no powers of two, and ones
    that are read within [2^-32, 2^32]."""
    torch = torch_cuda()
    rng = np.random.default_rng(7)
    pools, _ = cache(rng, "block", 40, 2, 64)
    tables = tables_of(rng, [600], 40)
    keep, starts = lists(rng, [600], [250], 2)
    scales = [np.exp2(rng.uniform(-20, 20, (40, 2))).astype(np.float32) for _ in range(2)]
    got, got_scales = run(pk, pools, scales, tables, keep, starts)
    from oracle.fp8 import e4m3_to_f64
    for i in range(2):
        want, want_scale = compact(pools[i], tables, keep, starts, scales[i])
        assert np.array_equal(got_scales[i], want_scale)
        # the quotient of the scales and the product are rounded in fp32: a value next to a tie may go to either side,
        # one step of its binade (2^-3 of it), 2^-9 for a subnormal
        a, b = e4m3_to_f64(got[i]), e4m3_to_f64(want)
        assert (np.abs(a - b) <= np.maximum(2.0 ** -3 * np.abs(b), 2.0 ** -9)).all()
        assert (a != b).mean() < 1e-4
    bad = [np.where(rng.random((40, 2)) < 0.3, x, 1.0).astype(np.float32) for x in (np.nan, 1e30)]
    clamped = [np.clip(np.nan_to_num(x, nan=2.0 ** -32), 2.0 ** -32, 2.0 ** 32).astype(np.float32) for x in bad]
    got, got_scales = run(pk, pools, bad, tables, keep, starts)
    for i in range(2):
        want, want_scale = compact(pools[i], tables, keep, starts, clamped[i])
        blocks = tables[0, :(250 + 15) // 16]
        assert np.array_equal(got_scales[i][blocks], want_scale[blocks])
        assert ((got[i] == want) | ((got[i] | want) & 0x7F == 0)).all()
    assert torch is not None
    check_device_error(0)


def test_positions_it_cannot_use_are_skipped_and_flagged(pk):
    """Out of order, twice the same, negative, beyond the table, in a released block:
    the token is left out, the others move, and nothing outside the table is written."""
    rng = np.random.default_rng(8)
    for kind in ("bf16", "block"):
        pools, scales = cache(rng, kind, 20, 2, 64)
        tables = tables_of(rng, [160], 16)
        keep, starts = lists(rng, [160], [40], 1)
        keep = np.sort(rng.choice(np.arange(1, 100), 40, replace=False)).astype(np.int32)
        for at, x, flag in ((7, keep[6], 256), (7, -1, 256), (39, 160, 256), (39, 2 ** 31 - 1, 256), (20, keep[18], 256)):
            bad = keep.copy()
            bad[at] = x
            got, _ = run(pk, pools, scales, tables, bad, starts)
            check_device_error(flag)
            free = np.setdiff1d(np.arange(20), tables[0])
            for i in range(2):
                assert np.array_equal(got[i][free], pools[i][free])
                j = at % 16
                if scales is None:
                    assert np.array_equal(got[i][tables[0, at // 16], :, j], pools[i][tables[0, at // 16], :, j])
        for loc in ([0, 41], [-1, 20], [2 ** 30, 2 ** 30 + 5]):   # a list beyond the entries
            got, _ = run(pk, pools, scales, tables, keep, np.array(loc, np.int32))
            check_device_error(256)
            assert all(np.array_equal(a, b) for a, b in zip(got, pools))
        t = tables.copy()
        t[0, keep[30] // 16] = -1
        run(pk, pools, scales, t, keep, starts)
        check_device_error(1)
        t[0, keep[30] // 16] = 20
        run(pk, pools, scales, t, keep, starts)
        check_device_error(1)


def test_another_stream_and_a_captured_graph(pk):
    torch = torch_cuda()
    rng = np.random.default_rng(9)
    for kind in ("bf16", "block"):
        pools, scales = cache(rng, kind, 60, 2, 128)
        tables = tables_of(rng, [500, 300], 60)
        keep, starts = lists(rng, [500, 300], [200, 250], 2)
        want, want_scales = run(pk, pools, scales, tables, keep, starts)
        got, _ = run(pk, pools, scales, tables, keep, starts, stream=torch.cuda.Stream())
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
        p = [dev(x) for x in pools]
        s = [None, None] if scales is None else [dev(x) for x in scales]
        t = [dev(x) for x in (tables, keep, starts)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pk.pa_compact_blocks(*p, *t, k_scale=s[0], v_scale=s[1])
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy().view(b.dtype), b) for a, b in zip(p, want))
        if scales is not None:
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(s, want_scales))
    check_device_error(0)


def test_refusals(pk):
    torch = torch_cuda()
    rng = np.random.default_rng(10)
    pools, scales = cache(rng, "block", 8, 2, 64)
    k, v, ks, vs = (dev(x) for x in (*pools, *scales))
    tab, keep, loc = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 4), (3,), (2,)))

    def call(k=k, v=v, tab=tab, keep=keep, loc=loc, **more):
        pk.pa_compact_blocks(k, v, tab, keep, loc, **more)

    call(k_scale=ks, v_scale=vs)
    call(keep=keep[:0])
    for over, kind in ((dict(v=v[:4]), ValueError), (dict(v=v.to(torch.int16)), ValueError), (dict(keep=keep.long()), TypeError),
                       (dict(keep=torch.zeros((3, 3), dtype=torch.int32, device="cuda")), ValueError),
                       (dict(keep=keep.cpu()), ValueError), (dict(loc=loc[:1]), ValueError), (dict(tab=tab.long()), TypeError),
                       (dict(k_scale=ks), ValueError), (dict(k_scale=ks[:4], v_scale=vs), ValueError),
                       (dict(k=k.float(), v=v.float()), TypeError), (dict(v=k), pk.PagedKVError),
                       (dict(k=k.to(torch.int16), v=v.to(torch.int16), k_scale=ks, v_scale=vs), TypeError)):
        with pytest.raises(kind):
            call(**over)
    check_device_error(0)
