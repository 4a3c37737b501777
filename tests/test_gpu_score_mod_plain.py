"""Without a cap, biases or a prefix the reshaped calls are the plain ones: pa_decode_sinks,
pa_decode_fp8_block, pa_prefill_sinks, pa_prefill_fp8_block on the same inputs. And what a
prefill that leaves a sequence out gives for the others.

Both sides are within assert_close's bound of fp64 (tests/_score_mod.py), so within twice
that of each other."""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.score_mod import paged_prefill
from oracle.sinks import dense_kv
from tests import test_gpu_score_mod_decode as dec
from tests import test_gpu_score_mod_prefill as pre
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._score_mod import compare, largest_sum, queries, weight_error
from tests._serving import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def near(a, b, c, q, rows, D, scale, floor=0.0):
    vmax = max(np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[i], int(n)))) for i, n in enumerate(c.ctx) if n > 0)
    weight = weight_error(D, largest_sum(q, c, rows, D, scale), 0.0, 2.0 ** -11) + floor / vmax
    a, b = bf16_bits_to_f64(a), bf16_bits_to_f64(b)
    assert np.isfinite(a).all() and np.isfinite(b).all()
    bound = 2 * (2.0 ** -8 * np.abs(b) * (1 + 2.0 ** -7) + 2 * weight * vmax) * (1 + 2.0 ** -7)
    assert (np.abs(a - b) <= bound).all(), (np.abs(a - b) / bound).max()


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (128, 8, 1), (64, 8, 2), (128, 2, 2)])
@pytest.mark.parametrize("window,sinks", [(100, 5), (0, 0), (400, 33)])
@pytest.mark.parametrize("pt", [0, 64])
def test_decode_as_the_plain_calls(pk, kind, D, H, Hk, window, sinks, pt):
    torch = torch_cuda()
    c = Cache(D + H, kind, [1, 17, 130, 300, 513, 700], Hk, D, window, sinks)
    q, scale = queries(1, 6, H, D), D ** -0.5
    got = dec.run(pk, c, q, scale, partition_tokens=pt)
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    args = dict(window=window, n_sinks=sinks, workspace=pk.decode_workspace(qd, 700, pt), partition_tokens=pt)
    if kind == "bf16":
        pk.pa_decode_sinks(out, qd, dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), scale, 700, **args)
    else:
        pk.pa_decode_fp8_block(out, qd, dev(c.k), dev(c.v), dev(c.k_scale), dev(c.v_scale), dev(c.tables), dev(c.ctx), scale,
                               700, **args)
    torch.cuda.synchronize()
    near(got, host_bits(out), c, q, [slice(b, b + 1) for b in range(6)], D, scale)
    check_device_error(0)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (128, 8, 1), (64, 8, 8)])
@pytest.mark.parametrize("window,sinks", [(100, 5), (0, 0), (400, 33)])
@pytest.mark.parametrize("splits", [0, 2])
def test_prefill_as_the_plain_calls(pk, kind, D, H, Hk, window, sinks, splits):
    torch = torch_cuda()
    ctx, chunk = [17, 300, 700], [3, 290, 130]
    c = Cache(D + H, kind, ctx, Hk, D, window, sinks, chunk)
    q, scale = queries(2, sum(chunk), H, D), D ** -0.5
    got = pre.run(pk, c, q, chunk, scale, splits=splits)
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    loc = pre.start_loc(chunk)
    args = dict(window=window, n_sinks=sinks, workspace=pk.prefill_workspace(qd, 3, Hk, 290, splits), splits=splits)
    if kind == "bf16":
        pk.pa_prefill_sinks(out, qd, dev(c.k), dev(c.v), dev(c.tables), dev(c.ctx), dev(loc), scale, 290, **args)
    else:
        pk.pa_prefill_fp8_block(out, qd, dev(c.k), dev(c.v), dev(c.k_scale), dev(c.v_scale), dev(c.tables), dev(c.ctx), dev(loc),
                                scale, 290, **args)
    torch.cuda.synchronize()
    near(got, host_bits(out), c, q, [slice(int(a), int(b)) for a, b in zip(loc[:-1], loc[1:])], D, scale,
         2.0 ** -17 * 8 if kind == "bf16" else 0.0)
    check_device_error(0)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("cap,prefix", [(20.0, None), (0.0, [0, 40, 150])])
def test_the_others_of_a_call_that_leaves_a_sequence_out(pk, kind, cap, prefix):
    """The first chunk is beyond its bound, then the second's is not in the cache: their rows
    are untouched, all others those of fp64."""
    torch = torch_cuda()
    ctx, chunk = [300, 40, 200], [280, 40, 60]
    loc = pre.start_loc(chunk)
    c = Cache(8, kind, ctx, 2, 128, chunk=chunk)
    q = queries(2, 380, 16, 128)
    rows = [slice(int(a), int(b)) for a, b in zip(loc[:-1], loc[1:])]
    for out_of, max_chunk, lens in ((0, 64, ctx), (1, 280, [300, 39, 200])):
        c.ctx = np.array(ctx, np.int32)
        ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, loc, 0.1, cap, None, prefix, k_scale=c.k_scale, v_scale=c.v_scale)
        c.ctx = np.array(lens, np.int32)
        out = torch.full((380, 16, 128), 0x1234, dtype=torch.int16, device="cuda")
        got = pre.run(pk, c, q, chunk, 0.1, cap, None, prefix, max_chunk=max_chunk, out=out)
        check_device_error(16)
        assert (got[rows[out_of]] == 0x1234).all()
        c.ctx = np.array(ctx, np.int32)
        for i in range(3):
            if i != out_of:
                alone = [rows[j] if j == i else slice(0, 0) for j in range(3)]
                full = got.copy()
                full[rows[out_of]] = 0
                want = ref.copy()
                want[rows[out_of]] = 0
                compare(full, want, q, c, alone, 128, 0.1, cap, 2.0 ** -11, 2.0 ** -17 * 8 if kind == "bf16" else 0.0, f"sequence {i}")
