"""Queries that are not finite, or beyond fp16, in one head (prefill: of one row): the other
heads' and rows' outputs are those of fp64. Tolerance: tests/_score_mod.py, a weight rounded
to fp16 (2^-11); V of a bf16 cache is staged within 2^-17 of the largest of its rows (prefill)."""
import numpy as np
import pytest

from oracle.score_mod import paged_decode, paged_prefill
from tests import test_gpu_score_mod_decode as dec
from tests import test_gpu_score_mod_prefill as pre
from tests._gpu import torch_cuda
from tests._score_mod import compare, queries, slopes_of
from tests._serving import Cache
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

NAN, INF, BEYOND = 0x7FC0, 0x7F80, int(f32_to_bf16_bits(np.array([1e6], np.float32))[0])
SHAPES = [(128, 8, 4), (128, 4, 1), (128, 16, 2), (128, 2, 2), (64, 8, 2)]


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", SHAPES)
@pytest.mark.parametrize("cap,alibi", [(30.0, False), (30.0, True), (300.0, False), (0.0, True)])
@pytest.mark.parametrize("bad", [NAN, INF, BEYOND])
def test_decode_keeps_heads_apart(pk, kind, D, H, Hk, cap, alibi, bad):
    c = Cache(D + H, kind, [300, 77], Hk, D)
    q, scale, slopes = queries(5, 2, H, D), D ** -0.5, slopes_of(H) if alibi else None
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, scale, cap, slopes, k_scale=c.k_scale, v_scale=c.v_scale)
    for head in (0, H - 1):
        mixed = q.copy()
        mixed[0, head, 3] = bad
        got = dec.run(pk, c, mixed, scale, cap, slopes).copy()
        got[0, head] = f32_to_bf16_bits(ref[0, head].astype(np.float32))
        compare(got, ref, q, c, [slice(0, 1), slice(1, 2)], D, scale, min(cap, 400.0), 2.0 ** -11, what=f"head {head}")
    pk.pa_get_device_error()


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", SHAPES)
@pytest.mark.parametrize("cap,alibi", [(30.0, False), (30.0, True), (300.0, False), (0.0, True)])
@pytest.mark.parametrize("bad", [NAN, INF, BEYOND])
def test_prefill_keeps_rows_and_heads_apart(pk, kind, D, H, Hk, cap, alibi, bad):
    chunk = [70, 33]
    c = Cache(D + H, kind, [300, 77], Hk, D, chunk=chunk)
    q, scale, slopes = queries(6, 103, H, D), D ** -0.5, slopes_of(H) if alibi else None
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, pre.start_loc(chunk), scale, cap, slopes, k_scale=c.k_scale,
                        v_scale=c.v_scale)
    floor = 2.0 ** -17 * 8 if kind == "bf16" else 0.0
    for row, head in ((0, 0), (69, H - 1)):
        mixed = q.copy()
        mixed[row, head, 3] = bad
        got = pre.run(pk, c, mixed, chunk, scale, cap, slopes).copy()
        got[row, head] = f32_to_bf16_bits(ref[row, head].astype(np.float32))
        compare(got, ref, q, c, [slice(0, 70), slice(70, 103)], D, scale, min(cap, 400.0), 2.0 ** -11, floor, f"row {row}")
    pk.pa_get_device_error()
