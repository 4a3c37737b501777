"""Slopes far above any score, up to the largest of fp32 and of either sign: the nearest key, or
the farthest, takes the whole weight. Tolerance: tests/_score_mod.py (a mean of one value: the
other weights are below 2^-900)."""
import numpy as np
import pytest

from oracle.score_mod import paged_decode, paged_prefill
from tests import test_gpu_score_mod_decode as dec
from tests import test_gpu_score_mod_prefill as pre
from tests._gpu import check_device_error, torch_cuda
from tests._score_mod import compare, queries
from tests._serving import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


@pytest.mark.parametrize("kind,D,H,Hk", [("bf16", 128, 4, 2), ("bf16", 128, 8, 1), ("bf16", 64, 2, 2), ("block", 128, 4, 1),
                                         ("block", 64, 2, 2)])
@pytest.mark.parametrize("slope", [1e3, 1e9, 1e30, 3e38])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("cap", [0.0, 30.0, 300.0])
def test_one_key_takes_all(pk, kind, D, H, Hk, slope, sign, cap):
    slopes, scale = np.full(H, sign * slope, np.float32), D ** -0.5
    c = Cache(3, kind, [700, 31], Hk, D, chunk=[150, 31])
    sc = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    q = queries(1, 2, H, D, 2.0)
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, scale, cap, slopes, **sc)
    compare(dec.run(pk, c, q, scale, cap, slopes, 64), ref, q, c, [slice(0, 1), slice(1, 2)], D, scale, cap, 2.0 ** -11)
    q = queries(2, 181, H, D, 2.0)
    for prefix in (None, [650, 0], [700, 31]):
        ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, pre.start_loc([150, 31]), scale, cap, slopes, prefix, **sc)
        got = pre.run(pk, c, q, [150, 31], scale, cap, slopes, prefix)
        rows = [slice(0, 150), slice(150, 181)]
        if prefix == [700, 31]:  # the middle row of the second sequence has two farthest keys: left out
            middle = 150 + 15
            got, ref = got.copy(), ref.copy()
            got[middle], ref[middle] = 0, 0.0
        compare(got, ref, q, c, rows, D, scale, cap, 2.0 ** -11, 2.0 ** -17 * 8 if kind == "bf16" else 0.0, f"prefix {prefix}")
    check_device_error(0)
