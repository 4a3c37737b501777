"""The largest caps over quiet blocks: they leave all scores as they are. Tolerance: tests/_score_mod.py."""
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


@pytest.mark.parametrize("kind,D,H,Hk", [("bf16", 128, 4, 2), ("bf16", 128, 8, 1), ("block", 128, 4, 1), ("block", 64, 2, 2)])
@pytest.mark.parametrize("kmag", [1.0, 2.0 ** -8])
@pytest.mark.parametrize("cap", [1e28, 2.0 ** 100])
def test_largest_caps_over_quiet_blocks(pk, kind, D, H, Hk, kmag, cap):
    c = Cache(3, kind, [200, 31], Hk, D, chunk=[150, 31], kmag=kmag)
    sc = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    q = queries(1, 2, H, D, 16.0 / kmag)
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, D ** -0.5, cap, None, **sc)
    compare(dec.run(pk, c, q, D ** -0.5, cap), ref, q, c, [slice(0, 1), slice(1, 2)], D, D ** -0.5, 400.0, 2.0 ** -11)
    q = queries(2, 181, H, D, 16.0 / kmag)
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, pre.start_loc([150, 31]), D ** -0.5, cap, None, **sc)
    compare(pre.run(pk, c, q, [150, 31], D ** -0.5, cap), ref, q, c, [slice(0, 150), slice(150, 181)], D, D ** -0.5, 400.0,
            2.0 ** -11, 2.0 ** -17 * 8 if kind == "bf16" else 0.0)
    check_device_error(0)
