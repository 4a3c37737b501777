"""Chunked prefill over an E4M3 cache with per-head scales: pa_prefill_fp8_block with
every block's row of scales the same. Against fp64 over the per-head cache; tolerance
as in the other tests of that call (scales need not be powers of two to be read)."""
import numpy as np
import pytest

from oracle.sinks import dense_kv, paged_prefill
from tests._gpu import check_device_error
from tests._serving import Cache, assert_close
from tests.test_gpu_sinks_prefill import WEIGHT, pk, run, start_loc  # noqa: F401 (pk: a fixture)
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

CTX, CHUNK = [1, 17, 300, 513], [1, 3, 65, 200]


@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 5)])
@pytest.mark.parametrize("splits", [0, 1])
def test_rows_of_equal_scales(pk, D, H, Hk, window, sinks, splits):
    c = Cache(D, "head", CTX, Hk, D, window, sinks, CHUNK)
    c.scale = D ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(H).standard_normal((sum(CHUNK), H, D)).astype(np.float32))
    ref = paged_prefill(q, c.k, c.v, c.tables, c.ctx, start_loc(CHUNK), c.scale, window, sinks, **c.scales())
    vm = max(np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[b], n))) for b, n in enumerate(CTX))
    c.kind = "block"
    c.k_scale, c.v_scale = (np.tile(s, (c.nb, 1)) for s in (c.k_scale, c.v_scale))
    assert_close(run(pk, c, q, CHUNK, splits), ref, WEIGHT, vm, f"D={D} window={window}")
    check_device_error(0)
