"""Partitions of the tensor-core decode in calls whose sequences may attend to
16,384 tokens or more, whatever their number: sizes up to 2,048 tokens, and
smaller ones for sequences far below the bound. Against fp64; tolerance as in the
other tests of these calls (what no query sees is NaN, its table entries -1)."""
import numpy as np
import pytest

from oracle.sinks import dense_kv, paged_decode
from tests._gpu import check_device_error
from tests._serving import Cache, assert_close
from tests.test_gpu_decode_partitions import decode, pk  # noqa: F401 (pk: a fixture)
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

SHORT = [1, 513, 2000, 16, 0, 700, 4096, 129, 31]
# (contexts, bound): below the length from which sequences are cut, at it, far above every context
CASES = [(SHORT[:6], 16383), (SHORT[:5] + [16384], 16384), (SHORT, 131072), ([9000, 300] * 6, 40000),
         ([5] * 40 + [3000], 20000)]


@pytest.mark.parametrize("kind,H,Hk", [("block", 4, 2), ("block", 8, 1), ("head", 4, 1), ("bf16", 16, 2)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (16367, 9), (300, 5)])
@pytest.mark.parametrize("ctx,bound", CASES)
def test_partitions_of_long_spans(pk, kind, H, Hk, window, sinks, ctx, bound):
    if window < 0 and kind != "block":
        window = 2 ** 30  # pa_decode_sinks needs one
    c = Cache(H + len(ctx), kind, ctx, Hk, 128, window, sinks)
    c.scale = 128 ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(H).standard_normal((len(ctx), H, 128)).astype(np.float32))
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, c.scale, window, sinks, **c.scales())
    vm = max(np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[b], int(n)))) for b, n in enumerate(ctx) if n > 0)
    # a merge of n partitions adds n roundings of 2^-24 to the sums
    weight = 2.0 ** -12 + (0 if kind == "bf16" else 2.0 ** -11) + 256 * 2.0 ** -24
    assert_close(decode(pk, c, q, bound), ref, weight, vm, f"{kind} {ctx} {bound}")
    check_device_error(0)
