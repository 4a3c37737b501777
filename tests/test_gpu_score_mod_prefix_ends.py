"""Prefixes at the ends of 32 bits: the least is none, the largest the whole context. What no
row sees is NaN or has table entry -1."""
import pytest

from tests._gpu import torch_cuda
from tests._serving import Cache
from tests.test_gpu_score_mod_prefill import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 8, 8)])
@pytest.mark.parametrize("cap,alibi", [(30.0, False), (0.0, True), (30.0, True)])
@pytest.mark.parametrize("window", [-1, 60])
@pytest.mark.parametrize("splits", [0, 2])
def test_least_and_largest_prefixes(pk, kind, D, H, Hk, cap, alibi, window, splits):
    ctx, chunk = [300, 300, 150, 40], [290, 100, 150, 40]
    prefix = [-2 ** 31, 2 ** 31 - 1, -2 ** 31 + 1, -1]
    check(pk, Cache(window + D, kind, ctx, Hk, D, window, 0, chunk), H, D, chunk, cap, alibi, prefix, splits)
