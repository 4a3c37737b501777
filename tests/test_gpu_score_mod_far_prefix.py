"""Windows that hide nothing, up to the largest number of 32 bits, under a prefix that shows
the first rows keys 70,000 positions ahead. Tolerance as in the prefill's tests."""
import functools

import numpy as np
import pytest

from oracle.score_mod import attend
from oracle.sinks import dense_kv
from tests._gpu import check_device_error, torch_cuda
from tests._score_mod import compare, queries, slopes_of
from tests._serving import Cache
from tests.test_gpu_score_mod_prefill import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


@functools.cache
def cache(kind, n, D):
    """The last 5,000 keys have a V of 3.5, so that a row that missed them shows it."""
    c = Cache(1, kind, [n], 1, D, chunk=[n])
    far = c.tables[0, (n - 5000) // 16:]
    c.v[far] = 0x4060 if kind == "bf16" else 0x7E
    if kind == "block":
        c.v_scale[far] = 2.0 ** -7
    return c


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("window", [70000, 2 ** 30, 2 ** 31 - 70000, 2 ** 31 - 65537, 2 ** 31 - 1])
@pytest.mark.parametrize("cap,alibi", [(30.0, False), (0.0, True)])
def test_no_window_hides_what_a_prefix_shows(pk, kind, window, cap, alibi):
    n, H, D = 70000, 2, 64
    c = cache(kind, n, D)
    c.window = window
    q, slopes = queries(3, n, H, D, 1.0), slopes_of(H) * np.float32(2.0 ** -8) if alibi else None
    got = run(pk, c, q, [n], D ** -0.5, cap, slopes, [n])
    check_device_error(0)
    k, v = dense_kv(c.k, c.k_scale, c.tables[0], n), dense_kv(c.v, c.v_scale, c.tables[0], n)
    rows = np.r_[0:20, 4000:4008, n - 20:n]
    ref = attend(q[rows], rows, k, v, D ** -0.5, cap, slopes, n)
    # biases of slopes 2^-12 and 2^-16 keep the scores' size below that of the derivation
    compare(got[rows], ref, q[rows], c, [slice(0, len(rows))], D, D ** -0.5, cap, 2.0 ** -11,
            2.0 ** -17 * 8 if kind == "bf16" else 0.0, f"window {window}")
