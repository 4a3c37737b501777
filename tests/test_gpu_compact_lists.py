"""Lists that a compaction cannot use, wherever in them the fault lies: among the positions
that stay before the first that moves, too."""
import numpy as np
import pytest

from tests._gpu import check_device_error, torch_cuda
from tests.test_gpu_compact import cache, run, tables_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


@pytest.mark.parametrize("kind", ["bf16", "head", "block"])
@pytest.mark.parametrize("heads", [1, 2])
@pytest.mark.parametrize("n,at,x", [(300, 5, 3), (100, 0, 1), (300, 255, 254), (300, 17, -7), (300, 20, 2 ** 31 - 1),
                                    (5000, 1234, 1233), (5000, 4998, 4997), (16, 15, 14)])
def test_a_fault_before_the_first_that_moves(pk, kind, heads, n, at, x):
    """All others stay where they are: the fault is flagged, and nothing changes."""
    rng = np.random.default_rng(n + at)
    nb = (n + 15) // 16 + 3
    pools, scales = cache(rng, kind, nb, 2, 64)
    tables = tables_of(rng, [n], nb)
    keep = np.tile(np.arange(n, dtype=np.int32), (heads, 1))
    keep[-1, at] = x
    got, got_scales = run(pk, pools, scales, tables, keep if heads > 1 else keep[0], np.array([0, n], np.int32))
    check_device_error(256)
    assert all(np.array_equal(a, b) for a, b in zip(got, pools))
    if scales:
        assert all(np.array_equal(a, b) for a, b in zip(got_scales, scales))


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("at,x", [(5, 3), (240, 100), (511, 510)])
def test_a_fault_with_tokens_behind_it_that_move(pk, kind, at, x):
    rng = np.random.default_rng(at)
    pools, scales = cache(rng, kind, 60, 2, 128)
    tables = tables_of(rng, [800], 60)
    keep = np.concatenate([np.arange(600), np.arange(650, 750)]).astype(np.int32)
    keep[at] = x
    got, _ = run(pk, pools, scales, tables, keep, np.array([0, 700], np.int32))
    check_device_error(256)
    free = np.setdiff1d(np.arange(60), tables[0])
    assert all(np.array_equal(a[free], b[free]) for a, b in zip(got, pools))


def test_positions_that_stay_beyond_the_table_are_flagged(pk):
    rng = np.random.default_rng(1)
    pools, scales = cache(rng, "bf16", 20, 2, 64)
    tables = tables_of(rng, [100], 20)
    for n, flag in ((112, 0), (113, 256), (400, 256)):
        got, _ = run(pk, pools, scales, tables, np.arange(n, dtype=np.int32), np.array([0, n], np.int32))
        check_device_error(flag)
        assert all(np.array_equal(a, b) for a, b in zip(got, pools))


def test_starts_that_decrease_are_flagged(pk):
    """The sequence between them is left as it was; the others move."""
    rng = np.random.default_rng(2)
    pools, scales = cache(rng, "bf16", 30, 2, 64)
    tables = tables_of(rng, [100, 100, 100], 30)
    keep = np.arange(50, 90, dtype=np.int32)
    got, _ = run(pk, pools, scales, tables, keep, np.array([0, 40, 20, 40], np.int32))
    check_device_error(256)
    for a, b in zip(got, pools):
        assert np.array_equal(a[tables[1]], b[tables[1]])
        for t, first, n in ((tables[0], 50, 40), (tables[2], 70, 20)):
            for j in range(n):
                k = first + j
                assert np.array_equal(a[t[j // 16], :, j % 16], b[t[k // 16], :, k % 16])
