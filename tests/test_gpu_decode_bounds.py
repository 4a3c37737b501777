"""Contexts beyond max_context_len in the decode calls with sinks and over
block-scaled E4M3: flagged, by however little, and read as max_context_len
tokens; the other sequences as ever. Against fp64 (what no query sees of the
shortened contexts is NaN); tolerance as in the other tests of these calls."""
import numpy as np
import pytest

from oracle.sinks import dense_kv, paged_decode
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._serving import Cache, assert_close
from tests.test_gpu_decode_partitions import pk  # noqa: F401 (a fixture)
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

CONTEXT = 16


def check(pk, kind, H, Hk, D, bound, over, window, sinks, partition_tokens=0):
    """`over`: by how much each context passes the bound (or, negative, stays below it)."""
    torch = torch_cuda()
    true = np.array([bound + o for o in over], np.int32)
    c = Cache(D + bound, kind, np.minimum(true, bound), Hk, D, window, sinks)
    c.scale = D ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(H).standard_normal((len(over), H, D)).astype(np.float32))
    ref = paged_decode(q, c.k, c.v, c.tables, c.ctx, c.scale, window, sinks, **c.scales())
    vm = max(np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[b], int(n)))) for b, n in enumerate(c.ctx) if n > 0)
    # a wider table, its entries past the bound a block of NaN
    free = [i for i in range(c.nb) if i not in set(c.tables[c.tables >= 0].tolist())][0]
    tables = np.pad(c.tables, ((0, 0), (0, (bound + 15) // 16 - c.tables.shape[1])), constant_values=-1)
    tables = np.pad(tables, ((0, 0), (0, 400)), constant_values=free)
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    sc = [None if s is None else dev(s) for s in (c.k_scale, c.v_scale)]
    a, b = (out, qd, dev(c.k), dev(c.v)), (dev(tables), dev(true), c.scale, bound)
    ws = pk.decode_workspace(qd, bound, partition_tokens)
    if kind == "block":
        pk.pa_decode_fp8_block(*a, *sc, *b, window=window, n_sinks=sinks, workspace=ws, partition_tokens=partition_tokens)
    else:
        pk.pa_decode_sinks(*a, *b, window, sinks, *sc, workspace=ws, partition_tokens=partition_tokens)
    torch.cuda.synchronize()
    check_device_error(CONTEXT if max(over) > 0 else 0)
    weight = 2.0 ** -12 + (0 if kind == "bf16" else 2.0 ** -11) + 256 * 2.0 ** -24
    assert_close(host_bits(out), ref, weight, vm, f"{kind} bound={bound} over={over} window={window}")


KINDS = [("block", 8, 2, 128), ("block", 4, 4, 64), ("head", 8, 1, 128), ("bf16", 16, 2, 128), ("bf16", 4, 1, 64)]


@pytest.mark.parametrize("kind,H,Hk,D", KINDS)
@pytest.mark.parametrize("bound", [17, 700, 3001])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (90, 5), (2500, 20)])
@pytest.mark.parametrize("over", [[1, 0, -16], [-1, 130, 6000, -9]])
def test_contexts_past_the_bound(pk, kind, H, Hk, D, bound, window, sinks, over):
    if window < 0 and kind != "block":
        pytest.skip("pa_decode_sinks has a window")
    for partition_tokens in (0, 64):
        check(pk, kind, H, Hk, D, bound, over, window, sinks, partition_tokens)


def test_a_bound_of_many_partitions(pk):
    """The kernel that merges many partitions counts them from the shortened context too."""
    for over in ([1, -4000, -30000], [0, 0], [4000]):
        check(pk, "block", 8, 1, 128, 40000, over, -1, 0)
    check(pk, "bf16", 8, 1, 128, 40000, [15, -39000], 30000, 100)


@pytest.mark.parametrize("kind,H,Hk,D", KINDS)
def test_a_bound_of_nothing(pk, kind, H, Hk, D):
    """max_context_len 0: rows of zeros, flagged where there is a context."""
    torch = torch_cuda()
    c = Cache(1, kind, [20, 0], Hk, D)
    qd = dev(f32_to_bf16_bits(np.random.default_rng(1).standard_normal((2, H, D)).astype(np.float32)))
    out = torch.full_like(qd, 0x7FC0)
    sc = [None if s is None else dev(s) for s in (c.k_scale, c.v_scale)]
    for ctx, flag in (([20, 0], CONTEXT), ([0, 0], 0)):
        a, b = (out, qd, dev(c.k), dev(c.v)), (dev(c.tables), dev(np.array(ctx, np.int32)), 0.1, 0)
        if kind == "block":
            pk.pa_decode_fp8_block(*a, *sc, *b)
        else:
            pk.pa_decode_sinks(*a, *b, 10, 4, *sc)
        torch.cuda.synchronize()
        assert (host_bits(out) == 0).all()
        check_device_error(flag)
