"""Default partitions of the tensor-core decode over block-scaled E4M3 and with
sinks: 512 .. 2048 tokens by the bound of the call, and smaller ones for
sequences far below it. Against fp64; tolerance as in the other tests of these
calls (what no query sees is NaN, its table entries -1)."""
import numpy as np
import pytest

from oracle.sinks import dense_kv, paged_decode
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._serving import Cache, assert_close
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def decode(pk, c, q, bound):
    torch = torch_cuda()
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    tables = np.pad(c.tables, ((0, 0), (0, (bound + 15) // 16 - c.tables.shape[1])), constant_values=-1)
    sc = [None if s is None else dev(s) for s in (c.k_scale, c.v_scale)]
    a, b = (out, qd, dev(c.k), dev(c.v)), (dev(tables), dev(c.ctx), c.scale, bound)
    ws = pk.decode_workspace(qd, bound)
    if c.kind == "block":
        pk.pa_decode_fp8_block(*a, *sc, *b, window=c.window, n_sinks=c.n_sinks, workspace=ws)
    else:
        pk.pa_decode_sinks(*a, *b, c.window, c.n_sinks, *sc, workspace=ws)
    torch.cuda.synchronize()
    return host_bits(out)


# (contexts, bound): one partition and several, a bound in one round of CTAs and in several, contexts
# at it, far below it and in between (where the partition is cut to a size of its own)
CASES = [([1], 131072), ([513], 513), ([4100], 4100), ([4100, 17, 1000], 131072), ([50000, 3, 1030, 0], 131072),
         ([65535, 40000, 5000, 512], 65535)]


@pytest.mark.parametrize("kind,H,Hk", [("block", 4, 2), ("block", 16, 2), ("head", 2, 2), ("bf16", 16, 2)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (600, 5), (45000, 40)])
@pytest.mark.parametrize("ctx,bound", CASES)
def test_partitions_of_few_sequences(pk, kind, H, Hk, window, sinks, ctx, bound):
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


def test_a_context_beyond_a_loose_bound_is_flagged(pk):
    """The bound is 40,000 in a table of 65,536: the excess is not attended."""
    c = Cache(3, "block", [65536, 700], 2, 128)
    c.scale = 128 ** -0.5
    q = f32_to_bf16_bits(np.random.default_rng(1).standard_normal((2, 4, 128)).astype(np.float32))
    torch = torch_cuda()
    qd = dev(q)
    out = torch.full_like(qd, 0x7FC0)
    pk.pa_decode_fp8_block(out, qd, dev(c.k), dev(c.v), dev(c.k_scale), dev(c.v_scale), dev(c.tables), dev(c.ctx),
                           c.scale, 40000, workspace=pk.decode_workspace(qd, 40000))
    torch.cuda.synchronize()
    check_device_error(16)
    got = host_bits(out)
    one = Cache(3, "block", [65536, 700], 2, 128)
    want = paged_decode(q[1:], one.k, one.v, one.tables[1:], one.ctx[1:], c.scale, -1, 0, **one.scales())
    vm = np.nanmax(np.abs(dense_kv(c.v, c.v_scale, c.tables[1], 700)))
    assert_close(got[1:], want, 2.0 ** -11 + 2.0 ** -12, vm)
