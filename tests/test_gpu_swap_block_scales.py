"""Preemption of a sequence in a block-scaled E4M3 cache: its codes are swapped
out and in again at other blocks, their rows of scales kept and put back by the
caller; in between other sequences overwrite the freed blocks and their scales.
Decode and prefill go on as if nothing had happened (the checks of a serving run)."""
import numpy as np
import pytest

from tests._gpu import check_device_error, dev, torch_cuda
from tests.test_gpu_serving_run import D, HK, Server, pk  # noqa: F401 (pk: a fixture)

pytestmark = pytest.mark.gpu


def test_a_preempted_sequence_keeps_its_scales(pk):
    torch = torch_cuda()
    sv = Server(pk, "block")
    for s in (1, 2):
        sv.bm.add_seq(s)
    sv.prefill([(1, 75), (2, 40)])
    sv.decode([1, 2])
    before = sv.held(1)

    out = sv.bm.swap_out(1)
    ids = dev(np.array(out, np.int32))
    hk, hv = (torch.empty((len(out), HK, 16, D), dtype=torch.uint8).pin_memory() for _ in range(2))
    pk.pa_swap_out_blocks(*sv.pools, ids, hk, hv)
    kept = [x[ids.long()].cpu() for x in sv.scales]

    quiet = sv.tokens
    sv.tokens = lambda n: [quiet(n)[0]] + [louder(x, 64.0) for x in quiet(n)[1:]]
    sv.append(2, 90)                        # takes the freed blocks, with other scales
    sv.tokens = quiet
    assert set(out) & set(sv.bm.block_table(2))

    back = sv.bm.swap_in(1)
    assert back != out
    new = dev(np.array(back, np.int32))
    pk.pa_swap_in_blocks(hk, hv, *sv.pools, new)
    for x, rows in zip(sv.scales, kept):
        x[new.long()] = rows.cuda()
    after = sv.held(1)
    assert all(np.array_equal(a, b) for a, b in zip(before, after))
    sv.decode([1])
    sv.prefill([(1, 20)])
    check_device_error(0)


def louder(bits, factor):
    from oracle.bf16 import bf16_bits_to_f64
    from workloads import f32_to_bf16_bits
    return f32_to_bf16_bits((bf16_bits_to_f64(bits) * factor).astype(np.float32))
