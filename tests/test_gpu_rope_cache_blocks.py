"""Block-scaled cache write: whose tokens a block's scale covers.

All of a call's tokens of a block (within 16 consecutive entries of
slot_mapping, in any order, skipped entries between them) get one scale, bit for
bit as ``oracle.rope_cache.block_scaled_write`` has it.
"""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.rope_cache import block_scaled_write
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests.test_gpu_rope_cache import Case, block_pools, pk, same_codes  # noqa: F401 (pk: a fixture)
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

SLOT, POSITION = 2, 256


def write_and_compare(pk, c, skipped, il=False, flags=0, pools=None):
    """skipped: truth value per token, left out by its slot or position."""
    torch = torch_cuda()
    kp0, vp0, ks0, vs0 = block_pools(c) if pools is None else pools
    _, hk, hv = c.parts()
    slots = np.where(skipped, -1, c.slots)
    kp, vp, ks, vs = (dev(x) for x in (kp0, vp0, ks0, vs0))
    q, k, v = c.dev_parts()
    out = torch.zeros((len(c.slots), c.H, c.D), dtype=torch.int16, device="cuda")
    pk.pa_rope_and_cache_fp8_block(out, q, k, v, kp, vp, ks, vs, dev(c.cs), dev(c.pos), dev(c.slots), interleaved=il)
    wk, wks = block_scaled_write(c.rotated(hk, il), kp0, ks0, slots)
    wv, wvs = block_scaled_write(bf16_bits_to_f64(hv).astype(np.float32), vp0, vs0, slots)
    assert np.array_equal(ks.cpu().numpy(), wks, equal_nan=True) and np.array_equal(vs.cpu().numpy(), wvs, equal_nan=True)
    assert same_codes(kp.cpu().numpy(), wk) and same_codes(vp.cpu().numpy(), wv)
    want_q = f32_to_bf16_bits(c.rotated(c.parts()[0], il))
    want_q[(c.pos < 0) | (c.pos >= len(c.cs))] = 0
    assert np.array_equal(host_bits(out), want_q)
    check_device_error(flags)
    return kp, vp, ks, vs


# KV heads and tokens so that a K/V warp looks at 1, 4 and 16 tokens
SIZES = [(2, 1, 128, 90), (2, 2, 64, 40), (8, 8, 128, 1000), (4, 8, 64, 3000), (8, 8, 128, 5000)]


@pytest.mark.parametrize("H,Hk,D,n", SIZES)
@pytest.mark.parametrize("il", [False, True])
def test_skipped_tokens_inside_a_block(pk, H, Hk, D, n, il):
    """A run of n tokens with a third of them skipped, by their slot or their
    position, below and beyond the range."""
    c = Case(n + D, [(5, n)], H, Hk, D, 32, n // 16 + 3)
    how = c.rng.integers(0, 12, n)
    how[:3] = [4, 0, 5]
    skipped = how < 4
    c.slots[how == 0] = -1
    c.slots[how == 1] = c.nb * 16 + 3
    c.pos[how == 2] = -7
    c.pos[how == 3] = len(c.cs)
    write_and_compare(pk, c, skipped, il, flags=SLOT | POSITION)


@pytest.mark.parametrize("H,Hk,D,n", SIZES)
def test_tokens_of_a_block_in_any_order(pk, H, Hk, D, n):
    """The tokens of every block shuffled; and two sequences' tokens in turn."""
    m = n // 16 * 16
    c = Case(n, [(0, m)], H, Hk, D, 64, m // 16 + 1)
    for b in range(m // 16):
        c.slots[16 * b:16 * b + 16] = 16 * b + c.rng.permutation(16)
    write_and_compare(pk, c, np.zeros(m, bool))
    half = n // 2
    c = Case(n, [(3, 2 * half)], H, Hk, D, 64, 2 * (half // 16 + 2))
    c.slots[0::2] = 3 + np.arange(half)
    c.slots[1::2] = (half // 16 + 2) * 16 + 9 + np.arange(half)
    # every other entry is another block's, so a block's 16 tokens span 31: eight at a time fit in 16
    for a in range(0, 2 * half, 16):
        part = Case(a, [(0, len(c.slots[a:a + 16]))], H, Hk, D, 64, c.nb)
        part.slots = c.slots[a:a + 16].copy()
        write_and_compare(pk, part, np.zeros(len(part.slots), bool))
        if a > 64:
            break


def test_a_first_slot_that_is_skipped(pk):
    """Without a token for its first slot a block keeps at least its earlier scale."""
    c = Case(3, [(16, 16)], 4, 2, 128, 64, 3)
    c.slots[0] = -1
    write_and_compare(pk, c, np.arange(16) == 0)


def test_padding_between_sequences(pk):
    """One token of each of 700 sequences, padding between and behind them."""
    n = 700
    c = Case(11, [(16 * i + i % 16, 1) for i in range(n)], 8, 8, 64, 64, n)
    skipped = c.rng.integers(0, 2, n).astype(bool)
    skipped[-90:] = True
    c.slots[skipped] = -1
    write_and_compare(pk, c, skipped)


def test_tokens_of_a_block_too_far_apart_are_flagged(pk):
    """Entries 0, 10 and 20 of one block: the last is beyond the 16 entries from
    the first, is not written, and flagged."""
    c = Case(5, [(16, 1), (64, 9), (17, 1), (96, 9), (18, 1)], 4, 2, 64, 32, 8)
    skipped = np.arange(21) == 20
    write_and_compare(pk, c, skipped, flags=SLOT)
