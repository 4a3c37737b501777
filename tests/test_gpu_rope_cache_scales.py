"""Block-scaled cache write into blocks whose scale it did not make itself."""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.fp8 import e4m3_to_f64
from tests.test_gpu_rope_cache import Case, block_pools, pk  # noqa: F401 (pk: a fixture)
from tests.test_gpu_rope_cache_blocks import write_and_compare

pytestmark = pytest.mark.gpu

FOREIGN = [np.nan, np.inf, -np.inf, 0.0, -1.0, 2.0 ** 40, 2.0 ** -40, 0.3, 1.5, 2.0 ** 32, 3.0 * 2.0 ** 31]


@pytest.mark.parametrize("old", FOREIGN)
@pytest.mark.parametrize("mag", [2.0 ** -12, 1.0, 2.0 ** 12])
def test_appending_to_a_block_with_a_foreign_scale(pk, old, mag):
    """Scales that the write does not make: the attention calls read them clamped
    to [2^-32, 2^32] (NaN as 2^-32), and so does the write, which leaves a power
    of two. Earlier tokens keep the value that those calls read: exactly while the
    scale stays, else to half an E4M3 step (2^-4 of the value, or 2^-10 of the new
    scale) besides one fp32 rounding of code times old over new scale, 2^-24; new
    tokens are within half a step of x."""
    for D in (64, 128):
        c = Case(8, [(16 + 9, 3)], 2, 2, D, 32, 3, mag=mag)
        kp0, vp0, ks0, vs0 = block_pools(c)
        ks0[1], vs0[1] = np.float32(old), np.float32(old)
        kp, vp, ks, vs = write_and_compare(pk, c, np.zeros(3, bool), pools=(kp0, vp0, ks0, vs0))
        read = np.float64(min(max(old, 2.0 ** -32), 2.0 ** 32)) if old == old else 2.0 ** -32
        for pool, was, scale, x in ((kp, kp0, ks, c.rotated(c.parts()[1], False)),
                                    (vp, vp0, vs, bf16_bits_to_f64(c.parts()[2]))):
            now = scale.cpu().numpy()[1].astype(np.float64)[:, None, None]
            assert ((now >= read * (1 - 2.0 ** -24)) & (now <= 2.0 ** 32)).all() and (np.frexp(now)[0] == 0.5).all()
            got = e4m3_to_f64(pool.cpu().numpy()[1]) * now
            before = e4m3_to_f64(was[1]) * np.float64(np.float32(read))
            rest = np.r_[0:9, 12:16]
            step = np.where(now == np.float32(read), 0.0, 1.0)
            assert (np.abs(got - before)[:, rest] <=
                    (step * (np.maximum(2.0 ** -4 * np.abs(before), 2.0 ** -10 * now) + 2.0 ** -24 * np.abs(before)))[:, rest]).all()
            new = np.moveaxis(np.asarray(x, np.float64), 0, 1)
            assert (np.abs(got[:, 9:12] - new) <= np.maximum(2.0 ** -4 * np.abs(new), 2.0 ** -10 * now) ).all()
