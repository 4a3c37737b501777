"""K and V of a block-scaled cache need a pool and a scale array each; one for both
is refused before anything is launched (no GPU needed)."""
import ctypes as C

import pytest


@pytest.mark.parametrize("same", ["pools", "scales"])
def test_one_array_for_both_is_refused(capi, same):
    a, b, c, d = (C.c_void_p(x << 20) for x in (1, 2, 3, 4))
    pools = (a, a) if same == "pools" else (a, b)
    scales = (c, c) if same == "scales" else (c, d)
    p = C.c_void_p(4096)
    assert capi.pa_rope_and_cache_fp8_block(None, None, p, p, *pools, *scales, None, None, p, 0, 0, 128, 128, 4, 0, 2, 64, 0,
                                            0, 0, 16, 16, None) == -1
