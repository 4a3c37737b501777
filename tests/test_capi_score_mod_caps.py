"""Caps that the calls take and refuse; none needs a GPU (a call without sequences returns first)."""
import numpy as np
import pytest

from tests.test_capi_score_mod import P, _dec, _pf


@pytest.mark.parametrize("call", [_dec, _pf])
@pytest.mark.parametrize("cap,status", [(2.0 ** 100, 0), (float(np.nextafter(np.float32(2 ** 100), np.float32(np.inf))), -1),
                                        (1e36, -1), (2e38, -1), (1e-30, 0), (50.0, 0)])
def test_caps_beyond_2_to_the_100_are_refused(capi, call, cap, status):
    for scales in (dict(), dict(ks=P, vs=P)):
        assert call(capi, B=0, cap=cap, **scales) == status
