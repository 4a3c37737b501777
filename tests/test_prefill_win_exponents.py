"""The windowed prefill's exponents of V on the CPU: their hand-over from the
converter warps to the softmax warps, and the arithmetic.

The hand-over is checked in the model of the kernel's roles (``run`` of
test_prefill_win_protocol), with the softmax warps' wait for their tile's
exponents added, as in the kernel's source: a softmax warp reads its tile's
exponents while it works on it, and no converter warp may have overwritten them.
"""
import inspect
import random
import re

import numpy as np
import pytest

from tests import test_prefill_win_protocol as protocol


def model():
    """``run`` with the exponents: each converter warp writes its quarter's and arrives at v_exp before it
    converts, a softmax warp waits for v_exp and reads them to the end of its tile."""
    src = inspect.getsource(protocol.run)

    def sub(a, b):
        nonlocal src
        assert src.count(a) == 1, a
        src = src.replace(a, b)

    sub('''                    assert mem["V", J % kVS] == J
''', '''                    assert mem["V", J % kVS] == J
                    mem["E", J % kVS, w] = J
                    B["v_exp", J % kVS].arrive()
                    yield
''')
    sub('''B["v_full", i], B["v_conv", i], B["v_free", i] = Bar(1), Bar(4), Bar(1)
''', '''B["v_full", i], B["v_conv", i], B["v_free", i], B["v_exp", i] = Bar(1), Bar(4), Bar(1), Bar(4)
''')
    sub('''                yield from wait("s_full", x, J & 1, J)
                assert mem["S", x] == J
                yield
''', '''                if EB == 2 and exp_wait:
                    yield from wait("v_exp", J % kVS, J // kVS & 1, J // kVS)
                yield from wait("s_full", x, J & 1, J)
                assert mem["S", x] == J
                for quarter in range(4 if EB == 2 else 0):
                    assert mem.get(("E", J % kVS, quarter)) == J
                    yield
                yield
''')
    sub('q_wait="q_free"):', 'q_wait="q_free", exp_wait=True):')
    names = dict(vars(protocol))
    exec(src, names)
    return names["run"]


@pytest.mark.parametrize("seed", range(6))
def test_softmax_warps_read_their_tiles_exponents(seed):
    run, rng = model(), random.Random(seed)
    for _ in range(25):
        run([rng.choice([1, 1, 2, 3, rng.randint(1, 9)]) for _ in range(rng.randint(1, 6))], 2, rng)


def test_without_the_wait_they_would_not():
    run, rng = model(), random.Random(0)
    with pytest.raises(AssertionError):
        for _ in range(60):
            run([rng.randint(1, 5) for _ in range(5)], 2, rng, exp_wait=False)


def test_the_kernel_waits_as_the_model_does():
    """The softmax warps' wait comes before that for their scores, and the exponents are written before the arrival."""
    src = re.sub(r"//[^\n]*", "", protocol.SRC)
    wait = src.index("pa::mbar_wait(bars.v_exp(vst), (uint32_t)vph, P.err, abort_flag);\n                if (ok) ok = pa::mbar_wait(bars.s_full(x)")
    assert wait > 0
    write = src.index("reinterpret_cast<float2*>(sm + L_::kVExp)[st * 4 + w4] =")
    assert "pa::mbar_arrive(bars.v_exp(st));" in src[write:write + 200]


LEAST = int(re.search(r"constexpr int kLeastExp = (-\d+);", protocol.SRC).group(1))


def staged(v):
    """fp64 of 32 keys' bf16-valued rows after staging: rounded to fp16 as v 2^(-8 - e), and taken back."""
    bits = v.astype(np.float32).view(np.uint32) >> 16 & 0x7FFF
    e = max(LEAST, min(0, (int(bits.max()) >> 7) - 127))
    f = np.uint32((119 - e) << 23).view(np.float32)
    with np.errstate(over="ignore"):
        return (v.astype(np.float32) * f).astype(np.float16).astype(np.float64) * 2.0 ** (8 + e), e


@pytest.mark.parametrize("scale", [0, -1, -6, -12, -20, -60, 3, 20])
def test_staged_values_keep_their_bits(scale):
    rng = np.random.default_rng(100 + scale)
    for _ in range(50):
        v = rng.standard_normal((32, 64)) * np.exp2(rng.integers(-30, 1, (32, 1)) * rng.integers(0, 2))
        v = (np.asarray(v * 2.0 ** scale, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)  # bf16 values
        got, e = staged(v)
        most = np.abs(v).max()
        assert (np.abs(got - v) <= 2.0 ** -17 * most).all()
        loud = np.abs(v) >= 2.0 ** -6 * most
        assert (got[loud] == v[loud]).all()
        assert e == (0 if most >= 1 else np.frexp(most)[1] - 1)


def test_staged_zeros_tiny_and_huge_values():
    assert staged(np.zeros((32, 64))) [1] == LEAST
    got, e = staged(np.full((32, 64), 2.0 ** -100))
    assert e == LEAST and (np.abs(got) <= 2.0 ** (LEAST - 17)).all()
    assert np.isinf(staged(np.full((32, 64), 2.0 ** 24))[0]).all()  # beyond 65504 * 2^8: flagged by the kernel
    assert (staged(np.full((32, 64), 255 * 2.0 ** 16))[0] == 255 * 2.0 ** 16).all()
