"""C ABI argument checks of the rotated cache write and of attention over
windows with sinks and block-scaled E4M3 caches; none needs a GPU."""
import ctypes as C

import pytest


# ------------------------------------------------- rotated cache write --

def _rope_args(**over):
    p = C.c_void_p(4096)
    a = dict(qo=C.c_void_p(8192), q=p, k=p, v=p, kp=p, vp=p, cs=p, pos=p, slots=p, ks=None, vs=None, qos=256, qs=256,
             kst=128, vst=128, T=4, H=4, Hk=2, D=64, rot=64, maxp=100, il=0, bs=16, nb=16)
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(Hk=0), -1), (dict(nb=-1), -1), (dict(D=96), -2), (dict(bs=8), -2),
    (dict(rot=24), -2), (dict(rot=80), -1), (dict(rot=-16), -1), (dict(q=None), -1), (dict(qo=None), -1),
    (dict(H=0), -1), (dict(k=None), -1), (dict(slots=None), -1), (dict(cs=None), -1), (dict(pos=None), -1),
    (dict(cs=C.c_void_p(4100)), -1), (dict(k=C.c_void_p(4104)), -1), (dict(q=C.c_void_p(4104)), -1),
    (dict(slots=C.c_void_p(4100)), -1), (dict(kst=64), -1), (dict(vst=132), -1), (dict(qs=0), -1), (dict(qos=128), -1),
    (dict(qo=C.c_void_p(4096), qs=512), -1), (dict(ks=C.c_void_p(4096)), -1),
    (dict(ks=C.c_void_p(4098), vs=C.c_void_p(4096)), -1),
])
def test_rope_argument_errors_need_no_device(capi, over, status):
    a = _rope_args(**over)
    tail = [a["qos"], a["qs"], a["kst"], a["vst"], a["T"], a["H"], a["Hk"], a["D"], a["rot"], a["maxp"], a["il"],
            a["bs"], a["nb"], None]
    assert capi.pa_rope_and_cache(a["qo"], a["q"], a["k"], a["v"], a["kp"], a["vp"], a["cs"], a["pos"], a["slots"],
                                  a["ks"], a["vs"], *tail) == status
    p = C.c_void_p(4096)
    if "ks" not in over:
        assert capi.pa_rope_and_cache_fp8_block(a["qo"], a["q"], a["k"], a["v"], a["kp"], a["vp"], p, p, a["cs"], a["pos"],
                                                a["slots"], *tail) == status
        if a["T"] > 0:
            assert capi.pa_rope_and_cache_fp8_block(a["qo"], a["q"], a["k"], a["v"], a["kp"], a["vp"], None, p, a["cs"],
                                                    a["pos"], a["slots"], *tail) == -1


# -------------------------------- decode: window with sinks, block scales --

def _dec(capi, fn, **over):
    p = C.c_void_p(4096)
    a = dict(out=C.c_void_p(8192), q=p, k=p, v=p, ks=None, vs=None, tab=p, ctx=p, scale=0.1, H=8, Hk=2, D=128, bs=16,
             B=4, maxb=64, maxctx=1024, nb=256, window=100, sinks=4, pt=0, ws=None, wsb=0)
    if fn == "pa_decode_fp8_block":
        a.update(ks=p, vs=p)
    a.update(over)
    return getattr(capi, fn)(a["out"], a["q"], a["k"], a["v"], a["ks"], a["vs"], a["tab"], a["ctx"], a["scale"], a["H"],
                             a["Hk"], a["D"], a["bs"], a["B"], a["maxb"], a["maxctx"], a["nb"], a["window"], a["sinks"],
                             a["pt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fn", ["pa_decode_sinks", "pa_decode_fp8_block"])
@pytest.mark.parametrize("over,status", [
    (dict(B=0), 0), (dict(window=-2), -1), (dict(sinks=-1), -1), (dict(D=96), -2), (dict(bs=32), -2),
    (dict(H=6, Hk=2), -2), (dict(H=7, Hk=2), -1), (dict(q=None), -1), (dict(out=C.c_void_p(4096)), -1),
    (dict(k=C.c_void_p(4104)), -1), (dict(pt=100), -1), (dict(maxb=8), -1), (dict(vs=None, ks=C.c_void_p(4096)), -1),
    (dict(ks=C.c_void_p(4098), vs=C.c_void_p(4096)), -1),
    # 100 + 2048 positions in 64-token partitions need split-K scratch; a window alone of 20 does not
    (dict(window=2000, sinks=100, maxctx=4096, maxb=256, pt=64), -3), (dict(B=-1), -1),
])
def test_decode_sinks_argument_errors_need_no_device(capi, fn, over, status):
    assert _dec(capi, fn, **over) == status


def test_decode_sinks_needs_a_window(capi):
    assert _dec(capi, "pa_decode_sinks", window=-1) == -1
    assert _dec(capi, "pa_decode_fp8_block", window=-1, B=0) == 0
    assert _dec(capi, "pa_decode_fp8_block", ks=None, vs=None) == -1


# ------------------------------- prefill: window with sinks, block scales --

def _pf(capi, fn, **over):
    p = C.c_void_p(4096)
    a = dict(out=C.c_void_p(8192), q=p, k=p, v=p, ks=p, vs=p, tab=p, ctx=p, loc=p, scale=0.1, H=8, Hk=2, D=128, bs=16,
             B=4, maxb=64, chunk=100, nb=256, window=100, sinks=4, splits=1, ws=None, wsb=0)
    a.update(over)
    scales = [a["ks"], a["vs"]] if fn == "pa_prefill_fp8_block" else []
    return getattr(capi, fn)(a["out"], a["q"], a["k"], a["v"], *scales, a["tab"], a["ctx"], a["loc"], a["scale"], a["H"],
                             a["Hk"], a["D"], a["bs"], a["B"], a["maxb"], a["chunk"], a["nb"], a["window"], a["sinks"],
                             a["splits"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fn", ["pa_prefill_sinks", "pa_prefill_fp8_block"])
@pytest.mark.parametrize("over,status", [
    (dict(B=0), 0), (dict(chunk=0), 0), (dict(window=-2), -1), (dict(sinks=-1), -1), (dict(D=96), -2), (dict(bs=32), -2),
    (dict(H=6, Hk=2), -2), (dict(H=7, Hk=2), -1), (dict(q=None), -1), (dict(loc=None), -1),
    (dict(out=C.c_void_p(4096)), -1), (dict(k=C.c_void_p(4104)), -1), (dict(splits=65), -1), (dict(splits=3), -3),
    (dict(nb=2 ** 27), -2), (dict(B=-1), -1),
])
def test_prefill_sinks_argument_errors_need_no_device(capi, fn, over, status):
    assert _pf(capi, fn, **over) == status


def test_prefill_scales_and_windows(capi):
    assert _pf(capi, "pa_prefill_sinks", window=-1) == -1
    for over in (dict(ks=None), dict(vs=None), dict(ks=C.c_void_p(4098))):
        assert _pf(capi, "pa_prefill_fp8_block", **over) == -1


def test_copy_blocks_with_scales_argument_errors(capi):
    p = C.c_void_p(4096)
    assert capi.pa_copy_blocks_fp8_block(p, p, None, p, p, 3, 2, 64, 16, 16, None) == -1
    assert capi.pa_copy_blocks_fp8_block(p, p, p, C.c_void_p(4098), p, 3, 2, 64, 16, 16, None) == -1
    assert capi.pa_copy_blocks_fp8_block(p, p, p, p, p, 3, 2, 64, 8, 16, None) == -2
    assert capi.pa_copy_blocks_fp8_block(p, p, p, p, None, 0, 2, 64, 16, 16, None) == 0


# ------------------------------------------------ block manager: sinks stay --

def test_release_between(capi):
    from paged_kv_cache_59_gb300 import BlockManager, PagedKVError
    bm = BlockManager(20, 16)
    bm.add_seq(1)
    bm.append_tokens(1, 200)                       # 13 blocks
    tab = bm.block_table(1)
    assert bm.release_between(1, 0, 0) == 0 and bm.release_between(1, 5, 31) == 0
    assert bm.release_between(1, 17, 100) == 4     # blocks 2..5; 1 holds position 16, 6 position 100
    assert bm.block_table(1) == tab[:2] + [-1] * 4 + tab[6:]
    assert bm.release_between(1, 17, 100) == 0 and bm.num_free() == 7 + 4
    assert bm.release_between(1, 16, 10 ** 9) == 7   # 1 and 6..11: the last block is not wholly before 200
    assert bm.block_table(1) == tab[:1] + [-1] * 11 + tab[12:]
    bm.fork(1, 2)
    assert bm.release_between(2, 0, 16) == 1 and bm.refcount(tab[0]) == 1
    for bad in ((-1, 5), (6, 5)):
        with pytest.raises(PagedKVError):
            bm.release_between(1, *bad)
    with pytest.raises(PagedKVError):
        bm.release_between(9, 0, 5)
    bm.free_seq(1), bm.free_seq(2)
    assert bm.num_free() == 20
