"""Argument checks of the reshaped scores and of the compaction, the host side of a
compaction, and the compaction kernel's order of reads and writes, replayed; none
needs a GPU."""
import ctypes as C
import random

import numpy as np
import pytest

INF, NAN = float("inf"), float("nan")
P = C.c_void_p(4096)


def _dec(capi, **over):
    a = dict(out=C.c_void_p(8192), q=P, k=P, v=P, ks=None, vs=None, tab=P, ctx=P, scale=0.1, cap=50.0, slopes=None, H=8,
             Hk=2, D=128, bs=16, B=4, maxb=64, maxctx=1024, nb=256, window=-1, sinks=0, pt=2048, ws=None, wsb=0)
    a.update(over)
    return capi.pa_decode_score_mod(a["out"], a["q"], a["k"], a["v"], a["ks"], a["vs"], a["tab"], a["ctx"], a["scale"],
                                    a["cap"], a["slopes"], a["H"], a["Hk"], a["D"], a["bs"], a["B"], a["maxb"], a["maxctx"],
                                    a["nb"], a["window"], a["sinks"], a["pt"], a["ws"], a["wsb"], None)


def _pf(capi, **over):
    a = dict(out=C.c_void_p(8192), q=P, k=P, v=P, ks=None, vs=None, tab=P, ctx=P, loc=P, scale=0.1, cap=50.0, slopes=None,
             prefix=None, H=8, Hk=2, D=128, bs=16, B=4, maxb=64, chunk=100, nb=256, window=-1, sinks=0, splits=1, ws=None,
             wsb=0)
    a.update(over)
    return capi.pa_prefill_score_mod(a["out"], a["q"], a["k"], a["v"], a["ks"], a["vs"], a["tab"], a["ctx"], a["loc"],
                                     a["scale"], a["cap"], a["slopes"], a["prefix"], a["H"], a["Hk"], a["D"], a["bs"],
                                     a["B"], a["maxb"], a["chunk"], a["nb"], a["window"], a["sinks"], a["splits"], a["ws"],
                                     a["wsb"], None)


@pytest.mark.parametrize("call", [_dec, _pf])
@pytest.mark.parametrize("over,status", [
    (dict(B=0), 0), (dict(B=0, cap=0.0), 0), (dict(cap=-1.0), -1), (dict(cap=NAN), -1), (dict(cap=INF), -1),
    (dict(cap=1e-40), -1), (dict(cap=1.0, scale=INF), -1), (dict(cap=3.4e38), -1), (dict(slopes=C.c_void_p(4098)), -1),
    (dict(window=-2), -1), (dict(sinks=-1), -1), (dict(ks=P), -1), (dict(vs=P), -1),
    (dict(ks=C.c_void_p(4098), vs=P), -1), (dict(D=96), -2), (dict(bs=32), -2), (dict(H=6, Hk=2), -2),
    (dict(H=7, Hk=2), -1), (dict(q=None), -1), (dict(out=P), -1), (dict(k=C.c_void_p(4104)), -1), (dict(B=-1), -1),
    (dict(B=65536), -2),
])
def test_score_mod_argument_errors_need_no_device(capi, call, over, status):
    assert call(capi, **over) == status


def test_decode_and_prefill_bounds(capi):
    assert _dec(capi, maxb=8) == -1 and _dec(capi, pt=100) == -1 and _dec(capi, pt=64) == -3
    assert _pf(capi, prefix=C.c_void_p(4098)) == -1 and _pf(capi, splits=65) == -1 and _pf(capi, splits=3) == -3
    assert _pf(capi, loc=None) == -1 and _pf(capi, nb=2 ** 27) == -2


def _compact(capi, **over):
    a = dict(k=P, v=C.c_void_p(8192), ks=None, vs=None, tab=P, keep=P, loc=P, heads=1, n=10, Hk=2, D=128, bs=16, eb=2, B=3,
             maxb=8, nb=64)
    a.update(over)
    return capi.pa_compact_blocks(a["k"], a["v"], a["ks"], a["vs"], a["tab"], a["keep"], a["loc"], a["heads"], a["n"], a["Hk"],
                                  a["D"], a["bs"], a["eb"], a["B"], a["maxb"], a["nb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(B=0), 0), (dict(n=0, keep=None), 0), (dict(B=-1), -1), (dict(n=-1), -1), (dict(heads=3), -1), (dict(heads=0), -1),
    (dict(eb=4), -1), (dict(D=96), -2), (dict(bs=8), -2), (dict(k=None), -1), (dict(v=P), -1), (dict(keep=None), -1),
    (dict(tab=None), -1), (dict(loc=None), -1), (dict(k=C.c_void_p(4104)), -1), (dict(keep=C.c_void_p(4098)), -1),
    (dict(ks=P), -1), (dict(ks=P, vs=C.c_void_p(8192)), -1), (dict(ks=P, vs=P, eb=1), -1),
    (dict(ks=C.c_void_p(4098), vs=P, eb=1), -1), (dict(B=65536), -2), (dict(Hk=0), -1),
])
def test_compact_argument_errors_need_no_device(capi, over, status):
    assert _compact(capi, **over) == status


# ------------------------------------------------------------- block manager --

def test_compact_releases_the_tail(capi):
    from paged_kv_cache_59_gb300 import BlockManager, PagedKVError
    bm = BlockManager(20, 16)
    bm.add_seq(1)
    bm.append_tokens(1, 100)                          # 7 blocks
    tab = bm.block_table(1)
    assert bm.compact(1, 100) == (tab, []) and bm.num_free() == 13     # nothing moves
    assert bm.compact(1, 33, 20) == (tab, [])
    assert bm.block_table(1) == tab[:3] and bm.seq_len(1) == 33 and bm.num_free() == 17
    slots, cow = bm.append_tokens(1, 1)
    assert slots == [tab[2] * 16 + 1] and not cow
    assert bm.compact(1, 32)[0] == tab[:3] and bm.block_table(1) == tab[:2]
    assert bm.compact(1, 0)[0] == tab[:2] and bm.seq_len(1) == 0 and bm.num_free() == 20
    assert bm.compact(1, 0) == ([], [])
    bm.append_tokens(1, 20)
    for bad in ((21, 0), (-1, 0), (10, 11), (10, -1)):
        with pytest.raises(PagedKVError):
            bm.compact(1, *bad)
    with pytest.raises(PagedKVError):
        bm.compact(9, 0)
    assert bm.seq_len(1) == 20


def test_compact_takes_private_copies_of_shared_blocks(capi):
    from paged_kv_cache_59_gb300 import BlockManager, PagedKVError
    bm = BlockManager(12, 16)
    bm.add_seq(1)
    bm.append_tokens(1, 90)                           # 6 blocks
    old = bm.block_table(1)
    bm.fork(1, 2)
    table, pairs = bm.compact(2, 50, 20)              # writes blocks 1, 2, 3
    assert [p[0] for p in pairs] == old[1:4] and table == [old[0]] + [p[1] for p in pairs] + old[4:]
    assert bm.block_table(2) == table[:4] and bm.block_table(1) == old
    assert [bm.refcount(b) for b in old] == [2, 1, 1, 1, 1, 1]
    assert bm.num_free() == 3
    bm.fork(1, 3)
    with pytest.raises(PagedKVError):                 # four copies, three free blocks: nothing changes
        bm.compact(3, 60, 0)
    assert bm.block_table(3) == old and bm.num_free() == 3
    bm.compact(3, 48, 48)                             # a plain cut moves nothing and copies nothing
    assert bm.block_table(3) == old[:3] and bm.num_free() == 3


def test_compact_and_the_prefix_cache(capi):
    from paged_kv_cache_59_gb300 import BlockManager
    bm = BlockManager(20, 16)
    bm.add_seq(1)
    tokens = list(range(96))
    bm.append_tokens(1, 96)
    assert bm.cache_blocks(1, tokens) == 6
    table, pairs = bm.compact(1, 64, 30)              # cached blocks are copied, not written
    assert len(pairs) == 3
    bm.add_seq_cached(2, tokens)
    assert bm.seq_len(2) == 96
    bm.add_seq(3)
    more = list(range(1000, 1096))
    bm.append_tokens(3, 96)
    bm.compact(3, 70, 40)
    assert bm.cache_blocks(3, more) == 2              # positions from 40 on are no longer the prompt's
    bm.fork(3, 4)
    assert bm.cache_blocks(4, more) == 0
    bm.free_seq(1), bm.free_seq(2), bm.free_seq(3)
    bm.add_seq(5)
    last = list(range(2000, 2100))
    bm.append_tokens(5, 50)
    bm.compact(5, 50)                                 # nothing moves, nor does a cut move anything
    bm.compact(5, 40, 40)
    bm.append_tokens(5, 60)
    assert bm.cache_blocks(5, last) == 6


def test_compact_refuses_released_destinations(capi):
    from paged_kv_cache_59_gb300 import BlockManager, PagedKVError
    bm = BlockManager(20, 16)
    bm.add_seq(1)
    bm.append_tokens(1, 100)
    bm.release_between(1, 16, 64)                     # blocks 1 .. 3
    for n, first in ((40, 0), (20, 20), (70, 17)):
        with pytest.raises(PagedKVError):
            bm.compact(1, n, first)
    assert bm.seq_len(1) == 100
    bm.compact(1, 16, 0)
    assert bm.seq_len(1) == 16


# ------------------------------------------------------ the kernel, replayed --

def first_moved(keep, threads=256):
    """compact.cu's search."""
    n, lo, length = len(keep), 0, len(keep)
    if n > threads:
        stays = sum(keep[i] == i for i in range(threads))
        if stays < threads:
            return stays
        lo, length = threads, n - threads
    while length > 0:
        step = (length + threads - 1) // threads
        stays = sum(t * step < length and keep[lo + t * step] == lo + t * step for t in range(threads))
        if step == 1:
            return lo + stays
        if stays == 0:
            return lo
        a, b = (stays - 1) * step, min(stays * step, length)
        lo += a + 1
        length = b - a - 1
    return lo


def test_first_moved_finds_the_first():
    rng = random.Random(1)
    for _ in range(3000):
        threads = rng.choice([2, 4, 256])
        n = rng.choice([1, 2, 5, 255, 256, 257, 300, 1000, 5000])
        first = rng.choice([0, 1, rng.randrange(n + 1), n, n - 1])
        gap = rng.randint(1, 9)
        keep = [j if j < first else j + gap for j in range(n)]
        assert first_moved(keep, threads) == first


def test_steps_never_read_what_an_earlier_one_wrote():
    """A step is stored when steps up to the next are loaded (block scales: when those
    of the next two are read). Whatever lies between, what a later step reads must
    still be the old content."""
    rng = np.random.default_rng(2)
    for trial in range(300):
        n_old = int(rng.integers(1, 900))
        n = int(rng.integers(1, n_old + 1))
        keep = np.sort(rng.choice(n_old, n, replace=False))
        T = int(rng.choice([16, 32, 128]))
        cells, scales = np.arange(n_old + 16), np.arange(n_old // 16 + 2)
        j0 = first_moved(list(keep)) // 16 * 16
        steps = max(0, -(-(n - j0) // T))

        def part(s):
            return slice(j0 + s * T, min(n, j0 + (s + 1) * T))

        held = {}
        for s in range(steps):
            for ahead in ((0, 1) if s == 0 else (1,)):
                if s + ahead < steps:
                    held[s + ahead] = cells[keep[part(s + ahead)]].copy()
            for ahead in ((0, 1, 2) if s == 0 else (2,)):  # (the two ahead of the first are read before it, too)
                if s + ahead < steps:
                    got = scales[keep[part(s + ahead)] // 16]
                    assert np.array_equal(got, keep[part(s + ahead)] // 16)
            assert np.array_equal(held[s], keep[part(s)])
            cells[part(s)] = -1 - held[s]
            scales[np.arange(part(s).start, part(s).stop) // 16] = -1


def test_the_capped_prefill_s_work_list(monkeypatch):
    """The plan's arithmetic with the start of a segment counted as kStartCap tiles."""
    import re

    import tests.test_prefill_win_protocol as m
    monkeypatch.setattr(m, "K_START", int(re.search(r"constexpr int kStartCap = (\d+);", m.SRC).group(1)))
    assert m.K_START == 2
    m.test_work_list_covers_every_tile_once()
    m.test_work_list_is_even()
