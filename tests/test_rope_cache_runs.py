"""Which warp writes which token in the block-scaled cache write, on the CPU.

``runs`` replays the lane arithmetic of write_block_scaled (rope_cache.cu): the
entries a warp holds, the leaders among its own, the members of each run, and
the flag. Every token that is not skipped has to be in exactly one run, with all
tokens of its block, for any split of the call over warps: two warps that share
a block would race for its scale.
"""
import random

import pytest

BS = 16


def runs(slots, n_blocks, per_warp):
    T = len(slots)
    block = lambda t: slots[t] // BS if 0 <= t < T and 0 <= slots[t] < n_blocks * BS else -1
    out, flagged = [], False
    for t0 in range(0, T, per_warp):
        first = [block(t0 + lane) for lane in range(32)]
        second = [block(t0 - 16 + lane if lane < 16 else t0 + 16 + lane) for lane in range(32)]
        todo = [lane for lane in range(per_warp) if first[lane] >= 0]
        while todo:
            l0 = todo[0]
            alike, alike2 = (sum(1 << i for i, b in enumerate(x) if b == first[l0]) for x in (first, second))
            todo = [lane for lane in todo if not alike >> lane & 1]
            if (alike2 & 0xffff) >> (l0 + 1):
                continue
            run = alike >> l0 & 0xffff
            out.append([t0 + l0 + i for i in range(BS) if run >> i & 1])
            flagged |= ((alike2 >> 16) << 16 | alike >> 16) >> l0 != 0
    return out, flagged


def draw(rng):
    """Slots of several sequences' chunks, some tokens skipped, blocks' tokens in any order."""
    slots, blk = [], 0
    for _ in range(rng.randint(1, 12)):
        n, at = rng.choice([1, 1, rng.randint(1, 20), rng.randint(1, 70)]), rng.randint(0, 15)
        chunk = list(range(blk * BS + at, blk * BS + at + n))
        blk = chunk[-1] // BS + 1
        if rng.random() < 0.3:
            by = {}
            for s in chunk:
                by.setdefault(s // BS, []).append(s)
            chunk = [s for b in by.values() for s in rng.sample(b, len(b))]
        skip = rng.choice([0, 0, 0.1, 0.5, 0.9])
        slots += [rng.choice([-1, 10 ** 6]) if rng.random() < skip else s for s in chunk]
        slots += [-1] * rng.choice([0, 0, 1, 17, 40])
    return slots, blk


@pytest.mark.parametrize("per_warp", [1, 4, 16])
def test_every_block_has_one_owner(per_warp):
    rng = random.Random(per_warp)
    for _ in range(400):
        slots, n = draw(rng)
        got, flagged = runs(slots, n, per_warp)
        want = {}
        for t, s in enumerate(slots):
            if 0 <= s < n * BS:
                want.setdefault(s // BS, []).append(t)
        assert sorted(got) == sorted(want.values()) and not flagged


@pytest.mark.parametrize("per_warp", [1, 4, 16])
def test_tokens_left_out_are_flagged(per_warp):
    """A block's tokens over more than 16 entries, each within 15 of the one
    before: one owner still, and a flag when that leaves some out."""
    rng = random.Random(per_warp)
    for _ in range(300):
        slots = [-1] * rng.randint(0, 20)
        for s in rng.sample(range(BS), rng.randint(2, BS)):
            slots += [s] + [rng.choice([-1, 32 + len(slots) * BS])] * rng.randint(0, 14)
        got, flagged = runs(slots, 10 ** 4, per_warp)
        mine = [r for r in got if 0 <= slots[r[0]] < BS]
        tokens = [t for t, s in enumerate(slots) if 0 <= s < BS]
        lost = [t for t in tokens if t > tokens[0] + 15]
        assert mine[0] == tokens[:len(tokens) - len(lost)]
        assert bool(lost) == flagged
