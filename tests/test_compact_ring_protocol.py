"""The compaction kernel's order of reads and writes, replayed: CTAs of a cluster that run at
any pace, copies that read memory at any time between their issue and the wait for them,
places noted S steps ahead in 8 buffers, and one barrier of the cluster a step. Whatever the
interleaving, each copy and each scale reads what was there before the call, no place of the
ring or of the notes is written while it may be read, and the tokens arrive."""
import os
import random
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_59_gb300", "csrc",
                        "compact.cu")).read()
NOTES = int(re.search(r"constexpr int kNotes = (\d+);", SRC).group(1))
STEPS = [int(x) for x in re.search(r"kSteps = BSC && C == 4 \? (\d+) : (\d+);", SRC).groups()]


class Cluster:
    """tokens: new position -> old position (None: cannot be used); `share` tokens a CTA and
    step. Cells and scales hold their old index, or ("new", ..) once written."""

    def __init__(self, rng, keep, first, ctas, share, steps_of_ring, barrier=True, ahead=None):
        self.rng, self.keep, self.first, self.ctas, self.share = rng, keep, first, ctas, share
        self.S = steps_of_ring
        self.ahead = self.S - 1 if ahead is None else ahead
        self.cells = {k: k for k in range(max(keep) + 17)}
        self.scales = {b: b for b in self.cells}
        self.steps = -(-(len(keep) - first) // (ctas * share))
        self.arrived, self.barrier = [0] * ctas, barrier

    def tokens(self, cta, s):
        a = self.first + (s * self.ctas + cta) * self.share
        return range(a, min(a + self.share, len(self.keep))) if s < self.steps else range(0)

    def cta(self, me):
        """What one CTA does, a yield wherever others may get ahead."""
        notes, ring, held, flying = {}, {}, {}, []

        def ask_scale(s):  # the load may read at any time until note(s), a step later
            held[s] = [self.keep[j] // 16 for j in self.tokens(me, s)]
            assert all(self.scales[b] == b for b in held[s]), "a scale was replaced before it was read"

        def note(s):
            assert all(self.scales[b] == b for b in held[s]), "a scale was replaced before it was read"
            assert notes.get(s % NOTES, (s - NOTES,))[0] <= s - NOTES and s - NOTES < self.stored[me]
            notes[s % NOTES] = (s, held.pop(s))

        def load(s):
            group = []
            if s < self.steps:
                assert notes.get(s % NOTES, (None,))[0] == s
                assert ring.get(s % self.S, (s - self.S,))[0] < self.stored[me], "a place of the ring is still to be stored"
                ring[s % self.S] = (s, {})
                group = [(s, j) for j in self.tokens(me, s)]
                self.rng.shuffle(group)
            flying.append(group)

        def fly(group, n):
            for _ in range(min(n, len(group))):
                s, j = group.pop()
                assert self.cells[self.keep[j]] == self.keep[j], "a token was replaced before it was read"
                ring[s % self.S][1][j] = self.keep[j]

        ask_scale(0)
        for s in range(self.S):
            note(s)
            ask_scale(s + 1)
            yield
        for s in range(self.ahead):
            load(s)
            yield
        for s in range(self.steps):
            note(s + self.S)
            ask_scale(s + self.S + 1)
            yield
            for g in flying:  # some of the copies have been made by now, in any order
                fly(g, self.rng.randint(0, len(g)))
            done = flying.pop(0)
            fly(done, len(done))
            yield
            self.arrived[me] += 1
            load(s + self.ahead)
            while self.barrier and min(self.arrived) <= s:
                yield
            at, got = ring[s % self.S]
            assert at == s and notes[s % NOTES][0] == s
            for j in self.tokens(me, s):
                self.cells[j] = ("new", got[j])
                self.scales[j // 16] = "new"
                if self.rng.random() < 0.2:
                    yield
            self.stored[me] = s + 1

    def run(self):
        self.stored = [0] * self.ctas
        left = [self.cta(c) for c in range(self.ctas)]
        while left:
            one = self.rng.choice(left)
            for _ in range(self.rng.choice([1, 1, 5, 200])):
                try:
                    next(one)
                except StopIteration:
                    left.remove(one)
                    break
        for j in range(self.first, len(self.keep)):
            assert self.cells[j] == ("new", self.keep[j])


def lists(rng):
    n_old = rng.choice([5, 40, 300, 900])
    n = rng.randint(1, n_old)
    keep = sorted(rng.sample(range(n_old), n))
    if rng.random() < 0.3:  # a shift by one: sources and destinations overlap everywhere
        keep = list(range(1, n + 1))
    first = next((j for j, k in enumerate(keep) if j != k), len(keep)) // 16 * 16
    return keep, first


@pytest.mark.parametrize("ring", sorted(set(STEPS)))
def test_any_interleaving_reads_what_was_there(ring):
    assert NOTES >= ring + 2
    rng = random.Random(ring)
    for _ in range(400):
        keep, first = lists(rng)
        Cluster(rng, keep, first, rng.choice([1, 2, 3, 8, 12, 16]), rng.choice([16, 32, 128]), ring).run()


def test_the_replay_sees_a_missing_barrier():
    rng, seen = random.Random(3), 0
    for _ in range(100):
        try:
            Cluster(rng, list(range(1, 700)), 0, 4, 16, max(STEPS), barrier=False).run()
        except AssertionError:
            seen += 1
    assert seen > 50


def test_the_replay_sees_a_ring_too_small():
    with pytest.raises(AssertionError):
        Cluster(random.Random(4), list(range(1, 700)), 0, 1, 16, max(STEPS), ahead=max(STEPS) + 1).run()
