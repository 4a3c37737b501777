"""Copies that a compaction asks for, under memory pressure: destinations are fresh, and
no block is read by one copy and written by another, as all of them run at once."""
import random

import numpy as np
import pytest

BS = 16


class Server:
    """A block manager with what its blocks hold (one number a token), and what each
    sequence ought to hold."""

    def __init__(self, blocks):
        from paged_kv_cache_59_gb300 import BlockManager
        self.bm, self.pool, self.want, self.next = BlockManager(blocks, BS), np.full((blocks, BS), -1), {}, 0

    def write(self, seq, n):
        slots, pairs = self.bm.append_tokens(seq, n)
        self.copy(pairs)
        new = list(range(self.next, self.next + n))
        self.next += n
        self.pool.reshape(-1)[slots] = new
        self.want[seq] = self.want.get(seq, []) + new

    def copy(self, pairs):
        sources, targets = [a for a, _ in pairs], [b for _, b in pairs]
        assert len(set(targets)) == len(targets) and not set(sources) & set(targets), pairs
        if pairs:
            self.pool[targets] = self.pool[sources]

    def move(self, tables, keeps):
        """pa_compact_blocks: the sequences of one call in either order, which may not matter."""
        ends = []
        for order in (1, -1):
            pool = self.pool.copy()
            for table, keep in list(zip(tables, keeps))[::order]:
                held = [pool[table[k // BS], k % BS] for k in keep]
                first = next((j for j, k in enumerate(keep) if j != k), len(keep)) // BS * BS
                for j in range(first, len(keep)):
                    pool[table[j // BS], j % BS] = held[j]
            ends.append(pool)
        assert np.array_equal(*ends)
        self.pool = ends[0]

    def check(self):
        for seq, want in self.want.items():
            table = self.bm.block_table(seq)
            got = [int(self.pool[table[i // BS], i % BS]) for i in range(len(want))]
            assert got == want and self.bm.seq_len(seq) == len(want), seq


def test_a_copied_block_is_not_handed_out_as_a_destination(capi):
    """Nothing is free; a cache entry younger than the sequence's own is evictable. The
    sequence's first block, once it is the cache's alone, is older than that."""
    s = Server(4)
    s.bm.add_seq(1)
    s.write(1, 32)
    tokens = [list(range(100, 132)), list(range(200, 216)), list(range(300, 316))]
    assert s.bm.cache_blocks(1, tokens[0]) == 2
    for seq in (2, 3):
        s.bm.add_seq(seq)
        s.write(seq, 16)
        assert s.bm.cache_blocks(seq, tokens[seq - 1]) == 1
        s.bm.free_seq(seq)
        del s.want[seq]
    assert s.bm.num_free() == 0
    old = s.bm.block_table(1)
    table, pairs = s.bm.compact(1, 20, 0)
    assert [a for a, _ in pairs] == old
    s.copy(pairs)
    keep = list(range(5, 25))
    s.move([table], [keep])
    s.want[1] = [s.want[1][k] for k in keep]
    s.check()


@pytest.mark.parametrize("seed", range(6))
def test_random_servers_short_of_blocks(capi, seed):
    from paged_kv_cache_59_gb300 import PagedKVError
    rng, several, moved, batches = random.Random(seed), 0, 0, 0
    for _ in range(150):
        s = Server(rng.randint(6, 14))
        prompts = [[rng.randrange(1000) for _ in range(BS * 5)] for _ in range(2)]
        ids = 0
        for _ in range(60):
            try:
                what, live = rng.random(), list(s.want)
                if what < 0.3 or not live:
                    ids += 1
                    prompt = rng.choice(prompts)
                    n = s.bm.add_seq_cached(ids, prompt)
                    table = s.bm.block_table(ids)
                    s.want[ids] = [int(x) for x in s.pool[table].reshape(-1)] if n else []
                    s.write(ids, rng.randint(1, len(prompt) - n + 9))
                    s.bm.cache_blocks(ids, prompt[:s.bm.seq_len(ids)])
                elif what < 0.4:
                    ids += 1
                    seq = rng.choice(live)
                    s.bm.fork(seq, ids)
                    s.want[ids] = list(s.want[seq])
                elif what < 0.55:
                    s.write(rng.choice(live), rng.randint(1, 20))
                elif what < 0.65:
                    seq = rng.choice(live)
                    s.bm.free_seq(seq)
                    del s.want[seq]
                elif what < 0.82:
                    some = rng.sample(live, rng.randint(1, len(live)))
                    keeps = [sorted(rng.sample(range(len(s.want[q])), rng.randint(0, len(s.want[q])))) for q in some]
                    firsts = [next((j for j, k in enumerate(keep) if j != k), len(keep)) for keep in keeps]
                    tables, pairs = s.bm.compact_batch(some, [len(k) for k in keeps], rng.choice([None, firsts]))
                    s.copy(pairs)
                    s.move(tables.tolist(), keeps)
                    batches += len(some) > 1 and len(pairs) > 1
                    for seq, keep in zip(some, keeps):
                        s.want[seq] = [s.want[seq][k] for k in keep]
                else:
                    seq = rng.choice(live)
                    n = len(s.want[seq])
                    keep = sorted(rng.sample(range(n), rng.randint(0, n)))
                    first = next((j for j, k in enumerate(keep) if j != k), len(keep))
                    table, pairs = s.bm.compact(seq, len(keep), rng.choice([0, first]) if keep else 0)
                    several += len(pairs) > 1
                    moved += 1
                    s.copy(pairs)
                    s.move([table], [keep])
                    s.want[seq] = [s.want[seq][k] for k in keep]
            except PagedKVError as e:
                assert "out of KV blocks" in str(e), e
            s.check()
    assert moved > 500 and several > 20 and batches > 20


def compact_together(s, keeps):
    tables, pairs = s.bm.compact_batch(list(keeps), [len(k) for k in keeps.values()])
    s.copy(pairs)
    s.move(tables.tolist(), list(keeps.values()))
    for seq, keep in keeps.items():
        s.want[seq] = [s.want[seq][k] for k in keep]
    s.check()
    return tables, pairs


def test_a_batch_copies_into_no_block_that_it_reads(capi):
    """One sequence's released tail is free when the next one's copies are asked for. With
    nothing else free the batch is refused, and nothing has changed."""
    from paged_kv_cache_59_gb300 import PagedKVError
    for spare in (0, 2):
        s = Server(7 + spare)
        for seq, n in ((1, 80), (2, 32)):
            s.bm.add_seq(seq)
            s.write(seq, n)
        s.bm.fork(2, 3)
        s.want[3] = list(s.want[2])
        keeps = {1: list(range(60, 80)), 3: list(range(3, 31))}
        if spare:
            tables, pairs = compact_together(s, keeps)
            assert len(pairs) == 2 and s.bm.num_free() == 3
            assert not {b for _, b in pairs} & set(tables[0].tolist())
            assert tables[1].tolist()[2:] == [-1] * 3
        else:
            before = [s.bm.block_table(q) for q in (1, 2, 3)]
            with pytest.raises(PagedKVError):
                compact_together(s, keeps)
            assert before == [s.bm.block_table(q) for q in (1, 2, 3)] and s.bm.num_free() == 0
            s.check()


def test_forks_of_one_parent_in_a_batch(capi):
    """The first keeps one block, the second three: what the second moves in place would be
    read by the first, were it not copied."""
    s = Server(20)
    s.bm.add_seq(1)
    s.write(1, 64)
    s.bm.fork(1, 2)
    s.want[2] = list(s.want[1])
    keeps = {1: list(range(33, 49)), 2: list(range(10, 50))}
    _, pairs = compact_together(s, keeps)
    assert len(pairs) == 4


def test_batches_that_are_refused(capi):
    from paged_kv_cache_59_gb300 import PagedKVError
    s = Server(8)
    for seq in (1, 2):
        s.bm.add_seq(seq)
        s.write(seq, 40)
    assert s.bm.compact_batch([], [])[1] == []
    for ids, lens, firsts in (([1, 1], [10, 10], None), ([1, 9], [10, 10], None), ([1, 2], [10, 41], None),
                              ([1, 2], [10, 10], [0, 11]), ([2], [-1], None)):
        with pytest.raises(PagedKVError):
            s.bm.compact_batch(ids, lens, firsts)
    for ids, lens, firsts in (([1], [1, 2], None), ([1], [1], [0, 0])):
        with pytest.raises(ValueError):
            s.bm.compact_batch(ids, lens, firsts)
    s.check()
    tables, pairs = s.bm.compact_batch([1, 2], [40, 0])
    assert pairs == [] and tables.shape == (2, 3)
    assert s.bm.seq_len(1) == 40 and s.bm.seq_len(2) == 0 and s.bm.num_free() == 5
