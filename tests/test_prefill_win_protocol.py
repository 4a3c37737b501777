"""The windowed prefill's protocols, on the CPU.

``run`` replays the roles of pa_prefill_win_kernel - K and V producers (one warp
for both with an E4M3 cache), four converter warps, the MMA thread and its
in-order tensor core, two warpgroups of four softmax warps - over several
segments, with their mbarrier waits, parities and named barriers, in random
interleavings. For every schedule it draws it checks that

- a parity wait passes only when the phase it means has completed (a wait two
  phases behind passes at once on the hardware);
- the run ends;
- each Q.K^T reads the Q of its segment and the K tile it names, each P.V the V
  tile it names and the P of all four warps, and none of them is overwritten
  while it is read; a softmax warp reads the S of its tile and, at a segment's
  end, the O of that segment.

``plan`` is the work list's arithmetic (pa_prefill_plan_even_kernel): every item's
tiles exactly once and in order, one piece of an item a CTA, distinct slots, and
the table that join_pieces reads. The stage counts and constants are read from
the kernel's source.
"""
import os
import random
import re

import pytest

from tests.conftest import ROOT

SRC = open(os.path.join(ROOT, "paged_kv_cache_59_gb300", "csrc", "prefill_win.cuh")).read()


def stages(EB):
    ks = int(re.search(r"constexpr int kKS = (\d+);", SRC).group(1))
    vs = re.search(r"constexpr int kVS = EB == 2 \? (\d+) : (\d+);", SRC)
    return ks, int(vs.group(1 if EB == 2 else 2))


class Bar:
    def __init__(self, n):
        self.n = self.left = n
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.n
            self.phase += 1

    def passes(self, parity):
        return (self.phase & 1) != parity


def run(segs, EB, rng, q_wait="q_free"):
    kKS, kVS = stages(EB)
    B = {}
    for i in range(kKS):
        B["k_full", i], B["k_conv", i], B["k_free", i] = Bar(1), Bar(4), Bar(1)
    for i in range(kVS):
        B["v_full", i], B["v_conv", i], B["v_free", i] = Bar(1), Bar(4), Bar(1)
    for i in range(2):
        B["raw_free", i], B["s_full", i], B["pv_done", i] = Bar(4), Bar(1), Bar(1)
    B["q_full", 0], B["q_free", 0] = Bar(4), Bar(1)
    named = [dict(soft=0, mma=0) for _ in range(2)]
    mem, queue, loads = {"Q": {}, ("P", 0): {}, ("P", 1): {}}, [], []

    def wait(name, i, parity, phase):
        while not B[name, i].passes(parity):
            yield
        assert B[name, i].phase > phase, (name, i, "passed early")

    def producer(operands):
        ring = {x: [0, 1, 0] for x in operands}  # stage, parity, fills
        J = 0
        for n in segs:
            for _ in range(n):
                for x in operands:
                    st, ph, fills = ring[x]
                    N = 1 if EB == 1 else (kVS if x else kKS)
                    name, i = ("raw_free", x) if EB == 1 else (("v_free", "k_free")[x == 0], st)
                    yield from wait(name, i, ph, fills // N - 1)
                    loads.append((("raw", x) if EB == 1 else ("KV"[x], st), J, (("k_full", "v_full")[x], 0 if EB == 1 else st)))
                    yield
                    st += 1
                    ring[x] = [st % N, ph ^ (st == N), fills + 1]
                J += 1

    def mma():
        J0 = 0
        kc = vc = 0
        k_ready = "k_full" if EB == 2 else "k_conv"
        for seg, n in enumerate(segs):
            yield from wait("q_full", 0, seg & 1, seg)
            yield from wait(k_ready, kc % kKS, kc // kKS & 1, kc // kKS)
            queue.extend(("qk", x, kc % kKS, J0, seg) for x in (0, 1))
            if n == 1:
                queue.append(("q_free",))
            kc += 1
            for j in range(n):
                more = j + 1 < n
                yield from wait("v_conv", vc % kVS, vc // kVS & 1, vc // kVS)
                if more:
                    yield from wait(k_ready, kc % kKS, kc // kKS & 1, kc // kKS)
                for x in (0, 1):
                    named[x]["mma"] += 1
                    while named[x]["soft"] < 4 * named[x]["mma"]:
                        yield
                    queue.append(("pv", x, vc % kVS, J0 + j, seg))
                    if more:
                        queue.append(("qk", x, kc % kKS, J0 + j + 1, seg))
                    if x == 1 and j + 2 == n:
                        queue.append(("q_free",))
                    yield
                vc += 1
                kc += more
            J0 += n

    def converter(w):
        J0 = 0
        for seg, n in enumerate(segs):
            if seg > 0 and q_wait == "q_free":
                yield from wait("q_free", 0, (seg - 1) & 1, seg - 1)
            elif seg > 0:
                yield from wait("s_full", 1, (J0 - 1) & 1, J0 - 1)
            mem["Q"][w] = seg
            yield
            B["q_full", 0].arrive()
            for J in range(J0, J0 + n):
                if EB == 2:
                    yield from wait("v_full", J % kVS, J // kVS & 1, J // kVS)
                    assert mem["V", J % kVS] == J
                    yield
                    B["v_conv", J % kVS].arrive()
                    continue
                for x, S, free, conv in ((0, kKS, "k_free", "k_conv"), (1, kVS, "v_free", "v_conv")):
                    yield from wait(("k_full", "v_full")[x], 0, J & 1, J)
                    if J >= S:
                        yield from wait(free, J % S, (J - S) // S & 1, (J - S) // S)
                    assert mem["raw", x] == J
                    yield
                    mem["KV"[x], J % S] = J
                    B["raw_free", x].arrive()
                    B[conv, J % S].arrive()
            J0 += n

    def softmax(x, w):
        J0 = 0
        for seg, n in enumerate(segs):
            for J in range(J0, J0 + n):
                yield from wait("s_full", x, J & 1, J)
                assert mem["S", x] == J
                yield
                if J > J0 and rng.random() < 0.3:  # a new reference rescales O
                    yield from wait("pv_done", x, (J - 1) & 1, J - 1)
                mem["P", x][w] = J
                named[x]["soft"] += 1
                # a named barrier has no phases: nobody may be a whole round ahead of the MMA warp
                assert named[x]["soft"] <= 4 * (named[x]["mma"] + 1)
                yield
            J0 += n
            yield from wait("pv_done", x, (J0 - 1) & 1, J0 - 1)
            for _ in range(2):  # the epilogue reads O
                assert mem["O", x] == (seg, J0 - 1)
                yield

    def tensor_core():
        while True:
            if queue:
                op = queue.pop(0)
                if op[0] == "q_free":
                    B["q_free", 0].arrive()
                elif op[0] == "qk":
                    _, x, st, J, seg = op
                    for _ in range(2):
                        assert mem["K", st] == J and all(mem["Q"][w] == seg for w in range(4)), op
                        yield
                    mem["S", x] = J
                    if x == 1:
                        B["k_free", st].arrive()
                    B["s_full", x].arrive()
                else:
                    _, x, st, J, seg = op
                    for _ in range(2):
                        assert mem["V", st] == J and all(mem["P", x][w] == J for w in range(4)), op
                        yield
                    mem["O", x] = (seg, J)
                    if x == 1:
                        B["v_free", st].arrive()
                    B["pv_done", x].arrive()
            yield

    def tma():
        while True:
            if loads:
                where, J, bar = loads.pop(rng.randrange(len(loads)))
                mem[where] = J
                B[bar].arrive()
            yield

    live = [producer([0]), producer([1])] if EB == 2 else [producer([0, 1])]
    live += [mma()] + [converter(w) for w in range(4)] + [softmax(x, w) for x in (0, 1) for w in range(4)]
    slow = rng.choice(live)  # one role that rarely runs
    hardware = [tensor_core(), tma()]
    for step in range(20000 + 20000 * sum(segs)):
        if not live:
            return
        g = rng.choice(live + hardware)
        if g is slow and rng.random() < 0.9:
            continue
        try:
            next(g)
        except StopIteration:
            live.remove(g)
    raise AssertionError("stuck")


@pytest.mark.parametrize("EB", [2, 1])
@pytest.mark.parametrize("seed", range(6))
def test_roles_hold_under_random_schedules(EB, seed):
    rng = random.Random(seed)
    for _ in range(25):
        run([rng.choice([1, 1, 2, 3, rng.randint(1, 9)]) for _ in range(rng.randint(1, 6))], EB, rng)


def test_a_mutated_protocol_is_caught():
    """Q's reload gated by the last tile's S, a barrier that can be two phases
    behind, instead of by the segment's last Q.K^T."""
    rng = random.Random(0)
    with pytest.raises(AssertionError):
        for _ in range(60):
            run([rng.randint(1, 5) for _ in range(5)], 2, rng, q_wait="s_full")


def test_named_barriers_balance():
    """Every key tile: one arrive of each softmax warp, one sync of the MMA warp a
    query tile, in loops that a failed wait does not leave."""
    src = re.sub(r"//[^\n]*", "", SRC)
    syncs = re.findall(r"bar\.sync (\d), (\d+);", src)
    arrives = re.findall(r"bar\.arrive %0, (\d+);", src)
    assert sorted(i for i, _ in syncs) == ["1", "2"] and arrives == ["160"] and {c for _, c in syncs} == {"160"}
    covered = 0
    for m in re.finditer(r"for \(int j = 0; j < g\.n_kt; \+\+j\) \{", src):
        depth, k = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[k], 0)
            k += 1
        body = src[m.end():k]
        n = len(re.findall(r"bar\.(?:sync|arrive) ", body))
        if n:
            covered += n
            assert not re.search(r"\b(break|continue)\b", body)
    assert covered == 3


# ------------------------------------------------------------- work list

K_START, K_LEAST = (int(x) for x in re.search(r"constexpr int kStart = (\d+), kLeast = (\d+);", SRC).groups())


def plan(nks, n_cta):
    n, T = len(nks), sum(k + K_START for k in nks if k > 0)
    count, most = sum(k > 0 for k in nks), max(nks + [0])
    work, cta = {}, [[0x7fffffff, 0, -1, 0] for _ in range(n_cta)]
    if count <= n_cta and most <= T // n_cta + 2 * K_START:
        for r, (it, k) in enumerate((it, k) for it, k in enumerate(nks) if k > 0):
            work[r], cta[r] = (it, 0, k, -1), [r, r + 1, -1, 0]
        return work, cta
    C, off, r = max(1, min(n_cta, T // (K_START + 4))), 0, 0
    for it, k in enumerate(nks):
        if k <= 0:
            continue
        c0, c1 = ((off + 1) * C - 1) // T, ((off + k + K_START) * C - 1) // T

        def cut(c):
            if c <= c0:
                return 0
            if c > c1:
                return k
            x = c * T // C - off - K_START
            return 0 if x < K_LEAST else k if x > k - K_LEAST else x

        ca, cb = c0, c1
        while cut(ca + 1) == 0:
            ca += 1
        while cut(cb) == k:
            cb -= 1
        assert c0 <= ca <= cb <= c1 < C
        for c in range(ca, cb + 1):
            assert r + c not in work and r + c < n + n_cta
            work[r + c] = (it, cut(c), cut(c + 1), -1 if ca == cb else 2 * c + 1 if c == ca else 2 * c)
            cta[c][0], cta[c][1] = min(cta[c][0], r + c), max(cta[c][1], r + c + 1)
            if c > ca:
                assert cta[c][2] == -1
                cta[c][2:] = [ca, cb - ca + 1]
        off, r = off + k + K_START, r + 1
    return work, cta


def test_work_list_covers_every_tile_once():
    R = random.Random(1)
    for _ in range(1500):
        n_cta = R.choice([1, 2, 7, 152])
        nks = [R.choice([0, 1, 2, 3, R.randint(0, 60), R.randint(0, 5)]) for _ in range(R.randint(1, R.choice([3, 40, 700])))]
        if R.random() < 0.2:
            nks = [R.randint(0, 1500)]
        work, cta = plan(nks, n_cta)
        got, slots = {}, set()
        for c, (first, end, _, _) in enumerate(cta):
            for w in range(first, end):
                it, a, b, slot = work[w]
                assert a < b
                got.setdefault(it, []).append((a, b, slot, c))
                if slot >= 0:
                    assert slot not in slots and slot < 2 * n_cta
                    slots.add(slot)
        for it, k in enumerate(nks):
            pieces = sorted(got.get(it, []))
            assert (k == 0) == (not pieces)
            if not k:
                continue
            assert pieces[0][0] == 0 and pieces[-1][1] == k and all(x[1] == y[0] for x, y in zip(pieces, pieces[1:]))
            if len(pieces) == 1:
                assert pieces[0][2] == -1
                continue
            ca = pieces[0][3]
            for i, (_, _, slot, c) in enumerate(pieces):
                assert slot == (2 * ca + 1 if i == 0 else 2 * (ca + i)) and slot >> 1 == c
                info = cta[c + 1 if slot & 1 else c]          # what join_pieces reads
                assert info[2] == ca and info[3] == len(pieces) and c - ca == i
                assert (ca + 1) * 8 + 7 < n_cta * 8           # its counter


def test_work_list_is_even():
    """Equal items on 152 CTAs: no CTA has more than a run's length and one start
    above the mean."""
    for n, k in ((256, 35), (400, 12), (153, 90), (1000, 6)):
        work, cta = plan([k] * n, 152)
        cost = [sum(work[w][2] - work[w][1] + K_START for w in range(f, e)) for f, e, _, _ in cta]
        mean = sum([k + K_START] * n) / 152
        assert max(cost) <= mean + K_START + 2 * K_LEAST
