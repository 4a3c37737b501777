"""Sequences of one manager compacted by one launch, as its tables and copies say: forks of one
parent, cached prompts. Every sequence holds what it kept, bit for bit."""
import numpy as np
import pytest

from tests._gpu import check_device_error, dev, host_bits, torch_cuda

pytestmark = pytest.mark.gpu

HK, D = 2, 64


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def held(pools, table, n):
    t = np.asarray(table)
    return [p[t].transpose(0, 2, 1, 3).reshape(-1, HK, D)[:n] for p in pools]


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("elem", [2, 1])
def test_batches_of_forks_and_cached_prompts(pk, seed, elem):
    torch = torch_cuda()
    rng = np.random.default_rng(seed)
    nb = 92
    kind = np.uint16 if elem == 2 else np.uint8
    pools = [dev(rng.integers(0, np.iinfo(kind).max, (nb, HK, 16, D)).astype(kind)) for _ in range(2)]
    bm = pk.BlockManager(nb, 16)
    prompt = [int(x) for x in rng.integers(0, 1000, 300)]
    bm.add_seq(1)
    bm.append_tokens(1, 300)
    bm.cache_blocks(1, prompt)
    bm.fork(1, 2)
    bm.add_seq_cached(3, prompt)
    bm.add_seq(4)
    bm.append_tokens(4, int(rng.integers(100, 400)))
    bm.add_seq(5)
    bm.append_tokens(5, 60)
    seqs = [int(x) for x in rng.permutation([1, 2, 3, 4, 5])[:4]]

    def content():
        return [host_bits(p) if elem == 2 else p.cpu().numpy() for p in pools]

    before = content()
    want = {s: held(before, bm.block_table(s), bm.seq_len(s)) for s in range(1, 6)}
    keeps = []
    for s in seqs:
        n = bm.seq_len(s)
        keeps.append(np.sort(rng.choice(n, int(rng.integers(0, min(n, 200))), replace=False)).astype(np.int32))
        want[s] = [x[keeps[-1]] for x in want[s]]
    tables, pairs = bm.compact_batch(seqs, [len(k) for k in keeps])
    if pairs:
        pk.pa_copy_blocks(*pools, dev(np.array(pairs, np.int64)))
    pk.pa_compact_blocks(*pools, dev(tables), dev(np.concatenate(keeps)), dev(np.concatenate([[0], np.cumsum([len(k) for k in keeps])]).astype(np.int32)))
    torch.cuda.synchronize()
    after = content()
    for s in range(1, 6):
        got = held(after, bm.block_table(s), bm.seq_len(s)) if bm.seq_len(s) else [np.zeros((0, HK, D), kind)] * 2
        assert all(np.array_equal(a, b) for a, b in zip(got, want[s])), s
    check_device_error(0)
