"""Requests served end to end with reshaped scores and compaction: a prompt with a prefix
read in both directions is written (pa_rope_and_cache) and prefilled, decoded, forked, and
the fork drops tokens (pa_bm_compact, the copies of shared blocks, pa_compact_blocks) while
its parent goes on; both decode on, in one batch, also from a captured graph.

The reference is attention in fp64 over what the cache holds, token by token of the logical
sequence, which is read back before every step; compaction is checked on that: what is
left is what was kept, bit for bit in bf16, and over E4M3 within one more rounding to the
block's new scale (2^-4 of the value, or half a subnormal step, 2^-10 of the scale)."""
import numpy as np
import pytest

from oracle.score_mod import attend
from oracle.sinks import dense_kv
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._score_mod import queries, slopes_of, weight_error
from tests._serving import assert_close
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

H, HK, D, MAXB, NB = 8, 2, 128, 24, 64


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


class Server:
    def __init__(self, pk, kind, cap, slopes):
        torch = torch_cuda()
        self.pk, self.kind, self.cap, self.slopes = pk, kind, cap, slopes
        self.bm = pk.BlockManager(NB, 16)
        dt = torch.int16 if kind == "bf16" else torch.uint8
        self.pools = [torch.full((NB, HK, 16, D), 0x7FC0 if kind == "bf16" else 0x7F, dtype=dt, device="cuda") for _ in range(2)]
        self.scales = None if kind == "bf16" else [torch.full((NB, HK), float("nan"), device="cuda") for _ in range(2)]
        self.sc = {} if kind == "bf16" else dict(k_scale=self.scales[0], v_scale=self.scales[1])
        self.seed = 0

    def append(self, seq, n):
        slots, cow = self.bm.append_tokens(seq, n)
        self.copy(cow)
        self.seed += 1
        rng = np.random.default_rng(self.seed)
        k, v = (dev(f32_to_bf16_bits(rng.standard_normal((n, HK, D)).astype(np.float32))) for _ in range(2))
        at = dev(np.array(slots, np.int64))
        if self.scales:
            self.pk.pa_rope_and_cache_fp8_block(None, None, k, v, *self.pools, *self.scales, None, None, at)
        else:
            self.pk.pa_rope_and_cache(None, None, k, v, *self.pools, None, None, at)

    def copy(self, pairs):
        if pairs:
            m = dev(np.array(pairs, np.int64))
            if self.scales:
                self.pk.pa_copy_blocks_fp8_block(*self.pools, *self.scales, m)
            else:
                self.pk.pa_copy_blocks(*self.pools, m)

    def held(self, seq):
        """K and V of the sequence's tokens, fp64, and each token's scales."""
        tab, n = self.bm.block_table(seq), self.bm.seq_len(seq)
        pools = [host_bits(p) if self.kind == "bf16" else p.cpu().numpy() for p in self.pools]
        scales = [None, None] if self.scales is None else [s.cpu().numpy() for s in self.scales]
        return [dense_kv(p, s, tab, n) for p, s in zip(pools, scales)], scales

    def check(self, got, q, positions, seq, prefix=0, what=""):
        (k, v), _ = self.held(seq)
        scale = D ** -0.5
        ref = attend(q, positions, k, v, scale, self.cap, self.slopes, prefix)
        from oracle.bf16 import bf16_bits_to_f64
        qa = np.abs(bf16_bits_to_f64(q))
        largest = max(float((qa[:, h * 4:(h + 1) * 4].reshape(-1, D) @ np.abs(k[:, h]).T).max()) for h in range(HK)) * scale
        vmax = np.abs(v).max()
        assert_close(got, ref, weight_error(D, largest, self.cap, 2.0 ** -11) + 2.0 ** -14 / vmax, vmax, what)

    def batch(self, seqs):
        tab, ctx = self.bm.build_batch(seqs, MAXB)
        return dev(tab), dev(ctx)

    def mods(self):
        return dict(softcap=self.cap, alibi_slopes=None if self.slopes is None else dev(self.slopes), **self.sc)

    def prefill(self, seq, n, prefix):
        q = queries(self.seed + 100, n, H, D)
        qd = dev(q)
        out = torch_cuda().full_like(qd, 0x7FC0)
        tab, ctx = self.batch([seq])
        self.pk.pa_prefill_score_mod(out, qd, *self.pools, tab, ctx, dev(np.array([0, n], np.int32)), D ** -0.5, n,
                                     prefix_lens=dev(np.array([prefix], np.int32)),
                                     workspace=self.pk.prefill_workspace(qd, 1, HK, n), **self.mods())
        total = self.bm.seq_len(seq)
        self.check(host_bits(out), q, np.arange(total - n, total), seq, prefix, f"prefill of {n}")

    def decode(self, seqs):
        for s in seqs:
            self.append(s, 1)
        q = queries(self.seed + 200, len(seqs), H, D)
        qd = dev(q)
        out = torch_cuda().full_like(qd, 0x7FC0)
        tab, ctx = self.batch(seqs)
        self.pk.pa_decode_score_mod(out, qd, *self.pools, tab, ctx, D ** -0.5, MAXB * 16, partition_tokens=64,
                                    workspace=self.pk.decode_workspace(qd, MAXB * 16, 64), **self.mods())
        got = host_bits(out)
        for i, s in enumerate(seqs):
            self.check(got[i:i + 1], q[i:i + 1], [self.bm.seq_len(s) - 1], s, 0, f"decode of {s}")

    def compact(self, seq, keep):
        """The sequence keeps these positions; the device work in stream order."""
        first = next((j for j, x in enumerate(keep) if x != j), len(keep))
        before, _ = self.held(seq)
        table, pairs = self.bm.compact(seq, len(keep), first)
        self.copy(pairs)
        self.pk.pa_compact_blocks(*self.pools, dev(np.array([table], np.int32)), dev(np.array(keep, np.int32)),
                                  dev(np.array([0, len(keep)], np.int32)), **self.sc)
        after, scales = self.held(seq)
        tab = self.bm.block_table(seq)
        for x in range(2):
            want = before[x][keep]
            if self.kind == "bf16":
                assert np.array_equal(after[x], want)
            else:
                s = scales[x][[tab[j // 16] for j in range(len(keep))]]
                assert (np.abs(after[x] - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s[..., None])).all()
        return len(pairs)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("cap,alibi", [(30.0, False), (0.0, True), (20.0, True)])
def test_prefix_prompt_decode_fork_compact_decode(pk, kind, cap, alibi):
    s = Server(pk, kind, cap, slopes_of(H) if alibi else None)
    s.bm.add_seq(1)
    s.append(1, 150)
    s.prefill(1, 150, 90)
    s.append(1, 37)
    s.prefill(1, 37, 90)
    for _ in range(3):
        s.decode([1])
    s.bm.fork(1, 2)
    rng = np.random.default_rng(9)
    n = s.bm.seq_len(2)
    keep = [0, 1, 2, 3] + sorted(int(x) for x in rng.choice(np.arange(4, n - 30), 60, replace=False)) + list(range(n - 30, n))
    free = s.bm.num_free()
    parent, _ = s.held(1)
    copies = s.compact(2, keep)
    assert copies == 6 and s.bm.num_free() == free - 6           # 94 tokens in private blocks
    assert all(np.array_equal(a, b) for a, b in zip(s.held(1)[0], parent))
    for _ in range(4):
        s.decode([1, 2])
    assert s.compact(1, list(range(s.bm.seq_len(1) - 50, s.bm.seq_len(1)))) == 0
    s.decode([2, 1])
    assert s.bm.seq_len(1) == 51 and len(s.bm.block_table(1)) == 4
    s.bm.free_seq(1), s.bm.free_seq(2)
    assert s.bm.num_free() == NB
    check_device_error(0)


def test_a_captured_step_compacts_and_decodes(pk):
    """Compaction and the decode behind it in one graph, on two caches with a workspace
    each, replayed one after the other and at the same time."""
    torch = torch_cuda()
    rng = np.random.default_rng(11)
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        pools = [dev(f32_to_bf16_bits(rng.standard_normal((40, HK, 16, D)).astype(np.float32))) for _ in range(2)]
        start = [p.clone() for p in pools]
        table = dev(np.arange(40, dtype=np.int32)[::-1].copy()[None])
        keep = np.sort(rng.choice(600, 300, replace=False)).astype(np.int32)
        q = queries(i, 1, H, D)
        qd, out = dev(q), torch.zeros((1, H, D), dtype=torch.int16, device="cuda")
        ctx, kd, loc = dev(np.array([300], np.int32)), dev(keep), dev(np.array([0, 300], np.int32))
        ws = pk.decode_workspace(qd, 640, 64)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for a, b in zip(pools, start):
                a.copy_(b)
            pk.pa_compact_blocks(*pools, table, kd, loc)
            pk.pa_decode_score_mod(out, qd, *pools, table, ctx, D ** -0.5, 640, softcap=25.0, workspace=ws, partition_tokens=64)
        k, v = (dense_kv(host_bits(p), None, table.cpu().numpy()[0], 600)[keep] for p in start)
        graphs.append((g, out, attend(q, [299], k, v, D ** -0.5, 25.0), np.abs(v).max(), (qd, pools, start, table, ctx, kd, loc, ws)))
    for rounds in range(6):
        for i, (g, out, *_r) in enumerate(graphs):
            if rounds < 3:
                g.replay()
                torch.cuda.synchronize()
            else:
                with torch.cuda.stream(streams[i]):
                    g.replay()
        torch.cuda.synchronize()
        for g, out, ref, vmax, _keep in graphs:
            assert_close(host_bits(out), ref, weight_error(D, 100.0, 25.0, 2.0 ** -16), vmax)
            out.zero_()
    check_device_error(0)
