"""A request served end to end with the rotated cache write, the windowed or
block-scaled attention and the block manager: a prompt prefilled in chunks,
decode steps, blocks released between the sinks and the window, a fork that
copies a block with its scales, and a decode step replayed from a CUDA graph.

The reference holds the logical sequence in fp64: k rotated by its position and
v, as the cache holds them (bf16, or E4M3 with the scale the block had when the
token was last encoded), which is read back from the cache; what is checked is
that every step attends to exactly the right tokens at the right places. Reading
back is itself checked against the fp64 rotation within one rounding of the cache
type: bf16 2^-8, E4M3 2^-4 of the value, or half a subnormal step of the block's
scale, 2^-10, once more for each time the scale grew (three at most here)."""
import numpy as np
import pytest

from oracle.bf16 import bf16_bits_to_f64
from oracle.fp8 import e4m3_to_f64
from oracle.rope_cache import rotate_f32, rotate_f64
from oracle.sinks import attend_rows
from tests._gpu import check_device_error, dev, host_bits, torch_cuda
from tests._serving import assert_close
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

H, HK, D, WINDOW, SINKS, MAXB, NB = 8, 2, 128, 70, 5, 24, 64


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


def table():
    a = np.arange(512)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Server:
    def __init__(self, pk, kind):
        torch = torch_cuda()
        self.pk, self.kind = pk, kind
        self.bm = pk.BlockManager(NB, 16)
        dt = torch.int16 if kind == "bf16" else torch.uint8
        self.pools = [torch.full((NB, HK, 16, D), 0x7F if kind != "bf16" else 0x7FC0, dtype=dt, device="cuda") for _ in range(2)]
        self.scales = [torch.full((NB, HK), float("nan"), device="cuda") for _ in range(2)] if kind != "bf16" else None
        self.cs = table()
        self.cs_dev = dev(self.cs)
        self.rng = np.random.default_rng(3)
        self.seqs = {}

    def tokens(self, n):
        return [f32_to_bf16_bits(self.rng.standard_normal((n, h, D)).astype(np.float32)) for h in (H, HK, HK)]

    def append(self, seq, n):
        """Takes n new tokens of seq into the cache; the device q, rotated."""
        torch = torch_cuda()
        first = len(self.seqs.setdefault(seq, ([], []))[0])
        slots, cow = self.bm.append_tokens(seq, n)
        if cow:
            m = dev(np.array(cow, np.int64))
            if self.scales:
                self.pk.pa_copy_blocks_fp8_block(*self.pools, *self.scales, m)
            else:
                self.pk.pa_copy_blocks(*self.pools, m)
        q, k, v = self.tokens(n)
        pos = np.arange(first, first + n)
        for i in range(n):
            self.seqs[seq][0].append(rotate_f64(k[i:i + 1], self.cs, pos[i:i + 1])[0])
            self.seqs[seq][1].append(bf16_bits_to_f64(v[i]))
        qd, kd, vd = dev(q), dev(k), dev(v)
        out = torch.empty_like(qd)
        a = (self.cs_dev, dev(pos), dev(np.array(slots, np.int64)))
        if self.scales:
            self.pk.pa_rope_and_cache_fp8_block(out, qd, kd, vd, *self.pools, *self.scales, *a)
        else:
            self.pk.pa_rope_and_cache(out, qd, kd, vd, *self.pools, *a)
        assert np.array_equal(host_bits(out), f32_to_bf16_bits(rotate_f32(q, self.cs, pos)))
        return out

    def release(self, seq):
        """Drops what no later query sees."""
        return self.bm.release_between(seq, SINKS, max(SINKS, len(self.seqs[seq][0]) - WINDOW))

    def held(self, seq):
        """The sequence's K and V as the cache holds them, NaN where released."""
        table_ = self.bm.block_table(seq)
        got = []
        for x in range(2):
            pool = self.pools[x].cpu().numpy()
            rows = []
            for b in table_:
                if b < 0:
                    rows.append(np.full((16, HK, D), np.nan))
                elif self.scales:
                    s = self.scales[x].cpu().numpy()[b].astype(np.float64)
                    rows.append(np.moveaxis(e4m3_to_f64(pool[b]) * s[:, None, None], 0, 1))
                else:
                    rows.append(np.moveaxis(bf16_bits_to_f64(pool[b].view(np.uint16)), 0, 1))
            n = len(self.seqs[seq][0])
            held = np.concatenate(rows)[:n]
            true = np.array(self.seqs[seq][x])
            ok = ~np.isnan(held)
            if self.scales:
                s = np.concatenate([np.full((16, HK), np.nan) if b < 0 else
                                    np.tile(self.scales[x].cpu().numpy()[b], (16, 1)) for b in table_])[:n][..., None]
                bound = np.maximum(2.0 ** -4 * np.abs(true) * 1.001, 4 * 2.0 ** -10 * np.broadcast_to(s, true.shape))
            else:
                bound = 2.0 ** -8 * np.abs(true) * 1.001 + 2.0 ** -22
            assert (np.abs(held - true)[ok] <= bound[ok]).all()
            got.append(held)
        return got

    def batch(self, ids):
        t, c = self.bm.build_batch(ids, MAXB)
        return dev(t), dev(c), c

    def check(self, out, q, rows):
        """rows: (sequence, first position, count) of out's rows in order."""
        at = 0
        for seq, p, n in rows:
            k, v = self.held(seq)
            qh = host_bits(q[at:at + n].contiguous())
            ref = attend_rows(qh, range(p, p + n), k, v, D ** -0.5, WINDOW, SINKS)
            # weights: fp16 P (2^-11) and 2^-12 for the scores of these unit normals
            assert_close(host_bits(out[at:at + n].contiguous()), ref, 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -17, float(np.nanmax(np.abs(v))))
            at += n

    def prefill(self, chunks):
        """chunks: (sequence, tokens)."""
        torch = torch_cuda()
        qs = [self.append(s, n) for s, n in chunks]
        q = torch.cat(qs)
        out = torch.zeros_like(q)
        tab, ctx, _ = self.batch([s for s, _ in chunks])
        lens = [n for _, n in chunks]
        loc = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        ws = self.pk.prefill_workspace(q, len(chunks), HK, max(lens))
        if self.scales:
            self.pk.pa_prefill_fp8_block(out, q, *self.pools, *self.scales, tab, ctx, loc, D ** -0.5, max(lens),
                                         window=WINDOW, n_sinks=SINKS, workspace=ws)
        else:
            self.pk.pa_prefill_sinks(out, q, *self.pools, tab, ctx, loc, D ** -0.5, max(lens), WINDOW, SINKS, workspace=ws)
        self.check(out, q, [(s, len(self.seqs[s][0]) - n, n) for s, n in chunks])

    def decode(self, ids):
        torch = torch_cuda()
        q = torch.cat([self.append(s, 1) for s in ids])
        out = torch.zeros_like(q)
        tab, ctx, c = self.batch(ids)
        ws = self.pk.decode_workspace(q, int(c.max()))
        if self.scales:
            self.pk.pa_decode_fp8_block(out, q, *self.pools, *self.scales, tab, ctx, D ** -0.5, int(c.max()),
                                        window=WINDOW, n_sinks=SINKS, workspace=ws)
        else:
            self.pk.pa_decode_sinks(out, q, *self.pools, tab, ctx, D ** -0.5, int(c.max()), WINDOW, SINKS, workspace=ws)
        self.check(out, q, [(s, len(self.seqs[s][0]) - 1, 1) for s in ids])


@pytest.mark.parametrize("kind", ["bf16", "block"])
def test_serving_run(pk, kind):
    sv = Server(pk, kind)
    for s in (1, 2):
        sv.bm.add_seq(s)
    sv.prefill([(1, 50), (2, 21)])
    sv.prefill([(1, 77), (2, 1)])
    assert sv.release(1) > 0
    for _ in range(5):
        sv.decode([1, 2])
    sv.bm.fork(2, 3)                       # aliases the partly filled block
    sv.seqs[3] = tuple(list(x) for x in sv.seqs[2])
    for _ in range(20):
        sv.decode([1, 2, 3])
        sv.release(1)
    sv.prefill([(3, 90), (1, 30)])
    sv.release(3)
    sv.decode([3, 1, 2])
    free = sv.bm.num_free()
    for s in (1, 2, 3):
        sv.bm.free_seq(s)
    assert sv.bm.num_free() == NB and free < NB
    check_device_error(0)


@pytest.mark.parametrize("kind", ["bf16", "block"])
def test_decode_step_from_a_graph(pk, kind):
    """Append, decode and the copy of the step's inputs captured once and replayed
    for several tokens: only the contents of the inputs change."""
    torch = torch_cuda()
    sv = Server(pk, kind)
    sv.bm.add_seq(1)
    sv.prefill([(1, 40)])
    qkv = torch.zeros((1, H + 2 * HK, D), dtype=torch.int16, device="cuda")
    pos, slot = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    tab, ctx = torch.full((1, MAXB), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = qkv[:, :H], qkv[:, H:H + HK], qkv[:, H + HK:]
    rot, out = (torch.zeros((1, H, D), dtype=torch.int16, device="cuda") for _ in range(2))
    ws = pk.decode_workspace(rot, 16 * MAXB, 64)

    def step():
        if sv.scales:
            pk.pa_rope_and_cache_fp8_block(rot, q, k, v, *sv.pools, *sv.scales, sv.cs_dev, pos, slot)
            pk.pa_decode_fp8_block(out, rot, *sv.pools, *sv.scales, tab, ctx, D ** -0.5, 16 * MAXB, window=WINDOW,
                                   n_sinks=SINKS, workspace=ws, partition_tokens=64)
        else:
            pk.pa_rope_and_cache(rot, q, k, v, *sv.pools, sv.cs_dev, pos, slot)
            pk.pa_decode_sinks(out, rot, *sv.pools, tab, ctx, D ** -0.5, 16 * MAXB, WINDOW, SINKS, workspace=ws,
                               partition_tokens=64)

    slot.fill_(-1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(40):
        n = len(sv.seqs[1][0])
        slots, _ = sv.bm.append_tokens(1, 1)
        hq, hk, hv = sv.tokens(1)
        sv.seqs[1][0].append(rotate_f64(hk, sv.cs, [n])[0])
        sv.seqs[1][1].append(bf16_bits_to_f64(hv[0]))
        qkv.copy_(dev(np.concatenate([hq, hk, hv], 1)))
        pos.fill_(n), slot.fill_(slots[0])
        t, c, _ = sv.batch([1])
        tab.copy_(t), ctx.copy_(c)
        g.replay()
        sv.check(out, rot, [(1, n, 1)])
        sv.release(1)
    check_device_error(0)


def test_copy_blocks_with_their_scales(pk):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    for hk, d in ((3, 64), (8, 128), (300, 64)):
        pools = [torch.randint(0, 256, (9, hk, 16, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        scales = [torch.rand((9, hk), generator=g, device="cuda") for _ in range(2)]
        want = [x.clone() for x in pools + scales]
        pairs = torch.tensor([[0, 4], [1, 5], [0, 8]], device="cuda")
        for x in want:
            for a, b in pairs.tolist():
                x[b] = x[a]
        pk.pa_copy_blocks_fp8_block(*pools, *scales, pairs)
        assert all(torch.equal(a, b) for a, b in zip(pools + scales, want))
        pk.pa_copy_blocks_fp8_block(*pools, *scales, pairs[:0])
        check_device_error(0)
        pk.pa_copy_blocks_fp8_block(*pools, *scales, torch.tensor([[9, 0], [0, -1]], device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(pools + scales, want))
        check_device_error(8)
    with pytest.raises(ValueError):
        pk.pa_copy_blocks_fp8_block(*pools, scales[0][:2], scales[1], pairs)
