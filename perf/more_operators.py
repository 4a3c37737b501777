"""Attention with reshaped scores over the paged cache, and the compaction of a cache, as a
timing harness measures them:

  decode   one query per sequence: scores capped by a tanh, biased by distance, or both,
           over all of the cache or a sliding window with sinks
  prefill  a chunk of queries per sequence over the same scores, also under a prefix mask
           (a row sees the keys of its sequence's prefix, later ones too)
  compact  the tokens of a sequence that stay move to its first positions, in place

With ``own`` false ``run`` computes each in elementary torch operations in 32 bits;
with ``own`` true it calls the library.

Conventions: a block holds 16 tokens; pools are [blocks][kv_heads][16][head_dim]; an
E4M3 element stands for code * scale[block][kv_head]. With s = scale * (q . k) the score
of key t for a query at position i is cap * tanh(s / cap) - slope[head] * |i - t| (cap 0:
s; no slopes: no bias). t is visible when t <= i or t < prefix, and, under a window, when
t >= i - window or t < sinks. Compaction gives position j what position keep[j] held; a
block of an E4M3 cache takes the largest of its new tokens' scales.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BS = 16
DEV = "cuda"


# ------------------------------------------------------------------- cases

def _attention(op, name, cache, heads, kv, dim, seqs, ctx_lo, ctx_hi, cap, alibi, window=-1, sinks=0, chunk_lo=1, chunk_hi=1,
               prefix=False, spread=6.0):
    return dict(name=name, op=op, cache=cache, heads=heads, kv=kv, dim=dim, seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, cap=cap,
                alibi=alibi, window=window, sinks=sinks, chunk_lo=chunk_lo, chunk_hi=chunk_hi, prefix=prefix, spread=spread)


def _compaction(name, cache, kv, dim, seqs, ctx_lo, ctx_hi, part, per_head):
    return dict(name=name, op="compact", cache=cache, kv=kv, dim=dim, seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, part=part,
                per_head=per_head)


def listed():
    return [
        # one short stream of a small model with capped scores: latency
        _attention("decode", "decode one stream cap bf16", "bf16", 8, 4, 64, 1, 333, 333, 50.0, False),
        # a serving batch of an 8B-shaped model with capped scores
        _attention("decode", "decode batch cap bf16", "bf16", 32, 8, 128, 64, 128, 4096, 50.0, False),
        # a batch of a 7B-shaped model with a head of keys for each query head and distance biases
        _attention("decode", "decode batch alibi bf16", "bf16", 32, 32, 128, 16, 700, 2048, 0.0, True, spread=2.0),
        # few long documents, 70B-shaped, capped, half the cache's bytes
        _attention("decode", "decode long cap e4m3", "e4m3", 64, 8, 128, 4, 99999, 131072, 30.0, False),
        # one ragged prompt of a small model: latency
        _attention("prefill", "prefill short cap bf16", "bf16", 8, 4, 64, 1, 77, 77, 50.0, False, chunk_lo=77, chunk_hi=77),
        # a chunk of a long prompt in a layer that sees a window, capped
        _attention("prefill", "prefill window cap bf16", "bf16", 32, 8, 128, 1, 16384, 16384, 50.0, False, window=4095,
                   chunk_lo=2048, chunk_hi=2048),
        # ragged chunks with distance biases, a head of keys for each query head
        _attention("prefill", "prefill ragged alibi bf16", "bf16", 32, 32, 128, 5, 300, 4096, 0.0, True, chunk_lo=33,
                   chunk_hi=777, spread=2.0),
        # prompts that begin with a prefix read in both directions, over E4M3, capped
        _attention("prefill", "prefill prefix cap e4m3", "e4m3", 32, 8, 128, 3, 1024, 2500, 30.0, False, chunk_lo=900,
                   chunk_hi=2048, prefix=True),
        # one short chat drops half of its tokens: latency
        _compaction("compact one chat bf16", "bf16", 8, 128, 1, 700, 700, 0.5, False),
        # a batch of chats keeps a third of its tokens, each KV head its own
        _compaction("compact batch per head bf16", "bf16", 8, 128, 32, 2000, 8192, 0.33, True),
        # one long document, where few sequences have to fill the machine
        _compaction("compact one document bf16", "bf16", 8, 128, 1, 131072, 131072, 0.6, False),
        # long documents in an E4M3 cache: blocks change their scales
        _compaction("compact documents e4m3", "e4m3", 8, 128, 6, 20000, 65536, 0.4, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128])
    case = dict(op=rng.choice(["decode", "prefill", "compact"]), cache=rng.choice(["bf16", "e4m3"]), kv=kv, dim=dim,
                lens_seed=rng.randrange(1 << 20))
    if case["op"] == "compact":
        ctx = _log_int(rng, 1, 65536)
        case.update(seqs=_log_int(rng, 1, max(1, min(128, 196608 // ctx))), ctx_lo=rng.randint(0, ctx), ctx_hi=ctx,
                    part=rng.choice([0.05, 0.3, 0.5, 0.8, 1.0]), per_head=rng.random() < 0.5)
        return case
    heads = kv * rng.choice([1, 2, 4, 8])
    windowed = rng.random() < 0.4
    case.update(heads=heads, cap=rng.choice([0.0, 20.0, 30.0, 50.0]), window=_log_int(rng, 1, 4096) if windowed else -1,
                sinks=rng.choice([0, 0, 1, 5, 33]) if windowed else 0, chunk_lo=1, chunk_hi=1, prefix=False,
                spread=rng.choice([1.0, 2.0, 6.0]))
    case["alibi"] = case["cap"] == 0.0 or rng.random() < 0.3
    if case["op"] == "decode":
        ctx = _log_int(rng, 1, 65536)
        case.update(seqs=_log_int(rng, 1, max(1, min(128, 196608 // ctx))), ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    else:
        chunk = _log_int(rng, 1, 1024)
        ctx = _log_int(rng, chunk, 6144)
        case.update(seqs=_log_int(rng, 1, max(1, min(8, 65536 // (chunk * heads)))), chunk_lo=rng.randint(1, chunk),
                    chunk_hi=chunk, ctx_lo=rng.randint(chunk, ctx), ctx_hi=ctx, prefix=rng.random() < 0.4)
    return case


def _lens(case):
    """(new tokens or kept ones, context, prefix) of each sequence, from the case alone."""
    r = random.Random(case.get("lens_seed", 11) * 1000003 + case["seqs"])
    got = []
    for _ in range(case["seqs"]):
        if case["op"] == "prefill":
            n = r.randint(case["chunk_lo"], case["chunk_hi"])
            c = max(n, r.randint(case["ctx_lo"], case["ctx_hi"]))
        else:
            c = r.randint(case["ctx_lo"], case["ctx_hi"])
            n = 1 if case["op"] == "decode" else min(c, int(math.ceil(c * case["part"])))
        got.append((n, c, r.randint(0, c) if case.get("prefix") else 0))
    return got


def _seen(case, p, prefix):
    """Positions that a query at position p attends to."""
    end = max(p + 1, prefix)
    first = max(0, p - case["window"]) if case["window"] >= 0 else 0
    return end - first + min(case["sinks"], first)


def work(case):
    kv, d = case["kv"], case["dim"]
    eb = 2 if case["cache"] == "bf16" else 1
    lens = _lens(case)
    if case["op"] == "compact":
        # the kept tokens that move (all, to within the first few) read and written, K and V, and the lists
        kept = sum(n for n, c, _ in lens if n < c)
        lists = 4 * kept * (kv if case["per_head"] else 1)
        scales = 16 * kv * sum((n + BS - 1) // BS for n, c, _ in lens if n < c) if eb == 1 else 0
        return {"bytes": max(1, 4 * eb * kept * kv * d + lists + scales), "flops": 0}
    h = case["heads"]
    rows = sum(n for n, _, _ in lens)
    read, pairs = [], 0
    for n, c, x in lens:
        if c == 0:
            continue
        lo = max(0, c - n - case["window"]) if case["window"] >= 0 else 0
        read.append(c - lo + min(case["sinks"], lo))
        pairs += sum(_seen(case, p, x) for p in range(c - n, c))
    blocks = sum((r + BS - 1) // BS for r in read)
    b = sum(read) * kv * d * 2 * eb + (blocks * kv * 8 if eb == 1 else 0) + rows * h * d * 4 + blocks * 4
    return {"bytes": b, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ inputs

def _power_scale(amax):
    """The smallest 2^e with amax <= 448 * 2^e (448 = 0.875 * 2^9), e >= -32."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-32, 32)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _pool(case, num_blocks, gen):
    """A filled cache: (k_pool, v_pool, k_scale, v_scale); scales are None in bf16."""
    shape = (num_blocks, case["kv"], BS, case["dim"])
    got, scales = [], []
    for _ in range(2):
        if case["cache"] == "bf16":
            x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
            got.append(x.normal_(generator=gen))
            scales.append(None)
            continue
        codes = torch.empty(shape, dtype=torch.uint8, device=DEV)
        scale = torch.empty(shape[:2], dtype=torch.float32, device=DEV)
        for a in range(0, num_blocks, 8192):  # the blocks of a long cache a slice at a time
            n = min(8192, num_blocks - a)
            x = torch.randn((n,) + shape[1:], generator=gen, device=DEV)
            # blocks and heads differ in magnitude
            x *= torch.exp2(torch.randn((n, case["kv"], 1, 1), generator=gen, device=DEV) * 0.7)
            scale[a:a + n] = _power_scale(x.abs().amax(dim=(2, 3)))
            codes[a:a + n] = (x / scale[a:a + n, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        got.append(codes)
        scales.append(scale)
    return got[0], got[1], scales[0], scales[1]


def _keep_list(case, lens, gen):
    """int32 [heads or 1][kept tokens]: of each sequence the first four tokens, the newest quarter of what stays,
    and tokens between picked at random; ascending."""
    rows = case["kv"] if case["per_head"] else 1
    parts = []
    for n, c, _ in lens:
        if n == 0:
            continue
        u = torch.rand((rows, c), generator=gen, device=DEV)
        u[:, :4] = 2.0
        u[:, c - (n + 3) // 4:] = 2.0
        parts.append(u.topk(n, dim=1).indices.sort(dim=1).values)
    if not parts:
        return torch.zeros((rows, 0), dtype=torch.int32, device=DEV)
    return torch.cat(parts, 1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kv, d = case["kv"], case["dim"]
    lens = _lens(case)
    order = random.Random(seed)
    need = [(c + BS - 1) // BS for _, c, _ in lens]
    num_blocks = max(1, sum(need) + sum(need) // 4)
    ids = list(range(num_blocks))
    order.shuffle(ids)
    tables = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    k_pool, v_pool, k_scale, v_scale = _pool(case, num_blocks, gen)
    starts = [0]
    for n, _, _ in lens:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    s = dict(case=case, k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale, tables=tables.to(DEV),
             starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
             # each row's (kept token's) sequence and place in it
             row_seq=torch.tensor([b for b, (n, _, _) in enumerate(lens) for _ in range(n)], dtype=torch.int64, device=DEV),
             row_at=torch.tensor([i for n, _, _ in lens for i in range(n)], dtype=torch.int64, device=DEV))
    if case["op"] == "compact":
        keep = _keep_list(case, lens, gen)
        s["keep"] = keep if case["per_head"] else keep[0]
        return s
    h = case["heads"]
    s.update(ctx=torch.tensor([c for _, c, _ in lens], dtype=torch.int32, device=DEV), scale=d ** -0.5,
             max_ctx=max(1, max(c for _, c, _ in lens)), max_chunk=max(n for n, _, _ in lens), slopes=None, prefix=None,
             q=torch.empty((rows, h, d), dtype=torch.bfloat16, device=DEV).normal_(std=case["spread"], generator=gen))
    if case["alibi"]:  # 2^(-8 (i + 1) / h)
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, h + 1, dtype=torch.float32, device=DEV) / h)
    if case["prefix"]:
        s["prefix"] = torch.tensor([x for _, _, x in lens], dtype=torch.int32, device=DEV)
    s["out"] = torch.zeros_like(s["q"])
    s["workspace"] = {}
    return s


# --------------------------------------------------------------- one pass

def run(s):
    compact = s["case"]["op"] == "compact"
    if own:
        return _own_compact(s) if compact else _own_attention(s)
    return _plain_compact(s) if compact else _plain_attention(s)


def _cache(s):
    """The written cache: E4M3 codes as the values they stand for in units of their scale."""
    if s["case"]["cache"] == "bf16":
        return [s["k_pool"], s["v_pool"]]
    return [s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn), s["k_scale"], s["v_scale"]]


def _own_compact(s):
    import paged_kv_cache_59_gb300 as pk
    pk.pa_compact_blocks(s["k_pool"], s["v_pool"], s["tables"], s["keep"], s["starts"], k_scale=s["k_scale"],
                         v_scale=s["v_scale"])
    return _cache(s)


def _own_attention(s):
    import paged_kv_cache_59_gb300 as pk
    c = s["case"]
    w = s["workspace"]
    if c["op"] == "decode":
        if "ws" not in w:
            w["ws"] = pk.decode_workspace(s["q"], s["max_ctx"])
        pk.pa_decode_score_mod(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["ctx"], s["scale"], s["max_ctx"],
                               softcap=c["cap"], alibi_slopes=s["slopes"], window=c["window"], n_sinks=c["sinks"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=w["ws"])
    else:
        if "ws" not in w:
            w["ws"] = pk.prefill_workspace(s["q"], c["seqs"], c["kv"], s["max_chunk"])
        pk.pa_prefill_score_mod(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["ctx"], s["starts"], s["scale"],
                                s["max_chunk"], softcap=c["cap"], alibi_slopes=s["slopes"], prefix_lens=s["prefix"],
                                window=c["window"], n_sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                workspace=w["ws"])
    return s["out"]


def _plain_compact(s):
    kv = s["case"]["kv"]
    keep = s["keep"].long().expand(kv, -1)                       # [kv][kept]
    head = torch.arange(kv, device=DEV)[:, None]
    src = s["tables"].long()[s["row_seq"], keep // BS]           # [kv][kept]
    dst = s["tables"].long()[s["row_seq"], s["row_at"] // BS]    # [kept]
    if s["case"]["cache"] == "bf16":
        s["k_pool"][dst, head, s["row_at"] % BS] = s["k_pool"][src, head, keep % BS]
        s["v_pool"][dst, head, s["row_at"] % BS] = s["v_pool"][src, head, keep % BS]
    else:
        _plain_compact_scaled(s, s["k_pool"], s["k_scale"], keep, head, src, dst)
        _plain_compact_scaled(s, s["v_pool"], s["v_scale"], keep, head, src, dst)
    return _cache(s)


def _plain_compact_scaled(s, pool, scale, keep, head, src, dst):
    old = scale[src, head]
    most = torch.zeros_like(scale).index_reduce_(0, dst, old.t().contiguous(), "amax")
    scale.copy_(torch.where(most > 0, most, scale))
    x = pool[src, head, keep % BS].view(torch.float8_e4m3fn).float() * (old / scale[dst, head])[..., None]
    pool[dst, head, s["row_at"] % BS] = x.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_attention(s):
    c = s["case"]
    n_seqs, h, kv, d = c["seqs"], c["heads"], c["kv"], c["dim"]
    decode = c["op"] == "decode"
    rows = 1 if decode else s["max_chunk"]
    ctx = s["ctx"].long()
    length = torch.ones_like(ctx) if decode else (s["starts"][1:] - s["starts"][:-1]).long()
    # the positions that any row of a sequence sees: the sinks, then all from the first row's window on
    sinks, window = c["sinks"], c["window"]
    width = min(s["max_ctx"], sinks + window + rows) if window >= 0 else s["max_ctx"]
    j = torch.arange(width, device=DEV)[None]
    low = (ctx - length - window).clamp(min=sinks)[:, None] if window >= 0 else torch.full_like(ctx, sinks)[:, None]
    pos = torch.where(j < sinks, j, low + j - sinks)
    inside = pos < ctx[:, None]
    pos = torch.where(inside, pos, 0)
    block = s["tables"].long().gather(1, pos // BS)
    block = torch.where(inside, block, 0)
    k, v = _plain_read(s["k_pool"], s["k_scale"], block, pos), _plain_read(s["v_pool"], s["v_scale"], block, pos)
    if decode:
        q = s["q"].float()[:, None]
    else:
        q = torch.zeros((n_seqs, rows, h, d), device=DEV)
        q[s["row_seq"], s["row_at"]] = s["q"].float()
    at = (ctx - length)[:, None] + torch.arange(rows, device=DEV)[None]  # the rows' positions
    seen = pos[:, None] <= at[..., None]
    if s["prefix"] is not None:
        seen |= pos[:, None] < s["prefix"].long()[:, None, None]
    if window >= 0:
        seen &= (pos[:, None] >= at[..., None] - window) | (pos[:, None] < sinks)
    seen &= inside[:, None]
    g = h // kv
    q = q.view(n_seqs, rows, kv, g, d).permute(0, 2, 3, 1, 4).reshape(n_seqs, kv, g * rows, d)
    score = (q @ k.permute(0, 2, 3, 1)).view(n_seqs, kv, g, rows, width) * s["scale"]
    if c["cap"] > 0:
        score = torch.tanh(score / c["cap"]) * c["cap"]
    if s["slopes"] is not None:
        far = (pos[:, None] - at[..., None]).abs().float()
        score = score - s["slopes"].view(1, kv, g, 1, 1) * far[:, None, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    out = p.view(n_seqs, kv, g * rows, width) @ v.permute(0, 2, 1, 3)
    out = out.view(n_seqs, kv, g, rows, d) / torch.where(total == 0, 1.0, total)
    out = out.permute(0, 3, 1, 2, 4).reshape(n_seqs, rows, h, d)
    s["out"].copy_(out[:, 0] if decode else out[s["row_seq"], s["row_at"]])
    return s["out"]


def _plain_read(pool, scale, block, pos):
    """[seqs][positions][kv][dim] in 32 bits."""
    x = pool[block, :, pos % BS]
    return x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale[block][..., None]


# ---------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_compact(s) if case["op"] == "compact" else _exact_attention(s)


def _to_e4m3(x):
    """The E4M3 value next to each x of |x| <= 448 (ties to even): steps of 2^-3 of the binade, 2^-9 at the least."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].long() - 4
    step = ((e + 1023) << 52).view(torch.float64)  # 2^e
    return torch.round(x / step) * step


def _exact_compact(s):
    c = s["case"]
    starts = s["starts"].tolist()
    pools = [p.double() if c["cache"] == "bf16" else p.view(torch.float8_e4m3fn).double() for p in (s["k_pool"], s["v_pool"])]
    scales = [] if c["cache"] == "bf16" else [s["k_scale"].double(), s["v_scale"].double()]
    for b in range(c["seqs"]):
        a, e = starts[b], starts[b + 1]
        if a == e:
            continue
        ids = s["tables"][b].long()
        to = ids[:(e - a + BS - 1) // BS]
        for g in range(c["kv"]):
            keep = (s["keep"][g] if c["per_head"] else s["keep"])[a:e].long()
            last = int(keep[-1]) // BS + 1
            for x, pool in enumerate(pools):
                value = pool[ids[:last], g].reshape(-1, c["dim"])[keep]
                if scales:
                    was = scales[x][ids[keep // BS], g]
                    now = torch.nn.functional.pad(was, (0, len(to) * BS - len(was)), value=0.0).view(-1, BS).amax(1)
                    scales[x][to, g] = now
                    value = _to_e4m3(value * (was / now.repeat_interleave(BS)[:len(was)])[:, None])
                tile = pool[to, g].reshape(-1, c["dim"])
                tile[:e - a] = value
                pool[to, g] = tile.view(-1, BS, c["dim"])
    return [*pools, *scales]


def _exact_attention(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts = s["starts"].tolist()
    prefix = [0] * c["seqs"] if s["prefix"] is None else s["prefix"].tolist()
    for b, n in enumerate(s["ctx"].tolist()):
        a, e = starts[b], starts[b + 1]
        if n == 0:
            continue
        blocks = s["tables"][b, :(n + BS - 1) // BS].long()
        at = torch.arange(n - (e - a), n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)[None]
        hidden = (t > at) & (t >= prefix[b])
        if c["window"] >= 0:
            hidden |= (t < at - c["window"]) & (t >= c["sinks"])
        for g in range(c["kv"]):
            kv = []
            for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])):
                x = pool[blocks, g]
                x = x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale[blocks, g, None, None].double()
                kv.append(x.reshape(-1, c["dim"])[:n])
            heads = slice(g * c["heads"] // c["kv"], (g + 1) * c["heads"] // c["kv"])
            w = torch.einsum("lhd,td->hlt", s["q"][a:e, heads].double(), kv[0]) * s["scale"]
            if c["cap"]:
                w = c["cap"] * torch.tanh(w / c["cap"])
            if c["alibi"]:
                w = w - s["slopes"][heads].double()[:, None, None] * (at - t).abs()
            w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
            out[a:e, heads] = torch.einsum("hlt,td->lhd", w, kv[1])
    return out
