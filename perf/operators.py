"""The serving operators around the paged cache, as a timing harness measures them:

  append   rotary position rotation of q and k with the write of k and v into the paged
           cache, held in bf16 or in E4M3 with one scale per (block, KV head)
  decode   one query per sequence over that cache, over all of it or over a sliding
           window with a few first tokens that stay visible (sinks)
  prefill  a causal chunk of queries per sequence over the same caches and masks

With ``own`` false ``run`` computes each in elementary torch operations in 32 bits;
with ``own`` true it calls the library.

Conventions: a block holds 16 tokens; pools are [blocks][kv_heads][16][head_dim]; an
E4M3 element stands for code * scale[block][kv_head]; scales are powers of two, the
smallest 2^e, -32 <= e <= 32, with max |x| <= 448 * 2^e over the block's tokens.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BS = 16
DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a 64-sequence batch of an 8B-shaped model, bf16 cache: a few
        # microseconds, where the launch counts
        dict(name="append 64 tokens bf16", op="append", cache="bf16", heads=32, kv=8, dim=128, seqs=64, chunk_lo=1,
             chunk_hi=1, pos_hi=4096, rot=128, interleaved=False),
        # prompt chunks of a 70B-shaped model: the bandwidth-bound end
        dict(name="append 8192 tokens bf16", op="append", cache="bf16", heads=64, kv=8, dim=128, seqs=4, chunk_lo=2048,
             chunk_hi=2048, pos_hi=32768, rot=128, interleaved=False),
        # the same decode step into an E4M3 cache: partly filled blocks whose scale may grow
        dict(name="append 64 tokens e4m3", op="append", cache="e4m3", heads=32, kv=8, dim=128, seqs=64, chunk_lo=1,
             chunk_hi=1, pos_hi=4096, rot=128, interleaved=False),
        # ragged prompt chunks that start and end inside blocks, pairs side by side
        dict(name="append ragged chunks e4m3", op="append", cache="e4m3", heads=32, kv=8, dim=128, seqs=9, chunk_lo=5,
             chunk_hi=1777, pos_hi=131072, rot=128, interleaved=True),
        # the smallest decode: four sequences, one head per KV head
        dict(name="decode tiny e4m3", op="decode", cache="e4m3", heads=4, kv=4, dim=64, seqs=4, ctx_lo=1, ctx_hi=37,
             window=-1, sinks=0),
        # a serving batch of an 8B-shaped model
        dict(name="decode batch e4m3", op="decode", cache="e4m3", heads=32, kv=8, dim=128, seqs=64, ctx_lo=128,
             ctx_hi=4096, window=-1, sinks=0),
        # few long documents, 70B-shaped: work has to be split over the context
        dict(name="decode long e4m3", op="decode", cache="e4m3", heads=64, kv=8, dim=128, seqs=4, ctx_lo=99999,
             ctx_hi=131072, window=-1, sinks=0),
        # long chats that keep a window and the first tokens, 7B-shaped
        dict(name="decode window sinks bf16", op="decode", cache="bf16", heads=32, kv=8, dim=128, seqs=32, ctx_lo=4096,
             ctx_hi=32768, window=4096, sinks=4),
        # one short stream with a small window: latency
        dict(name="decode one stream bf16", op="decode", cache="bf16", heads=8, kv=8, dim=64, seqs=1, ctx_lo=700,
             ctx_hi=700, window=127, sinks=5),
        # a chunk of a long prompt under window and sinks
        dict(name="prefill window sinks bf16", op="prefill", cache="bf16", heads=32, kv=8, dim=128, seqs=1,
             chunk_lo=2048, chunk_hi=2048, ctx_lo=16384, ctx_hi=16384, window=4096, sinks=4),
        # ragged chunks of several short prompts, head_dim 64, one head per KV head
        dict(name="prefill ragged window bf16", op="prefill", cache="bf16", heads=8, kv=8, dim=64, seqs=7, chunk_lo=1,
             chunk_hi=333, ctx_lo=17, ctx_hi=2001, window=255, sinks=17),
        # a chunk of a long prompt over an E4M3 cache, no window
        dict(name="prefill chunk e4m3", op="prefill", cache="e4m3", heads=32, kv=8, dim=128, seqs=2, chunk_lo=1024,
             chunk_hi=1024, ctx_lo=6000, ctx_hi=8192, window=-1, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    group = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    case = dict(op=rng.choice(["append", "decode", "prefill"]), cache=rng.choice(["bf16", "e4m3"]), heads=kv * group,
                kv=kv, dim=dim, lens_seed=rng.randrange(1 << 20))
    if case["op"] == "append":
        chunk = _log_int(rng, 1, 2048)
        case.update(seqs=_log_int(rng, 1, max(1, min(256, 8192 // chunk))), chunk_lo=rng.randint(1, chunk),
                    chunk_hi=chunk, pos_hi=_log_int(rng, chunk + 16, 131072), rot=rng.choice([dim, dim, dim // 2]),
                    interleaved=rng.random() < 0.5)
        return case
    windowed = case["cache"] == "bf16" or rng.random() < 0.4
    case.update(window=_log_int(rng, 1, 4096) if windowed else -1, sinks=rng.choice([0, 1, 4, 5, 16, 33]) if windowed else 0)
    if case["op"] == "decode":
        ctx = _log_int(rng, 1, 65536)
        case.update(seqs=_log_int(rng, 1, max(1, min(128, 196608 // ctx))), ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    else:
        chunk = _log_int(rng, 1, 1024)
        ctx = _log_int(rng, chunk, 6144)
        case.update(seqs=_log_int(rng, 1, max(1, min(8, 65536 // (chunk * case["heads"])))), chunk_lo=rng.randint(1, chunk),
                    chunk_hi=chunk, ctx_lo=rng.randint(chunk, ctx), ctx_hi=ctx)
    return case


def _lens(case):
    """(new tokens, context) of each sequence, from the case alone."""
    r = random.Random(case.get("lens_seed", 7) * 1000003 + case["seqs"])
    got = []
    for _ in range(case["seqs"]):
        if case["op"] == "append":
            n = r.randint(case["chunk_lo"], case["chunk_hi"])
            got.append((n, r.randint(n, case["pos_hi"])))
        elif case["op"] == "decode":
            got.append((1, r.randint(case["ctx_lo"], case["ctx_hi"])))
        else:
            n = r.randint(case["chunk_lo"], case["chunk_hi"])
            got.append((n, max(n, r.randint(case["ctx_lo"], case["ctx_hi"]))))
    return got


def _seen(case, p):
    """Positions that a query at position p attends to."""
    w = case["window"]
    first = max(0, p - w) if w >= 0 else 0
    return p + 1 - first + min(case["sinks"], first)


def work(case):
    h, kv, d = case["heads"], case["kv"], case["dim"]
    lens = _lens(case)
    tokens = sum(n for n, _ in lens)
    eb = 2 if case["cache"] == "bf16" else 1
    if case["op"] == "append":
        # q in and out, k and v in, codes or values out, angles, positions, slots, scales
        b = tokens * (4 * h * d + 4 * kv * d + 2 * eb * kv * d + 4 * case["rot"] + 16)
        blocks = sum((c + BS - 1) // BS - (c - n) // BS for n, c in lens)
        return {"bytes": b + (16 * blocks * kv if eb == 1 else 0), "flops": 3 * tokens * (h + kv) * case["rot"]}
    if case["op"] == "decode":
        read = [_seen(case, c - 1) if c else 0 for _, c in lens]
        pairs = sum(read)
    else:
        read, pairs = [], 0
        for n, c in lens:
            lo = max(0, c - n - case["window"]) if case["window"] >= 0 else 0
            read.append(c - lo + min(case["sinks"], lo))
            pairs += sum(_seen(case, p) for p in range(c - n, c))
    scales = sum((r + BS - 1) // BS for r in read) * kv * 8 if eb == 1 else 0
    b = sum(read) * kv * d * 2 * eb + scales + tokens * h * d * 4 + sum((r + BS - 1) // BS for r in read) * 4
    return {"bytes": b, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ inputs

def _power_scale(amax):
    """The smallest 2^e, -32 <= e <= 32, with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -32)).clamp(-32, 32)
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
            # tokens and heads differ in magnitude
            x *= torch.exp2(torch.randn((n, case["kv"], 1, 1), generator=gen, device=DEV) * 0.7)
            scale[a:a + n] = _power_scale(x.abs().amax(dim=(2, 3)))
            codes[a:a + n] = (x / scale[a:a + n, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        got.append(codes)
        scales.append(scale)
    return got[0], got[1], scales[0], scales[1]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    h, kv, d = case["heads"], case["kv"], case["dim"]
    lens = _lens(case)
    order = random.Random(seed)
    if case["op"] == "append":
        return _prepare_append(case, lens, gen, order)
    need = [(c + BS - 1) // BS for _, c in lens]
    num_blocks = max(1, sum(need) + sum(need) // 4)
    ids = list(range(num_blocks))
    order.shuffle(ids)
    tables = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    k_pool, v_pool, k_scale, v_scale = _pool(case, num_blocks, gen)
    rows = sum(n for n, _ in lens)
    s = dict(case=case, k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale, tables=tables.to(DEV),
             ctx=torch.tensor([c for _, c in lens], dtype=torch.int32, device=DEV), scale=d ** -0.5,
             max_ctx=max(1, max(c for _, c in lens)), max_chunk=max(n for n, _ in lens),
             q=torch.empty((rows, h, d), dtype=torch.bfloat16, device=DEV).normal_(generator=gen))
    s["out"] = torch.zeros_like(s["q"])
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    # each row's sequence and place in its chunk
    s["row_seq"] = torch.tensor([b for b, (n, _) in enumerate(lens) for _ in range(n)], device=DEV)
    s["row_at"] = torch.tensor([i for n, _ in lens for i in range(n)], device=DEV)
    s["workspace"] = {}
    return s


def _prepare_append(case, lens, gen, order):
    h, kv, d = case["heads"], case["kv"], case["dim"]
    tokens = sum(n for n, _ in lens)
    blocks = sum((c + BS - 1) // BS - (c - n) // BS for n, c in lens)
    num_blocks = blocks + blocks // 4 + 1
    ids = list(range(num_blocks))
    order.shuffle(ids)
    positions, slots, at = [], [], 0
    for n, c in lens:
        first = (c - n) // BS
        positions += range(c - n, c)
        slots += [ids[at + p // BS - first] * BS + p % BS for p in range(c - n, c)]
        at += (c + BS - 1) // BS - first
    qkv = torch.empty((tokens, (h + 2 * kv) * d), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    qkv *= torch.exp2(torch.randn((tokens, 1), generator=gen, device=DEV)).to(torch.bfloat16)
    k_pool, v_pool, k_scale, v_scale = _pool(case, num_blocks, gen)
    rot = case["rot"]
    top = case["pos_hi"]
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(top, dtype=torch.float64, device=DEV)[:, None] * freq
    slots = torch.tensor(slots, dtype=torch.int64)
    touched, index = torch.unique(slots // BS, return_inverse=True)
    return dict(case=case, q=qkv[:, :h * d].view(tokens, h, d), k=qkv[:, h * d:(h + kv) * d].view(tokens, kv, d),
                v=qkv[:, (h + kv) * d:].view(tokens, kv, d), k_pool=k_pool, v_pool=v_pool, k_scale=k_scale,
                v_scale=v_scale, cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                positions=torch.tensor(positions, dtype=torch.int64, device=DEV), slots=slots.to(DEV),
                # the blocks that the block manager handed out for these tokens, and each token's among them
                blocks=touched.to(DEV), block_of=index.to(DEV),
                q_out=torch.empty((tokens, h, d), dtype=torch.bfloat16, device=DEV))


# --------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own_append(s) if op == "append" else _own_attention(s)
    return _plain_append(s) if op == "append" else _plain_attention(s)


def _cache(s):
    """The written cache: E4M3 codes as the values they stand for in units of their scale."""
    if s["case"]["cache"] == "bf16":
        return [s["k_pool"], s["v_pool"]]
    return [s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn), s["k_scale"], s["v_scale"]]


def _own_append(s):
    import paged_kv_cache_59_gb300 as pk
    c = s["case"]
    if c["cache"] == "bf16":
        pk.pa_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["cos_sin"], s["positions"],
                             s["slots"], interleaved=c["interleaved"])
    else:
        pk.pa_rope_and_cache_fp8_block(s["q_out"], s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"],
                                       s["v_scale"], s["cos_sin"], s["positions"], s["slots"],
                                       interleaved=c["interleaved"])
    return [s["q_out"], *_cache(s)]


def _own_attention(s):
    import paged_kv_cache_59_gb300 as pk
    c = s["case"]
    w = s["workspace"]
    if c["op"] == "decode":
        if "ws" not in w:
            w["ws"] = pk.decode_workspace(s["q"], s["max_ctx"])
        if c["cache"] == "bf16":
            pk.pa_decode_sinks(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["ctx"], s["scale"], s["max_ctx"],
                               c["window"], c["sinks"], workspace=w["ws"])
        else:
            pk.pa_decode_fp8_block(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                                   s["ctx"], s["scale"], s["max_ctx"], window=c["window"], n_sinks=c["sinks"],
                                   workspace=w["ws"])
    else:
        if "ws" not in w:
            w["ws"] = pk.prefill_workspace(s["q"], c["seqs"], c["kv"], s["max_chunk"])
        if c["cache"] == "bf16":
            pk.pa_prefill_sinks(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["ctx"], s["starts"], s["scale"],
                                s["max_chunk"], c["window"], c["sinks"], workspace=w["ws"])
        else:
            pk.pa_prefill_fp8_block(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                                    s["ctx"], s["starts"], s["scale"], s["max_chunk"], window=c["window"],
                                    n_sinks=c["sinks"], workspace=w["ws"])
    return s["out"]


def _rotate(x, cos, sin, rot, interleaved):
    """x [tokens][heads][dim], cos and sin [tokens][rot / 2]: pairs (i, i + rot / 2), or (2i, 2i + 1)."""
    cos, sin = cos[:, None], sin[:, None]
    y, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    c = s["case"]
    rot = c["rot"]
    angle = s["cos_sin"][s["positions"]]
    cos, sin = angle[:, :rot // 2], angle[:, rot // 2:]
    block, offset = s["slots"] // BS, s["slots"] % BS
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, rot, c["interleaved"]))
    k, v = _rotate(s["k"].float(), cos, sin, rot, c["interleaved"]), s["v"].float()
    if c["cache"] == "bf16":
        s["k_pool"][block, :, offset] = k.to(torch.bfloat16)
        s["v_pool"][block, :, offset] = s["v"]
    else:
        _plain_write(s, s["k_pool"], s["k_scale"], k, offset)
        _plain_write(s, s["v_pool"], s["v_scale"], v, offset)
    return [s["q_out"], *_cache(s)]


def _plain_write(s, pool, scale, x, offset):
    """Writes x [tokens][kv][dim] into its blocks: a block written from its first slot takes the scale
    of the new tokens, another the larger of its own and theirs, and its other codes are encoded again."""
    blocks, at = s["blocks"], s["block_of"]
    n, kv = blocks.numel(), x.shape[1]
    amax = torch.zeros((n, kv), device=DEV).index_reduce_(0, at, x.abs().amax(-1), "amax")
    fresh = torch.zeros(n, device=DEV).index_reduce_(0, at, (offset == 0).float(), "amax")[:, None] > 0
    old = scale[blocks]
    new = torch.where(fresh, _power_scale(amax), torch.maximum(old, _power_scale(amax)))
    codes = pool[blocks]
    again = codes.view(torch.float8_e4m3fn).float() * (old / new)[:, :, None, None]
    codes = torch.where(fresh[:, :, None, None], codes, again.to(torch.float8_e4m3fn).view(torch.uint8))
    codes[at, :, offset] = (x / new[at][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    pool[blocks] = codes
    scale[blocks] = new


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
    k, v = _plain_read(s, s["k_pool"], s["k_scale"], block, pos), _plain_read(s, s["v_pool"], s["v_scale"], block, pos)
    if decode:
        q = s["q"].float()[:, None]
    else:
        q = torch.zeros((n_seqs, rows, h, d), device=DEV)
        q[s["row_seq"], s["row_at"]] = s["q"].float()
    at = (ctx - length)[:, None] + torch.arange(rows, device=DEV)[None]  # the rows' positions
    seen = inside[:, None] & (pos[:, None] <= at[..., None])
    if window >= 0:
        seen &= (pos[:, None] >= at[..., None] - window) | (pos[:, None] < sinks)
    g = h // kv
    q = q.view(n_seqs, rows, kv, g, d).permute(0, 2, 3, 1, 4).reshape(n_seqs, kv, g * rows, d)
    score = (q @ k.permute(0, 2, 3, 1)).view(n_seqs, kv, g, rows, width) * s["scale"]
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


def _plain_read(s, pool, scale, block, pos):
    """[seqs][positions][kv][dim] in 32 bits."""
    x = pool[block, :, pos % BS]
    return x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale[block][..., None]


# ---------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _turned(x, angle, rot, interleaved):
    """x as complex numbers, times e^(i angle)."""
    half = rot // 2
    x = x.double()
    z = torch.complex(*((x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])))
    z = z * torch.complex(angle[:, :half].double(), angle[:, half:].double())[:, None]
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        y[..., :half], y[..., half:rot] = z.real, z.imag
    return y


def _to_e4m3(x):
    """The E4M3 value next to each x of |x| <= 448 (ties to even): steps of 2^-3 of the binade, 2^-9 at the least."""
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    angle = s["cos_sin"][s["positions"]]
    q = _turned(s["q"], angle, c["rot"], c["interleaved"])
    new = [_turned(s["k"], angle, c["rot"], c["interleaved"]), s["v"].double()]
    slot = s["slots"]
    if c["cache"] == "bf16":
        pools = [s["k_pool"].double(), s["v_pool"].double()]
        for pool, x in zip(pools, new):
            pool.transpose(1, 2)[slot // BS, slot % BS] = x
        return [q, *pools]
    pools, scales = [], []
    first = torch.full((s["k_pool"].shape[0],), BS, device=DEV).scatter_reduce(0, slot // BS, slot % BS, "amin")
    for codes, scale, x in zip((s["k_pool"], s["v_pool"]), (s["k_scale"], s["v_scale"]), new):
        value = codes.view(torch.float8_e4m3fn).double()
        most = torch.zeros_like(scale, dtype=torch.float64)
        most = most.index_reduce(0, slot // BS, x.abs().amax(-1), "amax")
        m, e = torch.frexp(most.clamp(min=1e-30) / 448)
        least = torch.ldexp(torch.ones_like(most), torch.where(m == 0.5, e - 1, e).clamp(-32, 32))
        was = scale.double()
        now = torch.where(first[:, None] == 0, least, torch.where(first[:, None] < BS, torch.maximum(was, least), was))
        kept = _to_e4m3(value * (was / now)[:, :, None, None])
        value = torch.where((first == 0)[:, None, None, None], value, kept)
        value.transpose(1, 2)[slot // BS, slot % BS] = _to_e4m3(x / now[slot // BS][..., None])
        pools.append(value)
        scales.append(now)
    return [q, *pools, *scales]


def _exact_attention(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts = s["starts"].tolist()
    for b, n in enumerate(s["ctx"].tolist()):
        a, e = starts[b], starts[b + 1]
        if n == 0:
            continue
        blocks = s["tables"][b, :(n + BS - 1) // BS].long()
        at = torch.arange(n - (e - a), n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)[None]
        hidden = t > at
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
            w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
            out[a:e, heads] = torch.einsum("hlt,td->lhd", w, kv[1])
    return out
