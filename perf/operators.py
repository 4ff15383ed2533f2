"""What is measured of the serving and position operators: rotary positions, the
4-bit key/value cache (appending to it and reading it back), decoding over that
cache, and evicting from it by accumulated attention weight.

`run` computes a case in elementary torch operations, or with `own` set through
the package's entry points, on the same state.

The 4-bit cache, as both sides hold it: a byte tensor of
(pages, kv heads, page size / 16, block bytes).  A block is 16 tokens of one
head: key codes (16 x D/2 bytes), key scales (16 x D/group pairs of bf16), value
codes, value scales.  A group of `group` channels holds
s = bf16((max - min) / 15), m = min and the codes round((x - m) / s); it stands
for s * code + m.  Key channel 32 g + 8 j + i is nibble i of the row's 32-bit
word j D/32 + g; value channel 32 g + 4 r + i is nibble i of its 16-bit
half-word r D/32 + g."""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the queries and keys of one layer of a training step, rotated before
        # attention (the repository's T = 8192 training shape)
        dict(name="rope_train", op="rope", batch=2, tokens=8192, q_heads=16, kv_heads=16, dim=128, rotary=128,
             interleaved=False, dtype="bf16", scaled=False, fused=False, far=0, grad=False),
        # forward and gradient of a part-rotated head of 64 in the interleaved
        # layout, grouped heads, a ragged length, read from a fused projection
        dict(name="rope_grad", op="rope", batch=4, tokens=2999, q_heads=16, kv_heads=4, dim=64, rotary=32,
             interleaved=True, dtype="fp16", scaled=False, fused=True, far=0, grad=True),
        # a decoding step far into a scaled context, one token per sequence
        dict(name="rope_step", op="rope", batch=8, tokens=1, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", scaled=True, fused=True, far=900001, grad=False),
        # prompts of different lengths written to the cache: rotated, quantised, read back
        dict(name="append_prompts", op="append", batch=6, new=8192, past=0, kv_heads=8, dim=128, group=64, page=64,
             rotary=128),
        # a chunk per sequence behind what is cached, small pages that the chunk
        # starts and ends inside, half-size heads, finer groups, no rotation
        dict(name="append_chunk", op="append", batch=9, new=301, past=1003, kv_heads=4, dim=64, group=32, page=16,
             rotary=0),
        # one token for each sequence of a decoding batch
        dict(name="append_step", op="append", batch=32, new=1, past=4090, kv_heads=8, dim=128, group=64, page=64,
             rotary=128),
        # the first steps of one conversation: latency
        dict(name="decode_short", op="decode", batch=1, tokens=117, q_heads=8, kv_heads=2, dim=64, group=64, page=16,
             queries=1, ragged=False, weights=False),
        # a mixed serving batch with grouped heads: lengths from one token to thousands
        dict(name="decode_mixed", op="decode", batch=24, tokens=8111, q_heads=32, kv_heads=8, dim=128, group=32,
             page=16, queries=1, ragged=True, weights=False),
        # the repository's decoding shape: a head of its own for every query head, long caches
        dict(name="decode_long", op="decode", batch=8, tokens=32768, q_heads=32, kv_heads=32, dim=128, group=64,
             page=64, queries=1, ragged=False, weights=False),
        # checking a draft of four tokens, with the weights that eviction goes by
        dict(name="decode_draft", op="decode", batch=8, tokens=12345, q_heads=32, kv_heads=8, dim=128, group=64,
             page=64, queries=4, ragged=True, weights=True),
        # a batch brought back to its budget, some sequences far above it, some below
        dict(name="evict_batch", op="evict", batch=16, tokens=8191, kv_heads=8, dim=128, group=64, page=64,
             budget=2048, recent=256, ragged=True),
        # a long prompt cut down once
        dict(name="evict_prompt", op="evict", batch=1, tokens=60007, kv_heads=8, dim=64, group=32, page=32,
             budget=8192, recent=1024, ragged=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 32])
    if op == "rope":
        batch = log(1, 16)
        q_heads = kv_heads * rng.choice([1, 2, 4, 8]) if kv_heads < 32 else 32
        tokens = min(log(1, 16384), max(1, (1 << 19) // (batch * (q_heads + kv_heads))))
        return dict(op=op, batch=batch, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([dim, dim // 2, 20, dim - 2]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), scaled=rng.random() < 0.5, fused=rng.random() < 0.5,
                    far=rng.choice([0, log(1, 1 << 20)]), grad=rng.random() < 0.5)
    group, page = rng.choice([32, 64]), rng.choice([16, 32, 64, 128])
    if op == "append":
        batch = log(1, 32)
        new = min(log(1, 8192), max(1, 32768 // (batch * kv_heads) * 8))
        return dict(op=op, batch=batch, new=new, past=rng.choice([0, log(1, 4096)]), kv_heads=kv_heads, dim=dim,
                    group=group, page=page, rotary=rng.choice([0, dim, dim // 2]))
    if op == "decode":
        batch = log(1, 64)
        tokens = min(log(1, 65536), max(16, (1 << 22) // (batch * kv_heads)))
        return dict(op=op, batch=batch, tokens=tokens, q_heads=kv_heads * rng.choice([1, 3, 4, 8]), kv_heads=kv_heads,
                    dim=dim, group=group, page=page, queries=rng.choice([1, 1, 2, 5, 8]), ragged=rng.random() < 0.7,
                    weights=rng.random() < 0.4)
    batch = log(1, 16)
    tokens = min(log(16, 60000), max(16, (1 << 19) // (batch * kv_heads)))
    budget = max(8, int(tokens * rng.uniform(0.1, 0.98)))
    return dict(op=op, batch=batch, tokens=tokens, kv_heads=kv_heads, dim=dim, group=group, page=page, budget=budget,
                recent=int(budget * rng.uniform(0.0, 0.5)), ragged=rng.random() < 0.7)


def spread(count, most, least, phase, ragged):
    """`count` whole numbers of [least, most], the first `most`: the lengths of a batch."""
    if not ragged:
        return [most] * count
    return [most] + [least + int((most - least) * ((b * GOLDEN + phase) % 1.0)) for b in range(1, count)]


def lengths_of(case):
    """Tokens held by each sequence, the appended ones among them, and how many of them are new."""
    if case["op"] == "append":
        new = spread(case["batch"], case["new"], 0 if case["new"] > 1 else 1, 0.31, case["new"] > 1)
        past = spread(case["batch"], case["past"], case["past"] // 2, 0.17, case["past"] > 1)
        return [a + b for a, b in zip(new, past)], new
    # a ragged batch holds an empty sequence too: a slot whose request has ended
    held = spread(case["batch"], case["tokens"], 1, 0.53, case["ragged"])
    if case["ragged"] and case["batch"] > 3:
        held[2] = 0
    return held, None


def block_bytes(case):
    return 16 * (case["dim"] + 8 * case["dim"] // case["group"])


def work(case):
    d, op = case["dim"], case["op"]
    if op == "rope":
        size = DTYPES[case["dtype"]].itemsize
        n = case["batch"] * case["tokens"] * (case["q_heads"] + case["kv_heads"])
        passes = 2 if case["grad"] else 1
        # read and written once a direction; six operations for a pair's rotation
        return {"bytes": passes * (2 * n * d * size + 8 * case["tokens"]), "flops": passes * 3 * n * case["rotary"]}
    token = block_bytes(case) // 16  # codes and scales, keys and values
    held, new = lengths_of(case)
    if op == "append":
        n = sum(new) * case["kv_heads"]
        # keys and values in, codes out, codes in again, values out (every row of the padded answer)
        out = case["batch"] * max(new) * case["kv_heads"]
        return {"bytes": n * (4 * d + 2 * token) + out * 4 * d, "flops": n * (2 * d * 5 + 2 * d * 2 + 3 * case["rotary"])}
    if op == "decode":
        n = sum(held) * case["kv_heads"]
        rows = case["batch"] * case["q_heads"] * case["queries"]
        each = case["q_heads"] // case["kv_heads"] * case["queries"]
        return {"bytes": n * (token + (8 if case["weights"] else 0)) + rows * (4 * d + 4), "flops": 4 * d * n * each}
    n = sum(held) * case["kv_heads"]
    kept = sum(min(h, case["budget"]) for h in held) * case["kv_heads"]
    moved = moves_of(case)
    out = case["batch"] * case["kv_heads"]
    # weights and positions in and out, what moves, and the kept part read back
    return {"bytes": 8 * n + out * (8 * case["tokens"] + 4 * case["budget"]) + 2 * moved * token + kept * token
            + out * case["budget"] * 4 * d, "flops": 4 * n}


def moves_of(case):
    """Tokens that change their place: the kept ones behind the budget, the recent ones and a share of the others."""
    held, _ = lengths_of(case)
    budget, recent = case["budget"], case["recent"]
    over = [(h, min(recent, h - budget)) for h in held if h > budget]
    return int(sum(r + (budget - recent) * (h - budget - r) / max(1, h - recent) for h, r in over)) * case["kv_heads"]


# ------------------------------------------------------------------ inputs

def frequencies(case):
    """Radians per position of each rotated pair: base 10000, or stretched eightfold by parts
    (frequencies that turn less than once in 4096 positions divided by eight, those over 32 turns kept)."""
    r = case["rotary"]
    f = [10000.0 ** (-2 * i / r) for i in range(r // 2)]
    if case.get("scaled"):
        keep = [min(1.0, max(0.0, (4096 * x / (2 * math.pi) - 1) / 31)) for x in f]
        f = [x * k + x / 8 * (1 - k) for x, k in zip(f, keep)]
    return f


def amplitude(case):
    return 0.1 * math.log(8.0) + 1.0 if case.get("scaled") else 1.0


def turns(case):
    """The frequencies as the entry points take them: turns per position, in units of 2^-64."""
    return torch.tensor([round(x / (2 * math.pi) * 2.0 ** 64) for x in frequencies(case)], dtype=torch.int64,
                        device=DEVICE)


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE)


def heads_like(gen, n, heads, dim):
    """Keys or values (n, heads, dim) in bf16: normal, with a gain and an offset for each channel as projections have them."""
    gain = torch.rand(heads, dim, generator=gen, device=DEVICE) * 0.6 + 0.7
    shift = normal(gen, heads, dim) * 0.3
    return (normal(gen, n, heads, dim) * gain + shift).to(torch.bfloat16)


def paged(case, gen, held):
    """An empty pool with room for `held`, and the table of its pages in an order as a long-lived server has it."""
    need = [-(-h // case["page"]) for h in held]
    width = max(1, max(need))
    order = torch.randperm(sum(need) + 3, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pool = torch.zeros(sum(need) + 3, case["kv_heads"], case["page"] // 16, block_bytes(case), dtype=torch.uint8,
                       device=DEVICE)
    return pool, table


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def ends(counts):
    return ints([0] + torch.tensor(counts).cumsum(0).tolist())


def filled(case, gen, held):
    pool, table = paged(case, gen, held)
    total = sum(held)
    if total:
        step = max(1, (1 << 27) // (case["kv_heads"] * case["dim"]))
        gains = gen.initial_seed()
        sequence = torch.repeat_interleave(torch.arange(len(held), device=DEVICE), ints(held))
        slot = torch.arange(total, device=DEVICE) - ends(held)[:-1].long()[sequence]
        for lo in range(0, total, step):
            n = min(step, total - lo)
            part = torch.Generator(DEVICE).manual_seed(gains + 7 * lo + 1)
            write(pool, table, heads_like(part, n, case["kv_heads"], case["dim"]),
                  heads_like(part, n, case["kv_heads"], case["dim"]), sequence[lo:lo + n], slot[lo:lo + n],
                  case["group"])
    return pool, table


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    held, new = (None, None) if case["op"] == "rope" else lengths_of(case)
    s = {"case": case}
    if case["op"] == "rope":
        b, t, hq, hk, d = (case[n] for n in ("batch", "tokens", "q_heads", "kv_heads", "dim"))
        dtype = DTYPES[case["dtype"]]
        if case["fused"]:  # one projection's output, heads behind tokens, queries, keys and values side by side
            x = normal(gen, b, t, hq + 2 * hk, d).to(dtype).transpose(1, 2)
            s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        else:
            s["q"], s["k"] = normal(gen, b, hq, t, d).to(dtype), normal(gen, b, hk, t, d).to(dtype)
        if case["grad"]:
            s["q"], s["k"] = s["q"].detach().requires_grad_(), s["k"].detach().requires_grad_()
            s["gq"], s["gk"] = normal(gen, b, hq, t, d).to(dtype), normal(gen, b, hk, t, d).to(dtype)
        start = torch.randint(0, case["far"] // 8 + 1, (b, 1), generator=gen, device=DEVICE, dtype=torch.int32)
        s["positions"] = (torch.arange(t, device=DEVICE, dtype=torch.int32) + case["far"] + start).contiguous()
        s["table"] = turns(case)
    elif case["op"] == "append":
        total = sum(new)
        s["pool"], s["block_table"] = paged(case, gen, held)
        s["k"] = heads_like(gen, total, case["kv_heads"], case["dim"])
        s["v"] = heads_like(gen, total, case["kv_heads"], case["dim"])
        s["lengths"], s["cu_new"] = ints(held), ends(new)
        s["start"] = ints([h - n for h, n in zip(held, new)])
        s["table"] = turns(case) if case["rotary"] else None
    elif case["op"] == "decode":
        s["pool"], s["block_table"] = filled(case, gen, held)
        s["q"] = normal(gen, case["batch"], case["q_heads"], case["queries"], case["dim"]).to(torch.bfloat16)
        s["lengths"] = ints(held)
        if case["weights"]:
            shape = case["batch"], case["kv_heads"], s["block_table"].shape[1] * case["page"]
            s["weights"] = torch.rand(*shape, generator=gen, device=DEVICE) * 4
            s["weights_out"] = torch.zeros(*shape, device=DEVICE)
    else:
        s["pool"], s["block_table"] = filled(case, gen, held)
        s["lengths"] = ints(held)
        b, h, t = case["batch"], case["kv_heads"], case["tokens"]
        # accumulated weights: most tokens get little, some nothing at all yet, a few much
        s["weights"] = normal(gen, b, h, t).mul(2).exp() * (torch.rand(b, h, t, generator=gen, device=DEVICE) > 0.05)
        # an earlier eviction has left each head's tokens in an order of its own
        s["slot_positions"] = torch.argsort(torch.rand(b, h, t, generator=gen, device=DEVICE)
                                            + torch.arange(t, device=DEVICE) / 64.0, dim=-1).to(torch.int32)
    return s


# ------------------------------------------------------------------ plain forms

def rotate(x, positions, table, interleaved, scale, back=False):
    """x (..., T, D) in 32 bits, its first 2 * len(table) channels turned pair by pair; positions broadcast to (..., T)."""
    r = 2 * table.numel()
    angle = (positions.double()[..., None] * (table.double() / 2.0 ** 64)) % 1.0 * (2 * math.pi)
    cos, sin = (angle.cos() * scale).float(), (angle.sin() * scale).float()
    if back:
        sin = -sin
    part, rest = x[..., :r], x[..., r:]
    a, b = (part[..., ::2], part[..., 1::2]) if interleaved else (part[..., :r // 2], part[..., r // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, rest), -1)


def quantise(x, group):
    """Codes (n, heads, D) and scales (n, heads, D / group, 2) of bf16 values; a group that holds no finite range is NaN."""
    g = x.float().unflatten(-1, (-1, group))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((high - low) / 15).to(torch.bfloat16).float()
    s = torch.where(s < 2.0 ** -100, 0.0, s)
    bad = ~(high - low).isfinite()
    codes = torch.where(bad | (s == 0), 0.0, ((g - low) / s).round().clamp(0, 15))
    s, m = torch.where(bad, math.nan, s), torch.where(bad, math.nan, low)
    return codes.flatten(-2).nan_to_num().to(torch.uint8), torch.cat((s, m), -1).to(torch.bfloat16)


def regions(pool, group):
    """Views of the pool: key codes and scales, value codes and scales, each (pages, heads, blocks, 16, bytes)."""
    d = pool.shape[-1] // 16 * group // (group + 8)
    row, scale = d // 2, d // group * 4
    at, got = 0, []
    for size in (row, scale, row, scale):
        got.append(pool[..., at:at + 16 * size].unflatten(-1, (16, size)))
        at += 16 * size
    return got


def write(pool, table, k, v, sequence, slot, group):
    d, size = k.shape[-1], pool.shape[2] * 16
    page = table[sequence, slot // size].long()
    block, row = slot % size // 16, slot % 16
    kc, ks, vc, vs = regions(pool, group)
    codes, scales = quantise(k, group)
    codes = codes.unflatten(-1, (d // 32, 4, 8)).transpose(-3, -2).flatten(-3)
    kc[page, :, block, row] = codes[..., ::2] | codes[..., 1::2] << 4
    ks[page, :, block, row] = scales.flatten(-2).view(torch.uint8)
    codes, scales = quantise(v, group)
    codes = codes.unflatten(-1, (d // 32, 8, 4)).transpose(-3, -2).flatten(-3)
    vc[page, :, block, row] = codes[..., ::2] | codes[..., 1::2] << 4
    vs[page, :, block, row] = scales.flatten(-2).view(torch.uint8)


def values(pool, table, group):
    """What the pages of the table stand for: keys and values (B, heads, width * page size, D) in 32 bits."""
    got = []
    parts = regions(pool, group)
    for (codes, scales), shape in ((parts[:2], (4, -1, 8)), (parts[2:], (8, -1, 4))):
        codes = codes[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 4)
        scales = scales[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 4).contiguous().view(torch.bfloat16)
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        codes = codes.unflatten(-1, shape).transpose(-3, -2).flatten(-3).unflatten(-1, (-1, group))
        scales = scales.float().unflatten(-1, (-1, 2))
        got.append((codes.float() * scales[..., :1] + scales[..., 1:]).flatten(-2))
    return got


def rows_of(x, start, count, lengths):
    """Rows start .. start + count - 1 of each sequence in bf16, zeros behind its end."""
    at = start.long()[:, None] + torch.arange(count, device=x.device)
    live = at < lengths[:, None]
    at = at.clamp(max=x.shape[2] - 1)[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])
    return torch.where(live[:, None, :, None], x.gather(2, at), 0.0).to(torch.bfloat16)


def plain_rope(s):
    c, pos = s["case"], s["positions"][:, None]
    args = s["table"], c["interleaved"], amplitude(c)
    turned = [rotate(s[n].detach().float(), pos, *args).to(s[n].dtype) for n in ("q", "k")]
    if c["grad"]:
        turned += [rotate(s[n].float(), pos, *args, back=True).to(s[n].dtype) for n in ("gq", "gk")]
    return turned


def plain_append(s):
    c = s["case"]
    k, counts = s["k"], (s["cu_new"][1:] - s["cu_new"][:-1]).long()
    sequence = torch.repeat_interleave(torch.arange(c["batch"], device=k.device), counts, output_size=k.shape[0])
    slot = torch.arange(k.shape[0], device=k.device) - s["cu_new"].long()[sequence] + s["start"].long()[sequence]
    if c["rotary"]:
        k = rotate(k.float(), slot[:, None], s["table"], False, 1.0).to(k.dtype)
    write(s["pool"], s["block_table"], k, s["v"], sequence, slot, c["group"])
    return [rows_of(x, s["start"], c["new"], s["lengths"]) for x in values(s["pool"], s["block_table"], c["group"])]


def plain_decode(s):
    c = s["case"]
    k, v = values(s["pool"], s["block_table"], c["group"])
    n = c["queries"]
    q = s["q"].float().unflatten(1, (c["kv_heads"], -1)).flatten(2, 3)
    scores = q @ k.transpose(-1, -2) / math.sqrt(c["dim"])
    # the last `queries` tokens are the queries' own: each sees up to itself
    seen = s["lengths"][:, None] - torch.arange(n - 1, -1, -1, device=q.device)
    seen = seen.repeat(1, q.shape[2] // n)[:, None, :, None]
    alive = torch.arange(k.shape[2], device=q.device) < seen
    scores = torch.where(alive, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(alive, (scores - top).exp(), 0.0)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    v = torch.where(torch.arange(k.shape[2], device=q.device)[:, None] < s["lengths"][:, None, None, None], v, 0.0)
    o = (p @ v).unflatten(2, (-1, n)).flatten(1, 2).to(torch.bfloat16)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0].unflatten(2, (-1, n)).flatten(1, 2)
    if not c["weights"]:
        return [o, lse]
    live = torch.arange(k.shape[2], device=q.device) < s["lengths"][:, None, None]
    return [o, lse, torch.where(live, s["weights"] + p.sum(2), 0.0)]


def plain_evict(s):
    c, budget = s["case"], s["case"]["budget"]
    weights, where = s["weights"], s["slot_positions"]
    slot = torch.arange(c["tokens"], device=weights.device)
    live = (slot < s["lengths"][:, None, None]).expand_as(weights)
    newest = torch.where(live, where, -1).amax(-1, keepdim=True)
    rank = torch.where(where > newest - c["recent"], math.inf, weights)
    order = torch.argsort(torch.where(live, rank, -1.0), dim=-1, descending=True, stable=True)
    kept = torch.zeros_like(live).scatter_(-1, order[..., :budget], True) & live
    left = s["lengths"].clamp(max=budget)
    inside = slot < left[:, None, None]
    # the n-th kept token behind the new length takes the n-th place that falls free before it
    hole, mover = ~kept & inside, kept & ~inside
    place = (hole.cumsum(-1) - 1).clamp(min=0)
    movers = torch.argsort(~mover, dim=-1, stable=True)
    source = torch.where(hole, movers.gather(-1, place), slot)
    w = torch.where(inside, weights.gather(-1, source), 0.0)
    p = torch.where(inside, where.gather(-1, source), -1)
    source = torch.where(inside, source, -1)[..., :budget].to(torch.int32)
    k, v = values(s["pool"], s["block_table"], c["group"])
    at = source.clamp(min=0).long()[..., None].expand(-1, -1, -1, c["dim"])
    bare = (source < 0)[..., None]
    return [w, p, left, source, *(torch.where(bare, 0.0, x.gather(2, at)).to(torch.bfloat16) for x in (k, v))]


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": own_rope, "append": own_append, "decode": own_decode, "evict": own_evict}[op](state)
    return {"rope": plain_rope, "append": plain_append, "decode": plain_decode, "evict": plain_evict}[op](state)


def own_rope(s):
    import online_softmax_05_gb300 as fa
    c = s["case"]
    turned = fa.rope(s["q"], s["k"], s["table"], s["positions"], interleaved=c["interleaved"], amplitude=amplitude(c))
    if not c["grad"]:
        return list(turned)
    return [t.detach() for t in turned] + list(torch.autograd.grad(turned, (s["q"], s["k"]), (s["gq"], s["gk"])))


def own_append(s):
    import online_softmax_05_gb300 as fa
    c = s["case"]
    fa.kv4_append(s["pool"], s["k"], s["v"], s["block_table"], s["lengths"], s["cu_new"],
                  rotary=s["table"])
    return list(fa.kv4_read(s["pool"], s["block_table"], s["lengths"], start=s["start"], count=c["new"]))


def own_decode(s):
    import online_softmax_05_gb300 as fa
    if s["case"]["weights"]:
        return list(fa.attention_decode_kv4(s["q"], s["pool"], s["block_table"], s["lengths"], causal=True,
                                            weights=s["weights"], weights_out=s["weights_out"]))
    return list(fa.attention_decode_kv4(s["q"], s["pool"], s["block_table"], s["lengths"], causal=True))


def own_evict(s):
    import online_softmax_05_gb300 as fa
    c = s["case"]
    got = fa.kv4_evict(s["pool"], s["block_table"], s["lengths"], s["weights"], s["slot_positions"], c["budget"],
                       c["recent"])
    return list(got) + list(fa.kv4_read(s["pool"], s["block_table"], got[2], count=c["budget"]))


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "append": exact_append, "decode": exact_decode, "evict": exact_evict}[case["op"]](s)


def exact_turn(case, x, positions, back):
    """x (..., T, D) as complex numbers times amplitude * exp(i angle)."""
    f = torch.tensor(frequencies(case), dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(f, amplitude(case)), (-1.0 if back else 1.0) * positions.double()[..., None] * f)
    r = 2 * f.numel()
    x = x.detach().double()
    if case.get("interleaved"):
        z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, x[..., r:]), -1)


def exact_rope(s):
    names = ["q", "k"] + (["gq", "gk"] if s["case"]["grad"] else [])
    return [exact_turn(s["case"], s[n], s["positions"][:, None], n[0] == "g") for n in names]


def exact_append(s):
    c = s["case"]
    held, new = lengths_of(c)
    got = []
    for name in ("k", "v"):
        out = torch.zeros(c["batch"], c["kv_heads"], c["new"], c["dim"], dtype=torch.float64, device=s["k"].device)
        at = 0
        for b, n in enumerate(new):
            x = s[name][at:at + n].double().transpose(0, 1)
            at += n
            if name == "k" and c["rotary"] and n:
                place = torch.arange(held[b] - n, held[b], device=x.device)
                x = exact_turn(c, x, place, False).to(torch.bfloat16).double()
            y = x.reshape(c["kv_heads"], n, c["dim"] // c["group"], c["group"])
            low = y.min(-1, keepdim=True).values if n else y[..., :1]
            step = ((y.max(-1, keepdim=True).values - low) / 15).to(torch.bfloat16).double() if n else y[..., :1]
            out[b, :, :n] = (low + step * torch.round((y - low) / step)).reshape(c["kv_heads"], n, c["dim"])
        got.append(out)
    return got


def exact_values(s, b, n):
    """Keys and values (heads, n, D) of sequence b in 64 bits, each channel looked up at its byte."""
    c, pool = s["case"], s["pool"]
    d, group, size = c["dim"], c["group"], c["page"]
    at = torch.arange(n, device=pool.device)
    blocks = pool[s["block_table"][b].long()[at // size], :, at % size // 16].transpose(0, 1)
    channel, row = torch.arange(d, device=pool.device), at % 16
    g = channel // 32
    key = 8 * (channel % 32 // 8 * (d // 32) + g) + channel % 8
    val = 4 * (channel % 32 // 4 * (d // 32) + g) + channel % 4
    half = 8 * d + 64 * d // group
    got = []
    for base, place in ((0, key), (half, val)):
        byte = base + row[:, None] * (d // 2) + place // 2
        code = blocks.gather(2, byte[None].expand(c["kv_heads"], -1, -1)).long() >> 4 * (place % 2) & 15
        pair = base + 8 * d + row[:, None] * (4 * d // group) + channel // group * 4
        word = [blocks.gather(2, (pair + i)[None].expand(c["kv_heads"], -1, -1)).long() for i in range(4)]
        scale, low = ((word[i] << 16 | word[i + 1] << 24).to(torch.int32).view(torch.float32).double() for i in (0, 2))
        got.append(scale * code + low)
    return got


def exact_decode(s):
    c = s["case"]
    held, _ = lengths_of(c)
    each, n = c["q_heads"] // c["kv_heads"], c["queries"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=s["q"].device)
    w = torch.zeros(s["weights"].shape, dtype=torch.float64, device=s["q"].device) if c["weights"] else None
    for b, length in enumerate(held):
        if not length:
            continue
        k, v = exact_values(s, b, length)
        q = s["q"][b].double().reshape(c["kv_heads"], each, n, c["dim"])
        z = torch.einsum("hgid,htd->hgit", q, k) / math.sqrt(c["dim"])
        hidden = torch.arange(length, device=z.device)[None] > length - n + torch.arange(n, device=z.device)[:, None]
        z = z.masked_fill(hidden, -math.inf)
        total = torch.logsumexp(z, -1)
        p = torch.where(hidden, 0.0, (z - total[..., None]).exp()).nan_to_num(0.0)
        o[b] = torch.einsum("hgit,htd->hgid", p, v).reshape(c["q_heads"], n, c["dim"])
        lse[b] = total.reshape(c["q_heads"], n)
        if w is not None:
            w[b, :, :length] = s["weights"][b, :, :length].double() + p.sum((1, 2))
    return [o, lse] + ([w] if w is not None else [])


def exact_evict(s):
    c = s["case"]
    held, _ = lengths_of(c)
    weights, where = s["weights"].cpu().double().numpy(), s["slot_positions"].cpu().numpy()
    b, h, t = weights.shape
    w = torch.zeros(b, h, t, dtype=torch.float64)
    k = torch.zeros(b, h, c["budget"], c["dim"], dtype=torch.float64)
    v = torch.zeros_like(k)
    for i, length in enumerate(held):
        if not length:
            continue
        left = min(length, c["budget"])
        keys, vals = (x.cpu() for x in exact_values(s, i, length))
        for j in range(h):
            newest = where[i, j, :length].max()
            recent = where[i, j, :length] > newest - c["recent"]
            rank = np.lexsort((np.arange(length), np.where(recent, 0.0, -weights[i, j, :length]), ~recent))
            kept = set(rank[:left].tolist())
            movers = iter(sorted(a for a in kept if a >= left))
            source = [a if a in kept else next(movers) for a in range(left)]
            w[i, j, :left] = torch.from_numpy(weights[i, j, source])
            k[i, j, :left], v[i, j, :left] = keys[j, source], vals[j, source]
    return [w, None, None, None, k, v]
