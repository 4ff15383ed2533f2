"""What is measured of the attention whose queries are not the keys' own sequence:
cross attention to states of another length (forward, gradients, and a few rows
per sequence), attention of a tree of drafted tokens over the 4-bit paged cache,
and keeping the accepted part of such a tree in the cache.

`run` computes a case in elementary torch operations, or with `own` set through
the package's entry points, on the same state.

The 4-bit cache, as both sides hold it: a byte tensor of
(pages, kv heads, page size / 16, block bytes).  A block is 16 tokens of one
head: key codes (16 x D/2 bytes), key scales (16 x D/group pairs of bf16), value
codes, value scales.  A group of `group` channels holds
s = bf16((max - min) / 15), m = min and the codes round((x - m) / s); it stands
for s * code + m.  Key channel 32 g + 8 j + i is nibble i of the row's 32-bit
word j D/32 + g; value channel 32 g + 4 r + i is nibble i of its 16-bit
half-word r D/32 + g.

A tree of drafted tokens takes the last `places` slots of its sequence.
parents[b, i] is the place of i's parent, below i, or -1 behind the context; any
other value marks a place without a token, and what hangs on it."""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
GOLDEN = 0.6180339887498949
EMPTY = -2  # a place of a tree that holds no token
VOCABULARY = 32000


# ------------------------------------------------------------------ cases

def listed():
    return [
        # training: a decoder layer's attention to encoded texts of different lengths
        dict(name="cross_train", op="cross", batch=4, q_heads=16, kv_heads=16, queries=2048, keys=3000, dim=64,
             ragged=True, fused=True, grad=True),
        # training on long sources with grouped heads, every source of full length
        dict(name="cross_train_grouped", op="cross", batch=2, q_heads=32, kv_heads=8, queries=1024, keys=8192, dim=128,
             ragged=False, fused=False, grad=True),
        # the forward pass of prompts against sources of different lengths, one of them empty
        dict(name="cross_prompt", op="cross", batch=8, q_heads=32, kv_heads=32, queries=333, keys=3000, dim=128,
             ragged=True, fused=True, grad=False),
        # the largest: both sides long
        dict(name="cross_long", op="cross", batch=2, q_heads=16, kv_heads=16, queries=8192, keys=8192, dim=128,
             ragged=False, fused=False, grad=True),
        # one token of one conversation: latency
        dict(name="cross_token", op="cross", batch=1, q_heads=8, kv_heads=8, queries=1, keys=1500, dim=64,
             ragged=False, fused=True, grad=False),
        # a token for each sequence of a serving batch, grouped heads, sources of different lengths
        dict(name="cross_step", op="cross", batch=32, q_heads=32, kv_heads=8, queries=1, keys=3000, dim=128,
             ragged=True, fused=True, grad=False),
        # a few rows (beams, or a draft's tokens) against long sources: the repository's decoding shape
        dict(name="cross_rows", op="cross", batch=8, q_heads=32, kv_heads=32, queries=5, keys=32768, dim=128,
             ragged=False, fused=False, grad=False),
        # checking a small tree in a young conversation: latency
        dict(name="tree_small", op="tree", batch=1, places=8, tokens=117, q_heads=8, kv_heads=2, dim=64, group=64,
             page=16, ragged=False),
        # a serving batch with trees of different sizes over caches of different lengths, one sequence ended
        dict(name="tree_batch", op="tree", batch=8, places=32, tokens=12345, q_heads=32, kv_heads=8, dim=128, group=64,
             page=64, ragged=True),
        # wide trees and many query heads to a key/value head, fine groups, small pages
        dict(name="tree_wide", op="tree", batch=4, places=64, tokens=8111, q_heads=32, kv_heads=4, dim=128, group=32,
             page=16, ragged=True),
        # what follows a model's pass over a batch's trees: accept, keep, read back
        dict(name="keep_batch", op="keep", batch=32, places=16, tokens=4106, q_heads=8, kv_heads=8, dim=128, group=64,
             page=64, ragged=True),
        # large trees of a few sequences, small heads, finer groups, pages the tree starts and ends inside
        dict(name="keep_wide", op="keep", batch=5, places=61, tokens=1064, q_heads=4, kv_heads=4, dim=64, group=32,
             page=16, ragged=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["cross", "cross", "cross", "tree", "tree", "keep"])
    dim, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16, 32])
    batch = log(1, 32)
    if op == "cross":
        q_heads = kv_heads * rng.choice([1, 1, 2, 4, 7]) if kv_heads < 16 else kv_heads
        grad = rng.random() < 0.5
        queries = rng.choice([1, log(1, 64), log(16, 8192), log(16, 8192)])
        most = (1 << 30 if grad else 1 << 31) // (batch * q_heads * queries)  # scores
        most = min(most, (1 << 29 if grad else 1 << 30) // (batch * kv_heads * dim))  # elements of the keys
        queries = min(queries, (1 << 27) // (batch * q_heads * dim))
        return dict(op=op, batch=batch, q_heads=q_heads, kv_heads=kv_heads, queries=max(1, queries),
                    keys=max(1, min(log(1, 32768), most)), dim=dim, ragged=rng.random() < 0.6,
                    fused=rng.random() < 0.5, grad=grad)
    group, page, places = rng.choice([32, 64]), rng.choice([16, 32, 64, 128]), log(1, 64)
    if op == "keep":
        return dict(op=op, batch=batch, places=places, tokens=places + log(1, 4096), q_heads=kv_heads,
                    kv_heads=kv_heads, dim=dim, group=group, page=page, ragged=rng.random() < 0.7)
    each = rng.choice([1, 3, 4, 8])
    kv_heads = min(kv_heads, 64 // each)
    most = min((1 << 22) // (batch * kv_heads), (1 << 29) // (batch * kv_heads * each * places))
    return dict(op=op, batch=batch, places=places, tokens=max(places, min(log(1, 65536), most)),
                q_heads=kv_heads * each, kv_heads=kv_heads, dim=dim, group=group, page=page,
                ragged=rng.random() < 0.7)


def spread(count, most, least, phase, ragged):
    """`count` whole numbers of [least, most], the first `most`: the lengths of a batch."""
    if not ragged:
        return [most] * count
    return [most] + [least + int((most - least) * ((b * GOLDEN + phase) % 1.0)) for b in range(1, count)]


def lengths_of(case):
    """Keys of each sequence, or the tokens that the cache holds of it, its tree's places among them."""
    if case["op"] == "cross":
        held = spread(case["batch"], case["keys"], 1, 0.41, case["ragged"])
    else:
        held = spread(case["batch"], case["tokens"], case["places"], 0.53, case["ragged"])
    # a ragged batch holds an empty sequence too: a slot whose request has ended
    if case["ragged"] and case["batch"] > 3:
        held[2] = 0
    return held


def block_bytes(case):
    return 16 * (case["dim"] + 8 * case["dim"] // case["group"])


def work(case):
    d, held = case["dim"], lengths_of(case)
    if case["op"] == "cross":
        rows = case["batch"] * case["q_heads"] * case["queries"]
        keys = sum(held) * case["kv_heads"]
        pairs = sum(held) * case["q_heads"] * case["queries"]
        # queries and outputs, keys and values of the real lengths, a log-sum-exp a row
        size = {"bytes": 4 * rows * d + 4 * keys * d + 4 * rows, "flops": 4 * d * pairs}
        if case["grad"]:
            # the output's gradient, and the gradients of all three, padding too; four products and the recomputed scores
            every = case["batch"] * case["keys"] * case["kv_heads"]
            size = {"bytes": size["bytes"] + 4 * rows * d + 4 * every * d, "flops": size["flops"] + 10 * d * pairs}
        return size
    token = block_bytes(case) // 16  # codes and scales, keys and values
    if case["op"] == "tree":
        n = sum(held) * case["kv_heads"]
        rows = case["batch"] * case["q_heads"] * case["places"]
        return {"bytes": n * token + rows * (4 * d + 4) + 4 * case["batch"] * case["places"],
                "flops": 4 * d * n * (case["q_heads"] // case["kv_heads"]) * case["places"]}
    n = case["batch"] * case["places"] * case["kv_heads"]
    # keys and values in, codes out, about half of them moved, and the kept part read back into padded rows
    return {"bytes": n * (4 * d + token) + n * token + n // 2 * token + n * 4 * d, "flops": n * (2 * d * 5 + 2 * d * 2)}


# ------------------------------------------------------------------ inputs

def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE)


def heads_like(gen, n, heads, dim):
    """Keys or values (n, heads, dim) in bf16: normal, with a gain and an offset for each channel as projections have them."""
    gain = torch.rand(heads, dim, generator=gen, device=DEVICE) * 0.6 + 0.7
    shift = normal(gen, heads, dim) * 0.3
    return (normal(gen, n, heads, dim) * gain + shift).to(torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


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


def filled(case, gen, held):
    pool, table = paged(case, gen, held)
    total = sum(held)
    if total:
        step = max(1, (1 << 27) // (case["kv_heads"] * case["dim"]))
        gains = gen.initial_seed()
        sequence = torch.repeat_interleave(torch.arange(len(held), device=DEVICE), ints(held))
        before = torch.cumsum(ints(held).long(), 0) - ints(held)
        slot = torch.arange(total, device=DEVICE) - before[sequence]
        for lo in range(0, total, step):
            n = min(step, total - lo)
            part = torch.Generator(DEVICE).manual_seed(gains + 7 * lo + 1)
            write(pool, table, heads_like(part, n, case["kv_heads"], case["dim"]),
                  heads_like(part, n, case["kv_heads"], case["dim"]), sequence[lo:lo + n], slot[lo:lo + n],
                  case["group"])
    return pool, table


def trees(case, gen):
    """Parents (B, places): each token hangs on one of the few before it, as a draft is grown from its likeliest ends;
    of a ragged batch, the places behind a tree's size are empty."""
    b, n = case["batch"], case["places"]
    place = torch.arange(n, device=DEVICE)
    back = (torch.rand(b, n, generator=gen, device=DEVICE) ** 2 * torch.minimum(place, ints(9))).int()
    parents = (place - 1 - back).int()
    size = ints(spread(b, n, (n + 1) // 2, 0.23, case["ragged"]))
    return torch.where(place < size[:, None], parents, EMPTY).int().contiguous()


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    held = lengths_of(case)
    s = {"case": case, "lengths": ints(held)}
    b, d, hq, hk = case["batch"], case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "cross":
        tq, tk = case["queries"], case["keys"]
        if case["fused"]:  # heads behind tokens, keys and values side by side in one projection's output
            s["q"] = normal(gen, b, tq, hq, d).to(torch.bfloat16).transpose(1, 2)
            both = heads_like(gen, b * tk, 2 * hk, d).view(b, tk, 2 * hk, d).transpose(1, 2)
            s["k"], s["v"] = both[:, :hk], both[:, hk:]
        else:
            s["q"] = normal(gen, b, hq, tq, d).to(torch.bfloat16)
            s["k"], s["v"] = (heads_like(gen, b * tk, hk, d).view(b, tk, hk, d).transpose(1, 2).contiguous()
                              for _ in range(2))
        if not case["ragged"]:
            s["lengths"] = None
        if case["grad"]:
            s["q"], s["k"], s["v"] = (s[n].detach().requires_grad_() for n in "qkv")
            s["do"] = normal(gen, b, hq, tq, d).to(torch.bfloat16)
        return s
    n = case["places"]
    s["parents"] = trees(case, gen)
    s["pool"], s["block_table"] = filled(case, gen, held)
    if case["op"] == "tree":
        s["q"] = normal(gen, b, hq, n, d).to(torch.bfloat16)
        return s
    s["start"] = (s["lengths"] - n).clamp(min=0)
    counts = torch.where(s["lengths"] > 0, n, 0)
    s["cu_new"] = torch.cat((ints([0]), counts.cumsum(0).int()))
    total = sum(n for h in held if h)
    s["k"], s["v"] = heads_like(gen, total, hk, d), heads_like(gen, total, hk, d)
    # the model picks what was drafted as one place's child two times in three, something else otherwise
    s["tokens"] = torch.randint(0, VOCABULARY, (b, n), generator=gen, device=DEVICE)
    s["picks"] = torch.randint(0, VOCABULARY, (b, n), generator=gen, device=DEVICE)
    likely = torch.rand(b, n, generator=gen, device=DEVICE) < 0.67
    s["first"] = s["tokens"][:, 0].contiguous()
    hung = (s["parents"] >= 0) & likely
    drafted = torch.zeros(b, n + 1, dtype=torch.int64, device=DEVICE).scatter_reduce(
        1, torch.where(hung, s["parents"], n).long(), s["tokens"], "amax")[:, :n]
    s["picks"] = torch.where(drafted > 0, drafted, s["picks"])
    return s


# ------------------------------------------------------------------ the cache in plain torch

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
    row, scale = 16 * (d // 2), 16 * (d // group * 4)
    cuts = pool.split((row, scale, row, scale), -1)
    return [part.unflatten(-1, (16, -1)) for part in cuts]


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
    kc, ks, vc, vs = regions(pool, group)
    return [value(kc, ks, table, group, (4, -1, 8)), value(vc, vs, table, group, (8, -1, 4))]


def value(codes, scales, table, group, shape):
    codes = codes[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 4)
    scales = scales[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 4).contiguous().view(torch.bfloat16)
    codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    codes = codes.unflatten(-1, shape).transpose(-3, -2).flatten(-3).unflatten(-1, (-1, group))
    scales = scales.float().unflatten(-1, (-1, 2))
    return (codes.float() * scales[..., :1] + scales[..., 1:]).flatten(-2)


def rows_of(x, start, count, lengths):
    """Rows start .. start + count - 1 of each sequence in bf16, zeros behind its end."""
    at = start.long()[:, None] + torch.arange(count, device=x.device)
    live = at < lengths[:, None]
    at = at.clamp(max=x.shape[2] - 1)[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])
    return torch.where(live[:, None, :, None], x.gather(2, at), 0.0).to(torch.bfloat16)


# ------------------------------------------------------------------ plain forms

def softmax_of(scores, alive):
    """Weights and log-sum-exps of the rows; a row without a living score has weights 0 and -infinity."""
    scores = torch.where(alive, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(alive, (scores - top).exp(), 0.0)
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0), torch.where(total > 0, top + total.log(), -math.inf)[..., 0]


def plain_cross(s):
    c = s["case"]
    k, v = s["k"].detach().float(), s["v"].detach().float()
    scale, each = 1 / math.sqrt(c["dim"]), c["q_heads"] // c["kv_heads"]
    q = s["q"].detach().float().unflatten(1, (-1, each)).flatten(2, 3)  # the rows of a key/value head
    key = torch.arange(c["keys"], device=q.device)
    held = key.new_full((c["batch"],), c["keys"]) if s["lengths"] is None else s["lengths"]
    alive = (key < held[:, None])[:, None]  # (B, 1, keys)
    v = torch.where(alive[..., None], v, 0.0)
    k = torch.where(alive[..., None], k, 0.0)
    p, lse = softmax_of(q @ k.transpose(-1, -2) * scale, alive[:, :, None])
    o = p @ v
    out = o.unflatten(2, (each, -1)).flatten(1, 2).to(torch.bfloat16)
    if not c["grad"]:
        return [out, lse.unflatten(2, (each, -1)).flatten(1, 2)]
    do = s["do"].float().unflatten(1, (-1, each)).flatten(2, 3)
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.transpose(-1, -2)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k * scale).unflatten(2, (each, -1)).flatten(1, 2)
    dk = ds.transpose(-1, -2) @ q * scale
    return [out] + [x.to(torch.bfloat16) for x in (dq, dk, dv)]


def reached(parents):
    """(B, places, places): whether i is j or hangs on it, through places that hold tokens."""
    n = parents.shape[1]
    place = torch.arange(n, device=parents.device)
    root = parents == -1
    up = (parents[..., None] == place) & (place < place[:, None]) & (parents[..., None] >= 0)
    steps = torch.linalg.matrix_power(up.float() + torch.eye(n, device=parents.device), n) > 0
    alive = (steps & root[:, None]).any(-1)
    return steps & alive[..., None]


def plain_tree(s):
    c, n = s["case"], s["case"]["places"]
    k, v = values(s["pool"], s["block_table"], c["group"])
    q = s["q"].float().unflatten(1, (c["kv_heads"], -1)).flatten(2, 3)
    slot = torch.arange(k.shape[2], device=q.device)
    place = slot - (s["lengths"][:, None] - n)  # of each slot in its sequence's tree
    held = slot < s["lengths"][:, None]
    sees = reached(s["parents"]).gather(2, place.clamp(0, n - 1)[:, None].expand(-1, n, -1).long())
    # a place that holds no token sees nothing, the context neither
    filled_place = reached(s["parents"]).any(-1)[..., None]
    alive = held[:, None] & torch.where(place[:, None] < 0, filled_place, sees)
    alive = alive.repeat(1, q.shape[2] // n, 1)[:, None]
    p, lse = softmax_of(q @ k.transpose(-1, -2) / math.sqrt(c["dim"]), alive)
    v = torch.where(held[:, None, :, None], v, 0.0)
    o = (p @ v).unflatten(2, (-1, n)).flatten(1, 2).to(torch.bfloat16)
    return [o, lse.unflatten(2, (-1, n)).flatten(1, 2)]


def plain_keep(s):
    c, n, pool = s["case"], s["case"]["places"], s["pool"]
    size = pool.shape[2] * 16
    new = s["cu_new"].long()
    sequence = torch.repeat_interleave(torch.arange(c["batch"], device=pool.device), new[1:] - new[:-1],
                                       output_size=s["k"].shape[0])
    place = torch.arange(n, device=pool.device)
    at = torch.arange(s["k"].shape[0], device=pool.device) - new[sequence]
    write(pool, s["block_table"], s["k"], s["v"], sequence, s["start"].long()[sequence] + at, c["group"])
    # accepted: every token on the way is what the model picked before it
    parents, tokens = s["parents"], s["tokens"]
    reach = reached(parents)
    before = torch.where(parents == -1, s["first"][:, None], s["picks"].gather(1, parents.clamp(min=0).long()))
    wrong = tokens != before
    good = reach.any(-1) & ~(reach & wrong[:, None]).any(-1)
    depth = reach.sum(-1)
    best, end = torch.where(good, depth * n + (n - 1 - place), -1).max(-1)
    counts = torch.where(best >= 0, depth.gather(1, end[:, None])[:, 0], 0)
    way = reach.gather(1, end[:, None, None].expand(-1, 1, n))[:, 0]
    path = torch.where(way, place, n).sort(-1).values
    path = torch.where(place < counts[:, None], path, -1)
    follow = torch.where(counts > 0, s["picks"].gather(1, end[:, None])[:, 0], s["first"])
    # the accepted tokens move to the first of the tree's slots
    live = (s["lengths"] > 0)[:, None] & (path >= 0)
    source = s["start"].long()[:, None] + torch.where(live, path, place)
    target = s["start"].long()[:, None] + place
    width = s["block_table"].shape[1]
    row = [(torch.where(s["lengths"][:, None] > 0, s["block_table"].gather(1, (x // size).clamp(max=width - 1)), 0).long(),
            x % size // 16, x % 16) for x in (source, target)]
    page, block, r = (x[live] for x in row[0])
    to_page, to_block, to_r = (x[live] for x in row[1])
    kc, ks, vc, vs = regions(pool, c["group"])
    moved = kc[page, :, block, r], ks[page, :, block, r], vc[page, :, block, r], vs[page, :, block, r]
    kc[to_page, :, to_block, to_r], ks[to_page, :, to_block, to_r] = moved[:2]
    vc[to_page, :, to_block, to_r], vs[to_page, :, to_block, to_r] = moved[2:]
    lengths = torch.where(s["lengths"] > 0, s["start"] + counts, 0).int()
    k, v = (rows_of(x, s["start"], n, lengths) for x in values(pool, s["block_table"], c["group"]))
    return [path.int(), counts.int(), follow, lengths, k, v]


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"cross": own_cross, "tree": own_tree, "keep": own_keep}[op](state)
    return {"cross": plain_cross, "tree": plain_tree, "keep": plain_keep}[op](state)


def own_cross(s):
    import online_softmax_05_gb300 as fa
    if not s["case"]["grad"]:
        return list(fa.attention_forward_cross(s["q"], s["k"], s["v"], s["lengths"]))
    o = fa.cross_attention(s["q"], s["k"], s["v"], s["lengths"])
    return [o.detach()] + list(torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"]))


def own_tree(s):
    import online_softmax_05_gb300 as fa
    return list(fa.attention_tree_kv4(s["q"], s["pool"], s["block_table"], s["lengths"], s["parents"]))


def own_keep(s):
    import online_softmax_05_gb300 as fa
    fa.kv4_append(s["pool"], s["k"], s["v"], s["block_table"], s["lengths"], s["cu_new"])
    path, counts, follow = fa.tree_accept(s["parents"], s["tokens"], s["picks"], s["first"])
    lengths = fa.kv4_keep(s["pool"], s["block_table"], s["lengths"], path)
    k, v = fa.kv4_read(s["pool"], s["block_table"], lengths, start=s["start"], count=s["case"]["places"])
    return [path, counts, follow, lengths, k, v]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"cross": exact_cross, "tree": exact_tree, "keep": exact_keep}[case["op"]](s)


def exact_cross(s):
    c = s["case"]
    q, k, v = (s[n].detach() for n in "qkv")
    each = c["q_heads"] // c["kv_heads"]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v))
    for b, length in enumerate(lengths_of(c)):
        for h in range(c["q_heads"] if length else 0):
            x, y, z = q[b, h].double(), k[b, h // each, :length].double(), v[b, h // each, :length].double()
            score = torch.einsum("id,jd->ij", x, y) / c["dim"] ** 0.5
            lse[b, h] = torch.logsumexp(score, -1)
            p = score.sub_(lse[b, h][:, None]).exp_()
            o[b, h] = torch.einsum("ij,jd->id", p, z)
            if c["grad"]:
                g = s["do"][b, h].double()
                dv[b, h // each, :length] += torch.einsum("ij,id->jd", p, g)
                t = torch.einsum("id,jd->ij", g, z)
                t = (t - (p * t).sum(-1, keepdim=True)) * p / c["dim"] ** 0.5
                dq[b, h] = torch.einsum("ij,jd->id", t, y)
                dk[b, h // each, :length] += torch.einsum("ij,id->jd", t, x)
    return [o, dq, dk, dv] if c["grad"] else [o, lse]


def exact_values(s, b, slots):
    """Keys and values (heads, slots, D) of sequence b in 64 bits, each channel looked up at its byte."""
    c, pool = s["case"], s["pool"]
    d, group, size = c["dim"], c["group"], c["page"]
    at = torch.as_tensor(slots, device=pool.device)
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


def ways(parents):
    """For each place of one tree, the places from the root to it, or None where it holds no token."""
    found = []
    for i, p in enumerate(parents):
        if p == -1:
            found.append([i])
        else:
            found.append(found[p] + [i] if 0 <= p < i and found[p] is not None else None)
    return found


def exact_tree(s):
    c, n = s["case"], s["case"]["places"]
    each = c["q_heads"] // c["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=s["q"].device)
    every = s["parents"].tolist()
    for b, length in enumerate(lengths_of(c)):
        if not length:
            continue
        k, v = exact_values(s, b, range(length))
        hidden = torch.ones(n, length, dtype=torch.bool)
        for i, way in enumerate(ways(every[b])):
            if way is not None:
                hidden[i, :length - n] = False
                hidden[i, [length - n + j for j in way]] = False
        hidden = hidden.to(k.device)
        empty = hidden.all(-1)[:, None]
        for h in range(c["q_heads"]):
            z = s["q"][b, h].double() @ k[h // each].T / math.sqrt(c["dim"])
            z = z.masked_fill(hidden, -math.inf)
            lse[b, h] = torch.logsumexp(z, -1)
            o[b, h] = torch.where(empty, 0.0, torch.softmax(z, -1).nan_to_num(0.0) @ v[h // each])
    return [o, lse]


def exact_keep(s):
    """The kept tokens from the model's own keys and values, rounded to their codes in 64 bits."""
    c, n = s["case"], s["case"]["places"]
    parents, tokens, picks, first = (s[x].tolist() for x in ("parents", "tokens", "picks", "first"))
    k = torch.zeros(c["batch"], c["kv_heads"], n, c["dim"], dtype=torch.float64, device=s["k"].device)
    v = torch.zeros_like(k)
    at = 0
    for b, length in enumerate(lengths_of(c)):
        best = []
        for way in ways(parents[b]):
            if way is not None and len(way) > len(best):
                before = [first[b]] + [picks[b][j] for j in way[:-1]]
                if all(tokens[b][j] == x for j, x in zip(way, before)):
                    best = way
        if not length:
            continue
        for out, x in ((k, s["k"]), (v, s["v"])):
            y = x[at:at + n][best].double().transpose(0, 1)
            y = y.reshape(c["kv_heads"], len(best), c["dim"] // c["group"], c["group"])
            if best:
                low = y.min(-1, keepdim=True).values
                step = ((y.max(-1, keepdim=True).values - low) / 15).to(torch.bfloat16).double()
                y = low + step * torch.round((y - low) / step)
            out[b, :, :len(best)] = y.reshape(c["kv_heads"], len(best), c["dim"])
        at += n
    return [None, None, None, None, k, v]
