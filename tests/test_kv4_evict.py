"""Eviction by accumulated weight: what is kept, where it goes and what the cache and
its accounts hold afterwards, exactly; and a serving run of all the operators together."""
import math

import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_05_gb300 import build
    build.build()
    fa.load_library()


def chosen(weights, positions, length, budget, recent):
    """source slots by the definition: sorted(rank), holes filled by the movers in order."""
    left = min(length, budget)
    if length <= budget:
        return list(range(length))
    newest = max(int(p) for p in positions[:length])

    def key(i):
        if int(positions[i]) > newest - recent:
            return (0, 0.0, i)
        w = float(weights[i])
        return (2, 0.0, i) if math.isnan(w) else (1, -w, i)

    kept = set(sorted(range(length), key=key)[:left])
    movers = iter(sorted(i for i in kept if i >= left))
    return [i if i in kept else next(movers) for i in range(left)]


def check(c, w, p, budget, recent):
    pool, table, held = c.on()
    before = c.pool.copy()
    got_w, got_p, got_l, source = fa.kv4_evict(pool, table, held, w.cuda(), p.cuda(), budget, recent)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    B, H, S = w.shape
    want_w, want_p = torch.zeros(B, H, S), torch.full((B, H, S), -1, dtype=torch.int32)
    want_s = torch.full((B, H, budget), -1, dtype=torch.int32)
    want_pool = before.copy()
    parts = ref.sections(c.dim, c.group)

    def place(b, h, slot):
        return c.table[b][slot // c.page], h, slot % c.page // 16

    for b, n in enumerate(c.lengths):
        for h in range(H):
            src = chosen(w[b, h], p[b, h], n, budget, recent)
            want_s[b, h, :len(src)] = torch.tensor(src, dtype=torch.int32)
            want_w[b, h, :len(src)] = w[b, h, src]
            want_p[b, h, :len(src)] = p[b, h, src]
            for to, frm in enumerate(src):
                if to != frm:
                    for at, size in parts:
                        want_pool[place(b, h, to)][at + to % 16 * size:at + (to % 16 + 1) * size] = \
                            before[place(b, h, frm)][at + frm % 16 * size:at + (frm % 16 + 1) * size]
    assert torch.equal(source.cpu(), want_s)
    assert torch.equal(got_p.cpu(), want_p)
    assert np.array_equal(got_w.cpu().numpy(), want_w.numpy(), equal_nan=True)
    assert got_l.tolist() == [min(n, budget) for n in c.lengths]
    assert torch.equal(held.cpu(), torch.tensor(c.lengths, dtype=torch.int32))
    assert np.array_equal(pool.cpu().numpy(), want_pool)


def accounts(c, slots, seed, kind):
    g = torch.Generator().manual_seed(seed)
    shape = len(c.lengths), c.heads, slots
    w = torch.rand(shape, generator=g) * 5
    p = torch.arange(slots, dtype=torch.int32).expand(shape).contiguous()
    if kind == "ties":
        w = torch.randint(0, 3, shape, generator=g).float()
    elif kind == "equal":
        w = torch.ones(shape)
    elif kind == "odd":
        w = torch.randn(shape, generator=g)
        w[..., ::7], w[..., 1::11], w[..., 2::13] = math.nan, math.inf, -math.inf
        w[..., 3::5], w[..., 4::17] = 0.0, -0.0
        p = torch.stack([torch.stack([torch.randperm(slots, generator=g) for _ in range(c.heads)])
                         for _ in c.lengths]).to(torch.int32) * 3 - 40
    elif kind == "low bits":
        w = (torch.randint(0, 50, shape, generator=g).to(torch.int32) + 0x3f800000).view(torch.float32)
    return w, p


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd", "low bits"])
@pytest.mark.parametrize("lengths,budget,recent", [
    ([1, 0, 2], 1, 0), ([1, 0, 2], 1, 1), ([100, 64, 65, 0, 63], 64, 16), ([300, 17], 32, 32), ([257, 130], 128, 0),
    ([1500, 1025, 1024], 1000, 100)])
def test_eviction_is_exact(kind, lengths, budget, recent):
    c = ref.Batch(lengths, 2, 64, 32, 16, seed=budget)
    w, p = accounts(c, max(lengths) + 3, budget + recent, kind)
    check(c, w, p, budget, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", [(128, 64), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("page", [16, 80])
def test_every_format_moves_whole_records(dim, group, page):
    c = ref.Batch([201, 90], 3, dim, group, page, seed=page)
    w, p = accounts(c, 240, 3, "random")
    check(c, w, p, 77, 9)


@pytest.mark.gpu
def test_long_sequences():
    c = ref.Batch([40013, 9000], 1, 64, 64, 64, seed=2)
    w, p = accounts(c, 40013, 4, "low bits")
    check(c, w, p, 5001, 700)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,recent", [("low bits", 5000), ("ties", 0)])
def test_slots_beyond_shared_memory(kind, recent):
    # more slots than the CTAs of a cluster hold in shared memory: read again each pass
    c = ref.Batch([200003], 1, 64, 64, 64, seed=6)
    w, p = accounts(c, 200100, 7, kind)
    check(c, w, p, 30000, recent)


@pytest.mark.gpu
def test_evicting_twice_is_evicting_once():
    # what moved comes from behind the new length, so the same call on the same accounts
    # finds the same pool behind it and repeats the same moves
    c = ref.Batch([500, 300], 2, 64, 32, 16, seed=3)
    w, p = (t.cuda() for t in accounts(c, 500, 5, "random"))
    pool, table, held = c.on()
    a = fa.kv4_evict(pool, table, held, w, p, 128, 10)
    once = pool.clone()
    b = fa.kv4_evict(pool, table, held, w, p, 128, 10)
    assert torch.equal(pool, once) and all(torch.equal(x, y) for x, y in zip(a, b))
    # and going on from the new lengths changes nothing
    d = fa.kv4_evict(pool, table, a[2], a[0], a[1], 128, 10)
    assert torch.equal(pool, once) and torch.equal(d[0], a[0]) and torch.equal(d[2], a[2])


@pytest.mark.gpu
def test_attention_over_the_kept_tokens():
    c = ref.Batch([400, 77], 2, 128, 64, 32, seed=4)
    w, p = accounts(c, 416, 6, "random")
    pool, table, held = c.on()
    q = c.queries(8, 1)
    got = fa.kv4_evict(pool, table, held, w.cuda(), p.cuda(), 100, 20)
    o, lse = fa.attention_decode_kv4(q.cuda(), pool, table, got[2])
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    source = got[3].cpu()
    for b, n in enumerate(c.lengths):
        loaded = c.loaded(b)
        for h in range(2):
            src = source[b, h, :min(n, 100)].long().numpy()
            part = [x[h:h + 1, src] for x in loaded]
            rows = slice(4 * h, 4 * h + 4)
            wo, wl, _, most, weighed = ref.attend(q[b, rows].double().numpy(), part, 128 ** -0.5, True)
            assert (np.abs(o[b, rows].cpu().double().numpy() - wo) <= ref.o_tol(wo, most, weighed)).all()
            assert (np.abs(lse[b, rows].cpu().double().numpy() - wl) <= ref.lse_tol(wl, most)).all()


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported():
    c = ref.Batch([100, 60], 2, 64, 64, 16, seed=15)
    w, p = (t.cuda() for t in accounts(c, 112, 6, "random"))
    pool, table, held = c.on()
    keep = pool.clone()
    for bad in (torch.tensor([113, 60]), torch.tensor([-1, 60])):
        got = fa.kv4_evict(pool, table, bad.int().cuda(), w, p, 64, 4)
        assert fa.fa_get_device_status() == -11
        assert got[2].tolist() == [0, 60] and torch.equal(pool, keep)
    broken = table.clone()
    broken[0, :2] = -1
    fa.kv4_evict(pool, broken, held, w, p, 64, 4)
    assert fa.fa_get_device_status() == -13
    short = w[:, :, :90].contiguous(), p[:, :, :90].contiguous()   # accounts shorter than a sequence
    got = fa.kv4_evict(pool, table, held, *short, 64, 4)
    assert fa.fa_get_device_status() == -11 and got[2].tolist() == [0, 60]


@pytest.mark.gpu
def test_graph_and_stream():
    c = ref.Batch([500, 300], 2, 64, 32, 16, seed=3)
    w, p = (t.cuda() for t in accounts(c, 500, 5, "random"))
    pool, table, held = c.on()
    pool2 = pool.clone()
    want = fa.kv4_evict(pool, table, held, w, p, 128, 10)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fa.kv4_evict(pool2.clone(), table, held, w, p, 128, 10, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    static = w.flip(2).contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = fa.kv4_evict(pool2, table, held, static, p, 128, 10)
    static.copy_(w)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(cap, want)) and torch.equal(pool2, pool)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group,each", [(128, 64, 4), (64, 32, 2)])
def test_a_serving_run(dim, group, each):
    """Prompts appended, steps decoded with weights, the cache cut to its budget, steps
    again: after every step the output equals attention in 64 bits over the tokens that a
    plain simulation says each head still holds."""
    heads, page, budget, recent = 2, 16, 40, 8
    prompts, steps = [30, 57, 1], 24
    B, hq = len(prompts), heads * each
    rng = np.random.default_rng(dim)
    table_f = fa.rotary_frequencies(dim, scaling="parts", factor=4.0, original_length=256, device="cuda")
    amp = fa.rotary_amplitude(4.0)
    width = -(-(max(prompts) + steps + 1) // page)
    pool = fa.kv4_pool(B * width + 1, heads, dim, page_size=page, group=group)
    table = torch.from_numpy(rng.permutation(B * width + 1)[:B * width].reshape(B, width).astype(np.int32)).cuda()
    slots = width * page
    weights = torch.zeros(B, heads, slots, device="cuda")
    where = torch.full((B, heads, slots), -1, dtype=torch.int32, device="cuda")
    held = torch.tensor(prompts, dtype=torch.int32).cuda()
    seen = torch.tensor(prompts, dtype=torch.int64).cuda()
    # plain simulation: for each head the list of (position, account), in slots, and their records
    sim = [[[] for _ in range(heads)] for _ in range(B)]
    shadow = [[np.zeros((4, 0, dim)) for _ in range(heads)] for _ in range(B)]

    def new(n):
        return tuple(ref.bf16(rng.standard_normal((n, heads, dim))) for _ in range(2))

    def append(counts, first):
        k, v = new(sum(counts))
        cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
        pos = torch.cat([torch.arange(f, f + n) for f, n in zip(first, counts)])
        fa.kv4_append(pool, k.cuda(), v.cuda(), table, held, cu, rotary=table_f, positions=pos.cuda(), amplitude=amp,
                      weights=weights, slot_positions=where)
        turned = fa.rope(k.transpose(0, 1)[None].cuda(), None, table_f, pos.cuda(), amplitude=amp)[0].cpu()
        at = 0
        for b, n in enumerate(counts):
            for i in range(n):
                for h in range(heads):
                    kc, ksc, km = ref.quantise(turned[h, at].float().numpy(), group)
                    vc, vsc, vm = ref.quantise(v[at, h].float().numpy(), group)
                    wide = lambda x: np.repeat(x.astype(np.float64), group)  # noqa: E731
                    row = np.stack((wide(ksc) * kc, wide(km), wide(vsc) * vc, wide(vm)))[:, None]
                    shadow[b][h] = np.concatenate((shadow[b][h], row), 1)
                    sim[b][h].append(first[b] + i)
                at += 1

    append(prompts, [0] * B)
    for step in range(steps):
        append_at = seen.tolist()
        held += 1
        seen += 1
        append([1] * B, append_at)
        q = ref.bf16(rng.standard_normal((B, hq, 1, dim)))
        qr = fa.rope(q.cuda(), None, table_f, (seen - 1)[:, None], amplitude=amp)
        o, lse, _ = fa.attention_decode_kv4(qr, pool, table, held, weights=weights)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == 0
        for b in range(B):
            for h in range(heads):
                rows = slice(h * each, (h + 1) * each)
                loaded = [x[None] for x in shadow[b][h]]
                wo, wl, _, most, weighed = ref.attend(qr[b, rows].cpu().double().numpy(), loaded, dim ** -0.5, True)
                assert (np.abs(o[b, rows].cpu().double().numpy() - wo) <= ref.o_tol(wo, most, weighed)).all()
                assert (np.abs(lse[b, rows].cpu().double().numpy() - wl) <= ref.lse_tol(wl, most)).all()
                assert where[b, h, :int(held[b])].tolist() == sim[b][h]
        if step % 6 == 5:
            account = weights.cpu()
            lengths = held.tolist()
            weights, where, held, _ = fa.kv4_evict(pool, table, held, weights, where, budget, recent)
            for b in range(B):
                for h in range(heads):
                    src = chosen(account[b, h], sim[b][h], lengths[b], budget, recent)
                    sim[b][h] = [sim[b][h][i] for i in src]
                    shadow[b][h] = shadow[b][h][:, src]
            assert held.tolist() == [min(n, budget) for n in lengths]


@pytest.mark.gpu
def test_a_captured_step_between_other_work():
    """One serving step captured with fills, copies and library kernels before and between
    the operators, on a stream that waits for another: replays equal the eager step."""
    B, heads, hq, dim, page = 3, 2, 8, 128, 16
    c = ref.Batch([200, 33, 64], heads, dim, 64, page, seed=21, spare=2)
    pool, table, held = c.on()
    slots = table.shape[1] * page
    used = set(c.table[c.table >= 0].tolist())
    free = [i for i in range(c.pool.shape[0]) if i not in used]
    for b in range(2):          # the two spare pages go to the sequences that need one for a new token
        row = c.table[b]
        row[np.argmax(row < 0)] = free[b]
    c.lengths[2] = 60
    table = torch.from_numpy(c.table).cuda()
    held = torch.tensor(c.lengths, dtype=torch.int32).cuda()
    freq = fa.rotary_frequencies(dim, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    qkv = torch.randn(B, 1, hq + 2 * heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    weights = torch.rand(B, heads, slots, device="cuda", generator=g)
    where = torch.arange(slots, dtype=torch.int32, device="cuda").expand(B, heads, slots).contiguous()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def step(qkv, pool, held, weights, where):
        lengths = torch.zeros_like(held)
        lengths.copy_(held)
        lengths += 1
        x = qkv.transpose(1, 2)
        pos = (lengths - 1)[:, None]
        q = fa.rope(x[:, :hq], None, freq, pos)
        fa.kv4_append(pool, qkv[:, 0, hq:hq + heads], qkv[:, 0, hq + heads:], table, lengths, cu, rotary=freq,
                      positions=pos[:, 0].contiguous(), weights=weights, slot_positions=where)
        o, lse, w = fa.attention_decode_kv4(q, pool, table, lengths, weights=weights)
        o = o * 1.0
        got = fa.kv4_evict(pool, table, lengths, w, where, 50, 8)
        k, v = fa.kv4_read(pool, table, got[2], count=50)
        return [o, lse, *got, k, v, pool.clone()]

    base = [t.clone() for t in (qkv, pool, held, weights, where)]
    want = step(*[t.clone() for t in base])
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    static = [t.clone() for t in base]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*[t.clone() for t in base])        # what capture needs to have run once
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for _ in range(3):
        for s, b in zip(static, base):
            s.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    # and eagerly on another stream, ordered by events alone
    for _ in range(3):
        fresh = [t.clone() for t in base]
        fresh[0].mul_(1.0)
        ev = torch.cuda.Event()
        ev.record()
        side.wait_event(ev)
        with torch.cuda.stream(side):
            got = step(*fresh)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
