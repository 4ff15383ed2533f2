"""Which drafted tokens stand (tree_accept), keeping them in the 4-bit cache (kv4_keep),
and a decoder's step with drafts, all of it together."""
import struct

import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as ref
from tests.cross_ref import check as check_cross
from tests.cross_ref import reference
from tests.test_kv4_tree import check as check_tree
from tests.test_kv4_tree import trees, ways


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_05_gb300 import build
    build.build()
    fa.load_library()


def accepted(parents, tokens, picks, first):
    """(path, next) of one tree, place by place."""
    best = []
    for i, way in enumerate(ways(parents)):
        if way is None:
            continue
        way = sorted(way)
        before = [first] + [picks[j] for j in way[:-1]]
        if all(x is None or tokens[j] == x for j, x in zip(way, before)) and len(way) > len(best):
            best = way
    return best, picks[best[-1]] if best else (-1 if first is None else first)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("with_first", [True, False])
def test_accept(n, dtype, with_first):
    B = 67
    rng = np.random.default_rng(n)
    parents = trees(B, n, seed=n)
    parents[0] = -2
    parents[1] = np.arange(-1, n - 1)
    if n > 2:
        parents[2, -1] = -2147483648
    # few different tokens, so that picks agree with several children, or none
    tokens, picks = rng.integers(0, 3, (2, B, n))
    first = rng.integers(0, 3, B)
    tokens[1], picks[1], first[1] = 1, 1, 1  # the chain stands as a whole
    big = (1 << 40) if dtype is torch.int64 else 0  # differences in the upper half count
    cuda = [torch.from_numpy(x).to(dtype).cuda() for x in (tokens, picks, first)]
    cuda[1][5:] += big
    path, counts, follow = fa.tree_accept(torch.from_numpy(parents).cuda(), cuda[0], cuda[1],
                                          cuda[2] if with_first else None)
    picks = cuda[1].cpu().numpy()
    for b in range(B):
        want, after = accepted(parents[b], tokens[b], picks[b], first[b] if with_first else None)
        assert path[b].tolist() == want + [-1] * (n - len(want)), b
        assert counts[b] == len(want) and follow[b] == after, b
    assert counts[0] == 0 and counts[1] == n


def copy_token(c, pool, b, source, target):
    """Moves a token's record in a numpy pool."""
    for at, size in ref.sections(c.dim, c.group):
        where = [(c.table[b][s // c.page], s % c.page // 16, s % 16) for s in (source, target)]
        (p0, k0, r0), (p1, k1, r1) = where
        pool[p1, :, k1, at + r1 * size:at + (r1 + 1) * size] = c.pool[p0, :, k0, at + r0 * size:at + (r0 + 1) * size]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", [(128, 64), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("n,page", [(1, 16), (7, 16), (33, 48), (64, 16), (64, 64)])
def test_keep(dim, group, n, page):
    lengths = [n, n + 1, 0, n + 15, n + 77, n + 128, n + 200]
    c = ref.Batch(lengths, 3, dim, group, page, seed=n + dim)
    rng = np.random.default_rng(n)
    path = np.full((len(lengths), n), -1, np.int32)
    counts = [n, 0, min(2, n), min(3, n), (n + 1) // 2, min(1, n), n // 3]
    for b, k in enumerate(counts):
        path[b, :k] = np.sort(rng.choice(n, k, replace=False))
        if k + 1 < n:
            path[b, k + 1:] = rng.integers(-5, n + 5, n - k - 1)  # behind the first -1 nothing counts
    slots = c.table.shape[1] * page + 5
    weights = rng.random((len(lengths), 3, slots)).astype(np.float32)
    where = rng.integers(0, 1 << 20, (len(lengths), 3, slots)).astype(np.int32)
    want_pool, want_w, want_p = c.pool.copy(), weights.copy(), where.copy()
    for b, k in enumerate(counts):
        ctx = lengths[b] - n
        for i in range(k if lengths[b] else 0):
            copy_token(c, want_pool, b, ctx + path[b, i], ctx + i)
            want_w[b, :, ctx + i] = weights[b, :, ctx + path[b, i]]
            want_p[b, :, ctx + i] = where[b, :, ctx + path[b, i]]
    pool, table, held = c.on()
    w, p = torch.from_numpy(weights).cuda(), torch.from_numpy(where).cuda()
    new = fa.kv4_keep(pool, table, held, torch.from_numpy(path).cuda(), weights=w, slot_positions=p)
    assert fa.fa_get_device_status() == 0
    assert new.tolist() == [length - n + k if length else 0 for length, k in zip(lengths, counts)]
    assert held.tolist() == lengths
    assert np.array_equal(pool.cpu().numpy(), want_pool)
    assert np.array_equal(w.cpu().numpy(), want_w) and np.array_equal(p.cpu().numpy(), want_p)
    pool, table, held = c.on()
    fa.kv4_keep(pool, table, held, torch.from_numpy(path).cuda())
    assert np.array_equal(pool.cpu().numpy(), want_pool)


@pytest.mark.gpu
def test_bad_paths_lengths_and_pages_leave_the_sequence():
    c = ref.Batch([40, 50, 60], 2, 128, 64, 16, seed=3)
    good = [2, 5, -1, -1, -1, -1]
    for bad in ([5, 2, -1, 0, 0, 0], [0, 0, -1, 0, 0, 0], [6, -1, 0, 0, 0, 0], [-2, -1, 0, 0, 0, 0], [0, 1, 2, 3, 5, 5],
                [0, 1, 2, 3, 4, 6]):
        pool, table, held = c.on()
        new = fa.kv4_keep(pool, table, held, torch.tensor([good, bad, good], dtype=torch.int32, device="cuda"))
        assert fa.fa_get_device_status() == -11
        assert new.tolist() == [36, 50, 56]
        want = c.pool.copy()
        for b, n in ((0, 40), (2, 60)):
            for i, j in enumerate(good[:2]):
                copy_token(c, want, b, n - 6 + j, n - 6 + i)
        assert np.array_equal(pool.cpu().numpy(), want)
    for value in (5, -3, 10 ** 6):
        pool, table, held = c.on()
        held[1] = value
        new = fa.kv4_keep(pool, table, held, torch.tensor([good] * 3, dtype=torch.int32, device="cuda"))
        assert fa.fa_get_device_status() == -11 and new.tolist() == [36, value, 56]
        assert np.array_equal(pool.cpu().numpy(), want)
    pool, table, held = c.on()
    slots = torch.zeros(3, 2, 55, device="cuda")  # too few for the third
    new = fa.kv4_keep(pool, table, held, torch.tensor([good] * 3, dtype=torch.int32, device="cuda"), weights=slots)
    assert fa.fa_get_device_status() == -11 and new.tolist() == [36, 46, 60]
    pool, table, held = c.on()
    table[1, 3] = -1  # slots 48 and 49: place 4 and 5
    new = fa.kv4_keep(pool, table, held, torch.tensor([good] * 3, dtype=torch.int32, device="cuda"))
    assert fa.fa_get_device_status() == -13 and new.tolist() == [36, 46, 56]
    copy_token(c, want, 1, 44 + 2, 44)
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.gpu
def test_a_step_with_drafts():
    """Append a batch's trees, attend over the cache and over another sequence's states, accept, keep, and
    go on: captured once and replayed, against a cache that never held what was dropped."""
    B, heads, hq, n, dim, page = 3, 2, 8, 12, 64, 16
    rng = np.random.default_rng(5)
    past = [70, 20, 33]
    g = torch.Generator("cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    width = 12
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    pools = [fa.kv4_pool(B * width, heads, dim, page, 32) for _ in range(2)]
    lengths = torch.tensor(past, dtype=torch.int32, device="cuda")
    ends = lambda counts: torch.tensor(np.r_[0, np.cumsum(counts)], dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = normal(sum(past), heads, dim), normal(sum(past), heads, dim)
    for pool in pools:
        fa.kv4_append(pool, k, v, table, lengths, ends(past))
    states = normal(B, 2 * heads, 90, dim)  # keys and values of an encoder's states
    encoded = torch.tensor([90, 0, 41], dtype=torch.int32, device="cuda")

    held = lengths.clone()  # kept lengths; the graph's own buffers from here on
    parents = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    tokens, picks = (torch.zeros(B, n, dtype=torch.int64, device="cuda") for _ in range(2))
    first = torch.zeros(B, dtype=torch.int64, device="cuda")
    q, kn, vn = normal(B, hq, n, dim), normal(B * n, heads, dim), normal(B * n, heads, dim)
    cu = ends([n] * B)

    def step():
        grown = held + n
        fa.kv4_append(pools[0], kn, vn, table, grown, cu)
        o, lse = fa.attention_tree_kv4(q, pools[0], table, grown, parents)
        x, xl = fa.attention_forward_cross(o, states[:, :heads], states[:, heads:], encoded)
        path, counts, follow = fa.tree_accept(parents, tokens, picks, first)
        new = fa.kv4_keep(pools[0], table, grown, path)
        held.copy_(new)
        return grown, o, lse, x, xl, path, counts, follow

    start = held.clone()
    step()  # once before it is captured
    held.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    held.copy_(start)
    fa.kv4_append(pools[0], k, v, table, lengths, ends(past))
    now = list(past)
    for turn in range(3):
        tree = trees(B, n, seed=turn)
        parents.copy_(torch.from_numpy(tree))
        t, p = rng.integers(0, 2, (2, B, n))
        f = rng.integers(0, 2, B)
        tokens.copy_(torch.from_numpy(t)), picks.copy_(torch.from_numpy(p)), first.copy_(torch.from_numpy(f))
        for x in (q, kn, vn):
            x.copy_(normal(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == 0
        grown, o, lse, x, xl, path, counts, follow = out
        # the tree's attention, over the cache as it was before anything was dropped
        full = fa.kv4_pool(B * width, heads, dim, page, 32)
        full.copy_(pools[1])
        fa.kv4_append(full, kn, vn, table, grown, cu)
        c = ref.Batch([a + n for a in now], heads, dim, 32, page, seed=0)
        c.pool, c.table = full.cpu().numpy(), table.cpu().numpy()
        check_tree(c, q.cpu(), tree, o, lse)
        want = reference(o, states[:, :heads], states[:, heads:], encoded.tolist())
        check_cross("o", x, want)
        check_cross("lse", xl, want)
        # the other cache gets what stands, and nothing else
        rows, kept = [], []
        for b in range(B):
            way, after = accepted(tree[b], t[b], p[b], f[b])
            assert path[b, :len(way)].tolist() == way and counts[b] == len(way) and follow[b] == after
            rows += [b * n + i for i in way]
            kept.append(len(way))
            now[b] += len(way)
        assert held.tolist() == now
        if rows:
            fa.kv4_append(pools[1], kn[rows], vn[rows], table, held, ends(kept))
        for a, b in zip(fa.kv4_read(pools[0], table, held), fa.kv4_read(pools[1], table, held)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals (no GPU)

BASE = 1 << 24


def accept(parents=BASE, tokens=2 * BASE, picks=3 * BASE, first=4 * BASE, wide=1, B=3, N=5, path=5 * BASE, counts=6 * BASE,
           follow=7 * BASE):
    return fa.load_library().fa_tree_accept(parents, tokens, picks, first, wide, B, N, path, counts, follow, None)


def keep(pool=1 << 20, width=4, path=5 * BASE, N=5, lengths_out=6 * BASE, weights=None, positions=None, slots=0, D=64):
    c = struct.pack("QQQ7i4x", pool, 2 * BASE, 3 * BASE, 2, 2, D, 64, 16, 8, width)
    return fa.load_library().fa_kv4_keep(c, path, N, lengths_out, weights, positions, slots, None)


def test_refusals_of_the_c_abi():
    if torch.cuda.is_available():
        pytest.skip("good arguments would launch on made-up addresses")
    ok = (-5, -9)
    assert accept() in ok and accept(first=None) in ok and accept(N=64) in ok
    for name in ("parents", "tokens", "picks", "path", "counts", "follow"):
        assert accept(**{name: None}) == -1
        assert accept(**{name: 9 * BASE + 2}) == -4
    assert accept(first=9 * BASE + 4) == -4 and accept(first=9 * BASE + 4, wide=0) in ok
    assert accept(B=0) == -2 and accept(N=0) == -2 and accept(N=-1) == -2 and accept(B=1 << 30, N=64) == -2
    assert accept(N=65) == -3 and accept(wide=2) == -8
    assert accept(path=BASE) == -8 and accept(counts=5 * BASE + 8) == -8 and accept(follow=4 * BASE) == -8
    assert keep() in ok
    assert keep(path=None) == -1 and keep(lengths_out=None) == -1 and keep(pool=0) == -1
    assert keep(N=0) == -2 and keep(N=65) == -3 and keep(D=32) == -3
    assert keep(weights=9 * BASE) == -2 and keep(weights=9 * BASE, slots=64) in ok
    assert keep(path=5 * BASE + 1) == -4 and keep(positions=9 * BASE + 2, slots=64) == -4
    assert keep(lengths_out=3 * BASE) == -8                       # the lengths themselves
    assert keep(path=1 << 20) == -8
    assert keep(weights=9 * BASE, positions=9 * BASE, slots=64) == -8
    assert keep(weights=6 * BASE, slots=64) == -8


@pytest.mark.gpu
def test_refusals_of_the_python_entry_points():
    parents = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    for bad in (dict(parents=parents.long()), dict(parents=parents[0]), dict(tokens=tokens.float()),
                dict(tokens=tokens[:1]), dict(picks=tokens.int()), dict(first=tokens[0]), dict(picks=tokens.cpu()),
                dict(tokens=tokens.t().contiguous().t())):
        with pytest.raises(ValueError):
            fa.tree_accept(**{**dict(parents=parents, tokens=tokens, picks=tokens), **bad})
    with pytest.raises(ValueError):
        fa.tree_accept(parents.cpu(), tokens.cpu(), tokens.cpu())
    c = ref.Batch([40, 41], 2, 64, 64, 16, seed=1)
    pool, table, lengths = c.on()
    for bad in (dict(path=parents.long()), dict(path=parents[:1]), dict(path=parents.cpu()),
                dict(weights=torch.zeros(2, 2, 64, device="cuda", dtype=torch.float64)),
                dict(weights=torch.zeros(2, 2, 64, device="cuda"),
                     slot_positions=torch.zeros(2, 2, 60, device="cuda", dtype=torch.int32))):
        with pytest.raises(ValueError):
            fa.kv4_keep(**{**dict(pool=pool, block_table=table, lengths=lengths, path=parents), **bad})
    with pytest.raises(fa.FAError):
        fa.kv4_keep(pool, table, lengths, torch.full((2, 65), -1, dtype=torch.int32, device="cuda"))
