"""Attention of a tree of drafted tokens over the 4-bit cache, against attention in 64 bits
over what the cache stands for, every element."""
import ctypes
import struct

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


def ways(parents):
    """For each place, the set of places that it sees, or None where it holds no token."""
    found = []
    for i, p in enumerate(parents):
        if p == -1:
            found.append({i})
        else:
            found.append(found[p] | {i} if 0 <= p < i and found[p] is not None else None)
    return found


def trees(B, N, seed, empty=0.1):
    """Random trees, some places without a token."""
    rng = np.random.default_rng(seed)
    out = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            out[b, i] = rng.integers(max(-1, i - 9), i)
            if rng.random() < empty:
                out[b, i] = rng.choice([-2, i, i + 1, 1000, -1000])
    return out


def attend(q, loaded, scale, parents):
    """o, lse, and what the tolerances go by, as kv4_ref.attend has them, for a tree."""
    ks, km, vs, vm = loaded
    heads, length, dim = ks.shape
    hq, n, _ = q.shape
    see = np.zeros((n, length), bool)
    for i, way in enumerate(ways(parents)):
        if way is not None and length:
            see[i, :length - n] = True
            see[i, [length - n + j for j in way]] = True
    q = q.reshape(heads, -1, n, dim)
    hidden = ~see
    with np.errstate(all="ignore"):
        s = np.where(hidden, -np.inf, np.einsum("hgid,htd->hgit", q, ks + km) * scale)
        size = np.where(hidden, 0.0, np.einsum("hgid,htd->hgit", np.abs(q), np.abs(ks) + np.abs(km)) * abs(scale))
        top = s.max(-1, keepdims=True) if length else np.full(s.shape[:-1] + (1,), -np.inf)
        e = np.where(hidden, 0.0, np.exp(s - np.where(np.isneginf(top), 0.0, top)))
        total = e.sum(-1, keepdims=True)
        p = np.where(total == 0, 0.0, e / total)
        lse = np.where(total == 0, -np.inf, top + np.log(total))[..., 0]
        v = vs + vm
        o = np.stack([np.einsum("hgt,htd->hgd", p[:, :, i][..., see[i]], v[:, see[i]]) for i in range(n)], 2)
        weighed = np.stack([np.einsum("hgt,htd->hgd", p[:, :, i][..., see[i]], (np.abs(vs) + np.abs(vm))[:, see[i]])
                            for i in range(n)], 2)
    most = size.max(-1) if length else np.zeros(s.shape[:-1])
    flat = lambda x: x.reshape(hq, n, *x.shape[3:])  # noqa: E731
    return flat(o), flat(lse), flat(most), flat(weighed)


# Tolerances, from the kernel's arithmetic: a score is a sum of exact products in fp32, 17 chained matrix
# instructions, then scaled and offset: at most 32 roundings of 2^-23 of the sum of the absolute
# terms, so 2^-18 of it.  A weight carries that twice and 2^-20 for the exponential and the sums.  It and the
# value are rounded to bf16 (2^-8 each) for their product, and the output once more.
def score_tol(most):
    return most * 2.0 ** -18


def o_tol(o, most, weighed):
    return np.abs(o) * 2.0 ** -8 + weighed * (2.0 ** -7 + 2.0 ** -15 + 2.0 ** -20 + 2 * score_tol(most)[..., None]) + 2.0 ** -110


def lse_tol(lse, most):
    return score_tol(most) + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))


def check(c, q, parents, o, lse, scale=None):
    scale = c.dim ** -0.5 if scale is None else scale
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    for b in range(len(c.lengths)):
        wo, wl, most, weighed = attend(q[b].double().numpy(), c.loaded(b), scale, parents[b])
        assert np.array_equal(np.isneginf(lse[b]), np.isneginf(wl)), b
        assert np.array_equal(np.isnan(lse[b]), np.isnan(wl)), b
        fin = np.isfinite(wl)
        assert (np.abs(lse[b] - wl)[fin] <= lse_tol(wl, most)[fin]).all(), (b, np.abs(lse[b] - wl)[fin].max())
        assert np.array_equal(np.isnan(o[b]), np.isnan(wo)), b
        good = ~np.isnan(wo)
        off = (np.abs(o[b] - wo) - o_tol(wo, most, weighed))[good]
        assert off.size == 0 or off.max() <= 0, (b, off.max())


def run(c, hq, parents, scale=None, std=1.0):
    q = c.queries(hq, parents.shape[1], std)
    o, lse = fa.attention_tree_kv4(q.cuda(), *c.on(), torch.from_numpy(parents).cuda(), scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    check(c, q, parents, o, lse, scale)
    return q, o, lse


FORMATS = [(128, 64), (128, 32), (64, 64), (64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("each,n", [(1, 1), (4, 1), (3, 7), (1, 64), (2, 64), (4, 32), (5, 31), (8, 17), (5, 61), (33, 16)])
def test_lengths_from_the_tree_alone_to_many_pages(dim, group, each, n):
    c = ref.Batch([n, 0, n + 1, n + 15, n + 63, n + 64, n + 130, n + 300], 2, dim, group, 16, seed=dim + each * n)
    run(c, 2 * each, trees(8, n, seed=each + n))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_long_and_uneven_batches(dim, group, page):
    c = ref.Batch([4109, 13, 700, 0, 1999, 257], 3, dim, group, page, seed=page, spare=2)
    run(c, 12, trees(6, 13, seed=page))


@pytest.mark.gpu
@pytest.mark.parametrize("heads,each", [(1, 1), (1, 8), (40, 2)])
def test_one_long_sequence(heads, each):
    c = ref.Batch([9000], heads, 64, 64, 64, seed=heads)
    run(c, heads * each, trees(1, 24, seed=each))


@pytest.mark.gpu
@pytest.mark.parametrize("each", [1, 8])
def test_shapes_of_trees(each):
    n = 20
    parents = np.stack([
        np.arange(-1, n - 1),                                   # a chain
        np.full(n, -1),                                         # roots alone
        np.zeros(n) - (np.arange(n) == 0),                      # one root's children
        np.full(n, -2),                                         # no token at all
        np.r_[-2, np.arange(n - 1)],                            # all hang on an empty place
        np.r_[-1, 0, 5, 2, 3, 4, -1, 6, 7, np.full(n - 9, 7)],  # a parent behind its place, and what hangs on it
        np.r_[-1, np.full(n - 1, -2147483648)],
    ]).astype(np.int32)
    c = ref.Batch([100, 20, 333, 90, 64, 84, 85], 2, 128, 64, 16, seed=7)
    _, o, lse = run(c, 2 * each, parents)
    assert not o[3].any() and not o[4].any() and torch.isneginf(lse[3]).all()


@pytest.mark.gpu
def test_a_chain_is_causal_decoding():
    c = ref.Batch([500, 8, 77], 2, 128, 32, 16, seed=8)
    parents = np.tile(np.arange(-1, 7, dtype=np.int32), (3, 1))
    q, o, lse = run(c, 8, parents)
    o2, lse2 = fa.attention_decode_kv4(q.cuda(), *c.on(), causal=True)
    assert (lse - lse2).abs().max() <= 2.0 ** -16
    for b in range(3):
        wo, _, most, weighed = attend(q[b].double().numpy(), c.loaded(b), 128 ** -0.5, parents[b])
        assert (np.abs((o2[b].cpu().double().numpy() - wo)) <= o_tol(wo, most, weighed)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
def test_unusual_scales(scale):
    c = ref.Batch([333, 40], 2, 64, 32, 16, seed=5)
    run(c, 8, trees(2, 9, seed=5), scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("gain,std", [(8.0, 1.0), (1.0, 40.0), (2.0 ** -30, 1.0), (1.0, 2.0 ** -40), (2.0 ** 20, 2.0 ** -20),
                                      (2.0 ** 100, 2.0 ** -101), (2.0 ** -70, 2.0 ** 75), (2.0 ** 60, 2.0 ** -110)])
def test_magnitudes(gain, std):
    c = ref.Batch([700, 77], 2, 128, 64, 32, seed=6, gain=gain)
    run(c, 8, trees(2, 21, seed=6), std=std)


@pytest.mark.gpu
def test_values_up_to_the_largest():
    """Groups from 0 to bf16's largest, and to its lowest: 15 s + m is finite, sums of many too."""
    c = ref.Batch([900], 1, 64, 64, 64, seed=9)
    (at, size) = ref.sections(64, 64)[3]
    pairs = torch.from_numpy(c.pool[..., at:at + 16 * size].copy()).view(torch.bfloat16).view(-1, 2)
    live = ~pairs[:, 0].isnan()
    pairs[live] = torch.tensor([2.0 ** 124 * 1.0, -2.0 ** 127 * 1.9921875]).to(torch.bfloat16)
    c.pool[..., at:at + 16 * size] = pairs.view(torch.uint8).numpy().reshape(c.pool[..., at:at + 16 * size].shape)
    _, o, _ = run(c, 4, trees(1, 16, seed=9, empty=0))
    assert torch.isfinite(o).all() and o.abs().max() > 1e37


@pytest.mark.gpu
@pytest.mark.parametrize("gain,std,scale", [(1.0, 2.0 ** 110, 2.0 ** -113), (2.0 ** -95, 2.0 ** 110, 2.0 ** -18),
                                            (1.0, 2.0 ** 124, 2.0 ** -125), (2.0 ** 30, 2.0 ** 90, 2.0 ** -120)])
def test_queries_up_to_the_largest(gain, std, scale):
    c = ref.Batch([700, 77], 2, 128, 64, 32, seed=16, gain=gain)
    _, o, lse = run(c, 8, trees(2, 21, seed=16, empty=0), scale=scale, std=std)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
def test_keys_of_the_largest_in_every_channel():
    """Scores of 2^7: each of 128 channels near bf16's largest in the cache, the query small."""
    c = ref.Batch([300], 1, 128, 64, 16, seed=17)
    at, size = ref.sections(128, 64)[1]
    pairs = torch.from_numpy(c.pool[..., at:at + 16 * size].copy()).view(torch.bfloat16).view(-1, 2)
    pairs[~pairs[:, 0].isnan()] = torch.tensor([0.0, 2.0 ** 127 * 1.9921875]).to(torch.bfloat16)
    c.pool[..., at:at + 16 * size] = pairs.view(torch.uint8).numpy().reshape(c.pool[..., at:at + 16 * size].shape)
    q = torch.full((1, 2, 9, 128), 2.0 ** -121 * 1.9921875, dtype=torch.bfloat16)
    parents = trees(1, 9, seed=17, empty=0)
    o, lse = fa.attention_tree_kv4(q.cuda(), *c.on(), torch.from_numpy(parents).cuda(), scale=2.0 ** -8)
    assert fa.fa_get_device_status() == 0 and torch.isfinite(o).all()
    check(c, q, parents, o, lse, 2.0 ** -8)


def rescale(c, b, slot, section, group, value):
    """Sets the scales (s, m) of one group of one token, all heads."""
    at, size = ref.sections(c.dim, c.group)[section]
    page, block, r = c.table[b][slot // c.page], slot % c.page // 16, slot % 16
    pair = torch.tensor([value, value]).to(torch.bfloat16).view(torch.uint8).numpy()
    c.pool[page, :, block, at + r * size + 4 * group:at + r * size + 4 * group + 4] = pair


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("slots", [[0], [130], [127, 128], [5, 300, 301, 640], [899], list(range(0, 900, 128)),
                                   list(range(128, 900, 256))])
@pytest.mark.parametrize("value", [2.0 ** -18, 2.0 ** -60, 2.0 ** 12, 2.0 ** -17, 2.0 ** 11, -2.0 ** -20])
def test_keys_of_other_scales_among_ordinary_ones(dim, group, slots, value):
    """Tiles whose keys go as fp16 beside those that cannot, in every order; and the ends of fp16's range."""
    c = ref.Batch([900], 1, dim, group, 16, seed=18)
    for i, slot in enumerate(slots):
        rescale(c, 0, slot, 1, i % (dim // group), value)
    run(c, 4, trees(1, 11, seed=18, empty=0), std=2.0 ** -12 if value > 1 else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", [(128, 64), (128, 32), (64, 32)])
@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -18, 2.0 ** -24])
def test_small_queries_beside_large_ones(dim, group, small):
    """The large channels of a row meet keys of 0, so that only the small ones make its scores.  fp16 holds a
    row to half of 2^-24 where its largest is at least 2^8: 2^-33 of it for a channel, times s (n - 8),
    no more than the group's largest s n (a group's codes reach 15)."""
    c = ref.Batch([60], 1, dim, group, 16, seed=19)
    for slot in range(60):
        rescale(c, 0, slot, 1, 0, 0.0)
    q = c.queries(2, 9, 1.0)
    q[..., group:] *= small
    parents = trees(1, 9, seed=19, empty=0)
    scale = 1 / small
    o, lse = fa.attention_tree_kv4(q.cuda(), *c.on(), torch.from_numpy(parents).cuda(), scale=scale)
    assert fa.fa_get_device_status() == 0
    x = q[0].double().numpy()
    wo, wl, most, weighed = attend(x, c.loaded(0), scale, parents[0])
    most_key = np.abs(c.loaded(0)[0]).max()
    extra = scale * np.abs(x).max(-1) * 2.0 ** -33 * dim * most_key
    assert (np.abs(lse[0].cpu().double().numpy() - wl) <= lse_tol(wl, most) + extra).all()
    assert (np.abs(o[0].cpu().double().numpy() - wo) <= o_tol(wo, most, weighed) + 2 * (extra[..., None] * weighed)).all()


@pytest.mark.gpu
def test_pools_beyond_32_bits():
    """The same pages behind 2^32 bytes of a pool: attention and keeping."""
    c = ref.Batch([900, 70], 2, 128, 64, 16, seed=21)
    parents = torch.from_numpy(trees(2, 12, seed=21, empty=0)).cuda()
    q = c.queries(8, 12).cuda()
    pool, table, lengths = c.on()
    path = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
    path[:, :3] = torch.tensor([1, 4, 11], dtype=torch.int32)
    count, page_bytes = pool.shape[0], pool[0].numel()
    before = (1 << 32) // page_bytes + 1
    far = torch.empty(before + count, *pool.shape[1:], dtype=torch.uint8, device="cuda")
    far[before:] = pool
    far_table = torch.where(table >= 0, table + before, table)
    o, lse = fa.attention_tree_kv4(q, pool, table, lengths, parents)
    o2, lse2 = fa.attention_tree_kv4(q, far, far_table, lengths, parents)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a, b = fa.kv4_keep(pool, table, lengths, path), fa.kv4_keep(far, far_table, lengths, path)
    assert fa.fa_get_device_status() == 0
    assert torch.equal(a, b) and torch.equal(far[before:], pool)


@pytest.mark.gpu
def test_a_workspace_of_exactly_the_size_asked_for():
    c = ref.Batch([5000, 0, 700], 2, 128, 64, 16, seed=20)
    parents = torch.from_numpy(trees(3, 40, seed=20)).cuda()
    q = c.queries(8, 40).cuda()
    pool, table, lengths = c.on()
    want, want_lse = fa.attention_tree_kv4(q, pool, table, lengths, parents)
    need = fa.load_library().fa_kv4_tree_workspace(3, 8, 2, 40, 128, table.shape[1] * 16)
    assert need > 0
    around = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty_like(want_lse)
    held = struct.pack("QQQ7i4x", pool.data_ptr(), table.data_ptr(), lengths.data_ptr(), 3, 2, 128, 64, 16, pool.shape[0],
                       table.shape[1])
    stream = torch.cuda.current_stream().cuda_stream
    for size, rc in ((need, 0), (need - 1, None)):
        got = fa.load_library().fa_kv4_tree(held, q.data_ptr(), parents.data_ptr(), o.data_ptr(), lse.data_ptr(), 8, 40,
                                            ctypes.c_float(128 ** -0.5), around.data_ptr() + 256, size, stream)
        assert got == rc if rc is not None else got < 0
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert (around[:256] == 77).all() and (around[256 + need:] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("each,n", [(2, 20), (8, 40)])
def test_nan_tokens_reach_those_that_see_them_alone(dim, group, each, n):
    c = ref.Batch([n + 100, n + 3, 64 + n], 2, dim, group, 16, seed=10)
    parents = trees(3, n, seed=11, empty=0.05)
    rescale(c, 0, 100 + 3, 3, dim // group - 1, float("nan"))   # the last value group of a place
    rescale(c, 0, 100 + 7, 1, 0, float("nan"))                  # a key group of another
    rescale(c, 1, 3 + n - 1, 3, 0, float("nan"))                # a value group of a place that only it sees
    rescale(c, 2, 5, 3, 0, float("nan"))                        # a value group in the context
    q, o, lse = run(c, 2 * each, parents)
    assert o[0].isnan().any() and not o[0].isnan().all() and o[2].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_row(bad):
    c = ref.Batch([300], 2, 64, 32, 16, seed=12)
    parents = trees(1, 12, seed=12, empty=0)
    q = c.queries(4, 12)
    o, lse = fa.attention_tree_kv4(q.cuda(), *c.on(), torch.from_numpy(parents).cuda())
    q[0, 1, 5, 3] = bad
    o2, lse2 = fa.attention_tree_kv4(q.cuda(), *c.on(), torch.from_numpy(parents).cuda())
    assert o2[0, 1, 5].isnan().all() and lse2[0, 1, 5].isnan()
    o2[0, 1, 5], lse2[0, 1, 5] = o[0, 1, 5], lse[0, 1, 5]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_recorded():
    c = ref.Batch([200, 90, 150], 2, 128, 64, 16, seed=13)
    parents = torch.from_numpy(trees(3, 10, seed=13, empty=0)).cuda()
    q = c.queries(4, 10).cuda()
    pool, table, lengths = c.on()
    good, _ = fa.attention_tree_kv4(q, pool, table, lengths, parents)
    assert fa.fa_get_device_status() == 0
    for value in (9, -1, 10 ** 6):
        held = lengths.clone()
        held[1] = value
        o, lse = fa.attention_tree_kv4(q, pool, table, held, parents)
        assert fa.fa_get_device_status() == -11
        assert not o[1].any() and torch.isneginf(lse[1]).all()
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    for value in (-1, 10 ** 6):
        t = table.clone()
        t[1, 2] = value
        o, lse = fa.attention_tree_kv4(q, pool, t, lengths, parents)
        assert fa.fa_get_device_status() == -13
        assert torch.isfinite(o).all()
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    # entries behind the length are not read
    t = torch.full((3, table.shape[1] + 3), 10 ** 6, dtype=torch.int32, device="cuda")
    for b, n in enumerate(c.lengths):
        t[b, :-(-n // 16)] = table[b, :-(-n // 16)]
    o, _ = fa.attention_tree_kv4(q, pool, t, lengths, parents)
    assert fa.fa_get_device_status() == 0 and torch.equal(o, good)


@pytest.mark.gpu
def test_outputs_streams_and_graphs():
    c = ref.Batch([400, 64, 130], 2, 128, 64, 16, seed=14)
    parents = torch.from_numpy(trees(3, 30, seed=14)).cuda()
    q = c.queries(8, 30).cuda()
    pool, table, lengths = c.on()
    o, lse = fa.attention_tree_kv4(q, pool, table, lengths, parents)
    around = torch.full((q.numel() + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = around[32:-32].view(q.shape)
    got, _ = fa.attention_tree_kv4(q, pool, table, lengths, parents, out=out, lse=torch.empty_like(lse))
    assert got is out and torch.equal(out, o) and (around[:32] == 5).all() and (around[-32:] == 5).all()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [fa.attention_tree_kv4(q, pool, table, lengths, parents, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in many)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = fa.attention_tree_kv4(q, pool, table, lengths, parents)
    for held in ([400, 64, 130], [0, 31, 100]):
        lengths.copy_(torch.tensor(held, dtype=torch.int32))
        graph.replay()
        o, lse = fa.attention_tree_kv4(q, pool, table, lengths, parents)
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


# ------------------------------------------------------------------ refusals (no GPU)

def cache(pool=1 << 20, table=1 << 24, lengths=1 << 25, B=2, heads=2, D=64, group=64, page=16, pages=8, width=4):
    return struct.pack("QQQ7i4x", pool, table, lengths, B, heads, D, group, page, pages, width)


def call(c=None, q=1 << 26, parents=1 << 27, o=1 << 28, lse=1 << 29, Hq=4, N=5, scale=0.1,
         workspace=None, size=0):
    return fa.load_library().fa_kv4_tree(c or cache(), q, parents, o, lse, Hq, N, ctypes.c_float(scale), workspace, size,
                                         None)


def test_refusals_of_the_c_abi():
    if torch.cuda.is_available():
        pytest.skip("good arguments would launch on made-up addresses")
    assert call() in (-5, -9)
    assert call(N=64) in (-5, -9)
    for name in ("q", "parents", "o", "lse"):
        assert call(**{name: None}) == -1
        assert call(**{name: (1 << 30) + 2}) == -4
    assert call(c=cache(pool=0)) == -1
    assert call(N=0) == -2 and call(N=-3) == -2 and call(Hq=3) == -2 and call(Hq=0) == -2
    assert call(Hq=1 << 30) == -2
    assert call(N=65) == -3
    assert call(c=cache(D=96)) == -3 and call(c=cache(group=16)) == -3
    assert call(scale=float("nan")) == -8
    assert call(o=1 << 26) == -8 and call(lse=1 << 28) == -8 and call(o=1 << 20) == -8 and call(lse=1 << 27) == -8
    assert call(o=1 << 25) == -8
    query = fa.load_library().fa_kv4_tree_workspace
    assert query(0, 4, 2, 5, 64, 64) == -2 and query(2, 3, 2, 5, 64, 64) == -2 and query(2, 4, 2, 0, 64, 64) == -2
    assert query(2, 4, 2, 5, 64, 60) == -2 and query(2, 4, 2, 65, 64, 64) == -3 and query(2, 4, 2, 5, 96, 64) == -3


@pytest.mark.gpu
def test_refusals_of_the_python_entry_point():
    c = ref.Batch([40, 41], 2, 64, 64, 16, seed=1)
    pool, table, lengths = c.on()
    parents = torch.from_numpy(trees(2, 6, seed=1)).cuda()
    q = c.queries(4, 6).cuda()
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, :, :5]), dict(q=q.cpu()), dict(parents=parents.long()),
                dict(parents=parents[:, :5]), dict(parents=parents.cpu()), dict(parents=parents[:1].expand(2, -1)),
                dict(lengths=lengths[:1]), dict(out=torch.empty_like(q)[:1]),
                dict(lse=torch.empty(2, 4, 7, device="cuda"))):
        given = {**dict(q=q, pool=pool, block_table=table, lengths=lengths, parents=parents), **bad}
        with pytest.raises(ValueError):
            fa.attention_tree_kv4(**given)
    with pytest.raises(fa.FAError):
        fa.attention_tree_kv4(torch.zeros(2, 4, 65, 64, dtype=torch.bfloat16, device="cuda"), pool, table, lengths,
                              torch.zeros(2, 65, dtype=torch.int32, device="cuda"))
    with pytest.raises(fa.FAError):
        fa.attention_tree_kv4(torch.zeros(2, 3, 6, 64, dtype=torch.bfloat16, device="cuda"), pool, table, lengths, parents)
    with pytest.raises(fa.FAError):
        fa.attention_tree_kv4(q, pool, table, lengths, parents, out=q)
