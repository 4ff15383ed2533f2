"""Decoding over the 4-bit cache against attention in 64 bits over what the cache stands
for, every element (tolerances from the kernel's arithmetic: tests/kv4_ref.py)."""
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


def check(c, q, o, lse, scale, causal, weights=None, before=None):
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    w = None if weights is None else weights.cpu().double().numpy()
    for b, n in enumerate(c.lengths):
        wo, wl, p, most, weighed = ref.attend(q[b].double().numpy(), c.loaded(b), scale, causal)
        assert np.array_equal(np.isneginf(lse[b]), np.isneginf(wl))
        fin = np.isfinite(wl)
        assert (np.abs(np.where(fin, lse[b], 0) - np.where(fin, wl, 0)) <= ref.lse_tol(wl, most)).all(), b
        tol = ref.o_tol(wo, most, weighed)
        assert (np.abs(o[b] - wo) <= tol).all(), (b, float((np.abs(o[b] - wo) - tol).max()))
        if w is not None:
            base = np.zeros(w.shape[1:]) if before is None else before[b].astype(np.float64)
            want = base[:, :n] + p
            # each row's weight: its score's error (score and log-sum), 2^-20 for the exponential;
            # the sums round 2^-23 of the account per row
            rows = q.shape[1] // c.heads * q.shape[2]
            rel = 2 * ref.score_tol(most).max() + 2.0 ** -20
            assert (np.abs(w[b, :, :n] - want) <= p * rel + want * rows * 2.0 ** -23).all(), b
            assert np.array_equal(w[b, :, n:], base[:, n:])


def run(c, hq, tq, causal=True, scale=None, weights=False, std=1.0, seed=0):
    q = c.queries(hq, tq, std)
    pool, table, held = c.on()
    kw, before = {}, None
    if weights:
        slots = c.table.shape[1] * c.page
        before = c.rng.uniform(0, 3, (len(c.lengths), c.heads, slots)).astype(np.float32)
        kw = dict(weights=torch.from_numpy(before).cuda())
    got = fa.attention_decode_kv4(q.cuda(), pool, table, held, causal=causal, scale=scale, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    check(c, q, got[0], got[1], c.dim ** -0.5 if scale is None else scale, causal, got[2] if weights else None, before)
    return got


FORMATS = [(128, 64), (128, 32), (64, 64), (64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("each,tq", [(1, 1), (4, 1), (8, 1), (3, 2), (7, 1), (4, 4), (2, 8), (5, 5), (8, 8)])
def test_lengths_from_none_to_many_pages(dim, group, each, tq):
    # ends inside a 16-token block, inside a page, on both borders; an empty sequence; sequences
    # shorter than the queries, whose first rows see nothing
    c = ref.Batch([1, 0, 15, 16, 17, 2, 31, 33, 64, 95, 300], 2, dim, group, 16, seed=dim + each * tq)
    run(c, 2 * each, tq)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_long_and_uneven_batches(dim, group, page):
    c = ref.Batch([4109, 3, 700, 0, 1999, 257], 3, dim, group, page, seed=page, spare=2)
    run(c, 12, 1, weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("each,tq", [(1, 3), (4, 2), (6, 8), (16, 1), (40, 1), (128, 8)])
def test_weights_and_masks(each, tq, causal):
    c = ref.Batch([5, 1, 613, 0, 128], 2, 128, 64, 64, seed=each + tq)
    run(c, 2 * each, tq, causal=causal, weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
def test_unusual_scales(scale):
    c = ref.Batch([333, 40], 2, 64, 32, 16, seed=5)
    run(c, 8, 2, scale=scale, weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("gain,std", [(8.0, 1.0), (1.0, 40.0), (2.0 ** -30, 1.0), (1.0, 2.0 ** -40), (2.0 ** 20, 2.0 ** -20)])
def test_magnitudes(gain, std):
    # peaked rows, values far below and above what 16 bits of exponent hold
    c = ref.Batch([1000, 77], 2, 128, 64, 32, seed=6, gain=gain)
    run(c, 8, 1, std=std)


@pytest.mark.gpu
def test_scales_that_differ_from_token_to_token():
    # value scales over 12 powers of two within one sequence, large ones at tokens of small weight
    c = ref.Batch([500], 1, 128, 32, 64, seed=7)
    (at, size) = ref.sections(128, 32)[3]
    pairs = torch.from_numpy(c.pool[..., at:at + 16 * size].copy()).view(torch.bfloat16)
    shape = pairs.shape
    factor = torch.from_numpy(2.0 ** c.rng.integers(-6, 7, shape[:-1] + (shape[-1] // 2,))).float()
    pairs = (pairs.float().view(*shape[:-1], -1, 2) * factor[..., None]).to(torch.bfloat16).view(shape)
    c.pool[..., at:at + 16 * size] = pairs.view(torch.uint8).numpy()
    run(c, 4, 1)


@pytest.mark.gpu
def test_many_sequences_of_every_length():
    # more (sequence, head) pairs than CTAs, and every short length
    c = ref.Batch(list(range(0, 130)), 4, 64, 64, 16, seed=8)
    run(c, 16, 1, weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("each,tq,weights", [(3, 1, False), (4, 5, False), (4, 5, True)])
def test_many_more_heads_than_ctas_on_short_caches(dim, group, each, tq, weights):
    # several heads in one CTA, each with two warps' pieces or one; runs of empty sequences, at the end too
    c = ref.Batch([(i * 37) % 101 if i % 7 else 0 for i in range(90)] + [1, 0, 0], 8, dim, group, 16, seed=dim + tq)
    run(c, 8 * each, tq, weights=weights)


@pytest.mark.gpu
@pytest.mark.parametrize("each,tq", [(4, 1), (5, 3)])
@pytest.mark.parametrize("count", [33, 100, 300])
def test_many_sequences_beside_a_long_one(count, each, tq):
    # the line of units over more sequences than a warp has lanes: several whole heads in one
    # warp's stretch, heads cut between warps and between CTAs
    c = ref.Batch([(i * 37) % 97 for i in range(count - 2)] + [3001, 700], 2, 128, 64, 32, seed=count)
    run(c, 2 * each, tq, weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 4096])
def test_one_token_steps_and_page_borders(page):
    # lengths around the borders of units, pages and warps' stretches, one step at a time
    for n in (1, 16, 31, 32, 33, 511, 512, 513, 1023, 1024, 1025, 4096):
        run(ref.Batch([n], 1, 64, 32, page, seed=n), 3, 1)


@pytest.mark.gpu
def test_sequences_that_share_pages():
    # a common prefix held once: both tables name the same pages
    c = ref.Batch([200, 136], 2, 128, 64, 32, seed=17)
    c.table[1, :4] = c.table[0, :4]
    run(c, 8, 1, weights=True)


@pytest.mark.gpu
def test_one_long_sequence():
    c = ref.Batch([70001], 1, 128, 64, 64, seed=9)
    run(c, 8, 1, weights=True)


@pytest.mark.gpu
def test_nan_in_a_masked_or_unused_place_stays_there():
    # the pool of Batch has NaN scales wherever no token lies; a NaN token is seen by the rows
    # after it only, and only by its own head
    c = ref.Batch([40], 2, 64, 64, 16, seed=10)
    at, size = ref.sections(64, 64)[1]
    page, block, r = c.table[0][39 // 16], 0, 39 % 16
    c.pool[page, 0, block, at + r * size:at + (r + 1) * size] = 255
    q = c.queries(4, 3).cuda()
    pool, table, held = c.on()
    o, lse = fa.attention_decode_kv4(q, pool, table, held)
    assert fa.fa_get_device_status() == 0
    nan = torch.isnan(o).all(-1)[0].cpu()
    assert nan.tolist() == [[False, False, True]] * 2 + [[False] * 3] * 2
    assert torch.equal(torch.isnan(lse)[0].cpu(), nan)
    assert torch.equal(torch.isnan(o).any(-1)[0].cpu(), nan)


@pytest.mark.gpu
@pytest.mark.parametrize("first,count", [(640, 64), (1000, 1), (0, 3000), (2999, 1)])
@pytest.mark.parametrize("part", [1, 3])
def test_a_nan_token_is_seen_however_little_it_weighs(first, count, part):
    # whole stretches of a warp that are NaN, and single tokens, against rows whose other
    # scores are far above: keys spoil every output, values those of their group
    c = ref.Batch([3000], 1, 64, 32, 64, seed=18)
    at, size = ref.sections(64, 32)[part]
    for t in range(first, first + count):
        page, block, r = c.table[0][t // 64], t % 64 // 16, t % 16
        c.pool[page, 0, block, at + r * size:at + r * size + 4] = 255     # the first group's pair
    q = (c.queries(4, 1).float() * 30).to(torch.bfloat16).cuda()
    pool, table, held = c.on()
    o, lse = fa.attention_decode_kv4(q, pool, table, held)
    assert fa.fa_get_device_status() == 0
    if part == 1:
        assert torch.isnan(o).all() and torch.isnan(lse).all()
    else:
        assert torch.isnan(o[..., :32]).all() and torch.isfinite(o[..., 32:]).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
def test_a_bad_query_spoils_its_own_row():
    c = ref.Batch([100, 100], 2, 128, 64, 16, seed=11)
    q = c.queries(8, 1)
    pool, table, held = c.on()
    good, _ = fa.attention_decode_kv4(q.cuda(), pool, table, held)
    q[0, 2, 0, 5], q[1, 7, 0, 0] = math.nan, math.inf
    o, lse = fa.attention_decode_kv4(q.cuda(), pool, table, held)
    bad = torch.zeros(2, 8, 1, dtype=torch.bool)
    bad[0, 2], bad[1, 7] = True, True
    assert torch.isnan(o.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    assert torch.equal(o.cpu()[~bad], good.cpu()[~bad])


@pytest.mark.gpu
def test_in_place_out_of_place_and_first_accounts():
    c = ref.Batch([200, 90], 2, 64, 32, 32, seed=12)
    pool, table, held = c.on()
    q = c.queries(8, 2).cuda()
    w0 = torch.rand(2, 2, 224, device="cuda")
    w = w0.clone()
    a = fa.attention_decode_kv4(q, pool, table, held, weights=w)
    assert a[2].data_ptr() == w.data_ptr()
    out = w0.clone()
    b = fa.attention_decode_kv4(q, pool, table, held, weights=w0, weights_out=out)
    assert torch.equal(a[2], b[2])
    first = torch.full_like(w0, -1.0)
    d = fa.attention_decode_kv4(q, pool, table, held, weights_out=first)
    for i, n in enumerate(c.lengths):
        assert torch.equal(first[i, :, n:], torch.full_like(first[i, :, n:], -1.0))
        # the weights of a row sum to one: 2^-20 each way for exponential and sums
        assert torch.allclose(first[i, :, :n].sum(-1), torch.full((2,), 8.0, device="cuda"), atol=8 * 2.0 ** -16)
    o, lse = fa.attention_decode_kv4(q, pool, table, held)
    assert torch.equal(o, d[0]) and torch.equal(o, a[0]) and torch.equal(lse, a[1])


@pytest.mark.gpu
def test_same_call_same_bits_on_streams_and_in_graphs():
    c = ref.Batch([3000, 1, 900, 64], 2, 128, 64, 16, seed=13)
    pool, table, held = c.on()
    q = c.queries(8, 1).cuda()
    o, lse, w = fa.attention_decode_kv4(q, pool, table, held, weights_out=torch.zeros(4, 2, 3008, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 4:      # overlapping calls do not share a workspace
        out = torch.zeros(4, 2, 3008, device="cuda")
        torch.cuda.synchronize()
        got.append(fa.attention_decode_kv4(q, pool, table, held, weights_out=out, stream=s))
    torch.cuda.synchronize()
    for a in got:
        assert all(torch.equal(x, y) for x, y in zip(a, (o, lse, w)))
    # two graphs captured one after the other, replayed in turn on changed lengths and queries
    qs, ls = q.clone(), held.clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.attention_decode_kv4(qs, pool, table, ls))
        graphs.append(g)
    for lengths in ([3000, 1, 900, 64], [17, 0, 901 - 5, 3]):
        ls.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = fa.attention_decode_kv4(qs, pool, table, ls)
        for g, out in zip(graphs, outs):
            for t in out:
                t.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert fa.fa_get_device_status() == 0


@pytest.mark.gpu
def test_c_entry_takes_its_own_workspace_or_refuses_a_small_one():
    import ctypes
    c = ref.Batch([2500, 20], 2, 64, 64, 16, seed=14)
    pool, table, held = c.on()
    q = c.queries(4, 1).cuda()
    want = fa.attention_decode_kv4(q, pool, table, held)
    from online_softmax_05_gb300.kv4 import _cache
    packed = _cache(pool, table, held)[0]
    lib, o, lse = fa.load_library(), torch.empty_like(q), torch.empty(2, 4, 1, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert lib.fa_kv4_decode(packed, q.data_ptr(), o.data_ptr(), lse.data_ptr(), 4, 1, 0.125, 1, None, None, 0, None, 0,
                             st) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    need = lib.fa_kv4_decode_workspace(2, 4, 2, 1, 64, c.table.shape[1] * 16, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert lib.fa_kv4_decode(packed, q.data_ptr(), o.data_ptr(), lse.data_ptr(), 4, 1, 0.125, 1, None, None, 0,
                             ws.data_ptr(), need - 1, st) == -10
    assert isinstance(ctypes.c_int(need).value, int)


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported():
    c = ref.Batch([100, 60], 2, 64, 64, 16, seed=15)
    pool, table, held = c.on()
    q = c.queries(4, 1).cuda()
    good, lse = fa.attention_decode_kv4(q, pool, table, held)
    for bad in (torch.tensor([table.shape[1] * 16 + 1, 60]), torch.tensor([-4, 60])):
        o, l2 = fa.attention_decode_kv4(q, pool, table, bad.int().cuda())
        assert fa.fa_get_device_status() == -11
        assert not o[0].any() and torch.isneginf(l2[0]).all() and torch.equal(o[1], good[1])
    for page in (-1, c.pool.shape[0], 2 ** 31 - 1):
        broken = table.clone()
        broken[0, 2] = page
        o, l2, w = fa.attention_decode_kv4(q, pool, broken, held, weights_out=torch.zeros(2, 2, 112, device="cuda"))
        assert fa.fa_get_device_status() == -13
        assert torch.equal(o[1], good[1]) and torch.isfinite(o).all() and torch.isfinite(w).all()
        assert not w[0, :, 32:48].any()
    w = torch.zeros(2, 2, 64, device="cuda")      # accounts shorter than the sequence
    fa.attention_decode_kv4(q, pool, table, held, weights=w)
    assert fa.fa_get_device_status() == -11
    assert not w[0].any() and w[1].any()


@pytest.mark.gpu
def test_reading_back_and_decoding_in_bf16_agree():
    # the same attention through attention_decode on what kv4_read returns: the values there
    # are rounded to bf16 (2^-8), the scores by as much of their terms
    c = ref.Batch([256, 256], 4, 128, 64, 64, seed=16)
    pool, table, held = c.on()
    q = c.queries(4, 1).cuda()
    o, _ = fa.attention_decode_kv4(q, pool, table, held, causal=False)
    k, v = fa.kv4_read(pool, table, held)
    o2, _ = fa.attention_decode(q, k, v)
    for b in range(2):
        ks, km, vs, vm = c.loaded(b)
        q64 = q[b].cpu().double().numpy()
        size = np.einsum("hid,htd->hit", np.abs(q64), np.abs(ks + km)).max() * 128 ** -0.5
        bound = (2.0 ** -7 + 2 * size * 2.0 ** -8) * np.abs(vs + vm).max()
        assert np.abs((o[b] - o2[b]).cpu().double().numpy()).max() <= bound


def rescaled(c, part, factor=1.0, minima=None, steps=None):
    """Multiplies the (s, m) pairs of the keys (part 1) or values (3) by `factor`, which broadcasts to
    (pages, heads, blocks, 16, groups); `steps` and `minima` replace s and m first."""
    at, size = ref.sections(c.dim, c.group)[part]
    pairs = torch.from_numpy(c.pool[..., at:at + 16 * size].copy()).view(torch.bfloat16)
    x = pairs.double().view(*pairs.shape[:-1], 16, -1, 2)
    for i, given in ((0, steps), (1, minima)):
        if given is not None:
            x[..., i] = torch.where(x[..., i].isnan(), x[..., i], torch.as_tensor(given, dtype=torch.float64))
    x = x * torch.as_tensor(factor, dtype=torch.float64)[..., None]
    pairs = x.float().to(torch.bfloat16).view(pairs.shape)     # powers of two: exact
    c.pool[..., at:at + 16 * size] = pairs.view(torch.uint8).numpy()


def place(c, b, t):
    """The pool's (page, block, row) of a token."""
    return c.table[b][t // c.page], t % c.page // 16, t % 16


# a head to a CTA; cut over CTAs; whole heads in a warp; several heads a CTA, joined by a warp each
SHAPES = [([117, 40], 2, 4, 1), ([5000, 77], 2, 4, 2), ([30, 31, 900], 2, 16, 1), ([(i * 37) % 101 for i in range(90)], 8, 4, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("lengths,heads,each,tq", SHAPES)
def test_values_near_the_largest_bf16_numbers_stay_finite(lengths, heads, each, tq, dim, group):
    # groups that span 2^125 and minima of -2^123, as kv4_append stores them and kv4_read returns them
    c = ref.Batch(lengths, heads, dim, group, 64, seed=21)
    rescaled(c, 3, 2.0 ** 122)
    got = run(c, heads * each, tq)
    assert torch.isfinite(got[0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("lengths,heads,each,tq", SHAPES)
@pytest.mark.parametrize("apart", [11, 14, 16, 20, 30, 100])
def test_groups_whose_scales_lie_far_apart(lengths, heads, each, tq, dim, group, apart):
    # one group's values 2^20 to 2^100 times the others'; D = G = 64 has one group: its heads instead
    c = ref.Batch(lengths, heads, dim, group, 64, seed=22)
    factor = torch.ones(heads, 1, 1, dim // group, dtype=torch.float64)
    factor[(slice(None), 0, 0, 0) if dim > group else (0,)] = 2.0 ** apart
    rescaled(c, 3, factor * 2.0 ** (-apart // 2))
    run(c, heads * each, tq)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("lengths,heads,each,tq", SHAPES)
@pytest.mark.parametrize("apart", [13, 16, 20, 30])
def test_a_huge_value_of_little_weight_hides_no_other(lengths, heads, each, tq, dim, group, apart):
    # the token that weighs least holds values 2^20 or 2^30 times the others'
    c = ref.Batch(lengths, heads, dim, group, 64, seed=23)
    pool, table, held = c.on()
    q = c.queries(heads * each, tq, 3.0)
    factor = torch.ones(*c.pool.shape[:3], 16, dim // group, dtype=torch.float64)
    for b, n in enumerate(lengths):
        if n < 2 * tq:
            continue
        p = ref.attend(q[b].double().numpy(), c.loaded(b), dim ** -0.5, True)[2]
        for h, t in enumerate(p[:, :n - tq].argmin(-1)):
            page, block, r = place(c, b, t)
            factor[page, h, block, r] = 2.0 ** apart
    rescaled(c, 3, factor)
    pool = torch.from_numpy(c.pool).cuda()
    o, lse = fa.attention_decode_kv4(q.cuda(), pool, table, held)
    assert fa.fa_get_device_status() == 0
    check(c, q, o, lse, dim ** -0.5, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("first", [0, 320, 640])
@pytest.mark.parametrize("apart", [30, 50])
def test_a_stretch_of_huge_values_of_little_weight(apart, first, dim, group):
    # 128 tokens whose scores are 0, far below the others' largest, with values 2^30 or 2^50 times the others'
    c = ref.Batch([768, 700], 2, dim, group, 64, seed=29)
    keys, values = (torch.ones(*c.pool.shape[:3], 16, dim // group, dtype=torch.float64) for _ in range(2))
    for b in range(2):
        for t in range(first, min(first + 128, c.lengths[b])):
            page, block, r = place(c, b, t)
            keys[page, :, block, r], values[page, :, block, r] = 0.0, 2.0 ** apart
    rescaled(c, 1, keys)
    rescaled(c, 3, values)
    q = c.queries(8, 1, 6.0)
    pool, table, held = c.on()
    o, lse = fa.attention_decode_kv4(q.cuda(), pool, table, held)
    assert fa.fa_get_device_status() == 0
    check(c, q, o, lse, dim ** -0.5, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", [(128, 64), (128, 32), (64, 64)])
@pytest.mark.parametrize("first", [0, 300, 699])
def test_a_huge_scale_whose_codes_are_zero_adds_nothing(dim, group, first):
    # all minima 0; one token's scale is 2^24 times the others', its codes 0: what is left is the others' sum
    c = ref.Batch([700], 2, dim, group, 64, seed=24)
    page, block, r = place(c, 0, first)
    factor = torch.ones(*c.pool.shape[:3], 16, dim // group, dtype=torch.float64)
    factor[page, :, block, r] = 2.0 ** 24
    rescaled(c, 3, factor, minima=0.0)
    at, size = ref.sections(dim, group)[2]
    c.pool[page, :, block, at + r * size:at + (r + 1) * size] = 0
    run(c, 8, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [30, 118, -118])
@pytest.mark.parametrize("each,tq", [(1, 2), (4, 4), (2, 8)])
@pytest.mark.parametrize("length", [9, 33, 700, 5000])
def test_a_token_that_a_row_does_not_see_does_not_touch_it(length, each, tq, apart):
    # the last token's values 2^118 times the others', or all others 2^118 times its own: the rows
    # before it do not see it
    c = ref.Batch([length, 1], 2, 128, 64, 64, seed=25)
    page, block, r = place(c, 0, length - 1)
    factor = torch.full((*c.pool.shape[:3], 16, 2), 2.0 ** max(0, -apart), dtype=torch.float64)
    factor[page, :, block, r] = 2.0 ** max(0, apart)
    rescaled(c, 3, factor)
    got = run(c, 2 * each, tq)
    assert torch.isfinite(got[0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("each,tq", [(4, 1), (4, 4)])
def test_finite_queries_of_any_size_give_finite_scores(dim, group, each, tq):
    # queries up to 2^124 over keys of 2^-120 (flat groups: a step of 0), and ordinary queries beside them
    c = ref.Batch([300, 40], 2, dim, group, 64, seed=26)
    rescaled(c, 1, 2.0 ** -120, steps=0.0)
    q = c.queries(2 * each, tq)
    q[:, ::2] *= 2.0 ** 122
    pool, table, held = c.on()
    w = torch.zeros(2, 2, c.table.shape[1] * 64, device="cuda")
    o, lse, w = fa.attention_decode_kv4(q.cuda(), pool, table, held, weights_out=w)
    assert fa.fa_get_device_status() == 0
    check(c, q, o, lse, dim ** -0.5, True, w)


@pytest.mark.gpu
@pytest.mark.parametrize("each", [2, 4])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_query_of_a_row_that_sees_nothing(bad, each):
    # two tokens, four queries: the first two rows see nothing, whatever they hold; a bad row spoils the
    # accounts of the tokens that it sees and of no other
    c = ref.Batch([2, 40], 2, 64, 32, 16, seed=27)
    q = c.queries(2 * each, 4)
    q[0, 0, :2, 3], q[1, 0, 1, 3] = bad, bad
    pool, table, held = c.on()
    o, lse, w = fa.attention_decode_kv4(q.cuda(), pool, table, held, weights_out=torch.zeros(2, 2, 48, device="cuda"))
    assert fa.fa_get_device_status() == 0
    assert not o[0, :, :2].any() and torch.isneginf(lse[0, :, :2]).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(w[0]).all() and torch.isfinite(lse[0, :, 2:]).all()
    assert torch.isnan(o[1, 0, 1]).all() and torch.isnan(lse[1, 0, 1])
    assert torch.isnan(w[1, 0, :38]).all() and torch.isfinite(w[1, 0, 38:]).all() and torch.isfinite(w[1, 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lengths,each", [([2500, 20], 2), ([2500, 20], 12), ([100, 20], 2), ([9000] * 3 + [5] * 40, 3)])
def test_a_workspace_of_exactly_the_size_asked_for(lengths, each, weights):
    c = ref.Batch(lengths, 2, 128, 64, 64, seed=28)
    pool, table, held = c.on()
    q = c.queries(2 * each, 1).cuda()
    slots = c.table.shape[1] * 64
    account = lambda: torch.full((len(lengths), 2, slots), 3.0, device="cuda") if weights else None  # noqa: E731
    want = fa.attention_decode_kv4(q, pool, table, held, weights_out=account())
    from online_softmax_05_gb300.kv4 import _cache
    lib, o, lse, w = fa.load_library(), torch.empty_like(q), torch.empty(q.shape[:3], device="cuda"), account()
    need = lib.fa_kv4_decode_workspace(len(lengths), 2 * each, 2, 1, 128, slots, int(weights))
    ws = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    rc = lib.fa_kv4_decode(_cache(pool, table, held)[0], q.data_ptr(), o.data_ptr(), lse.data_ptr(), 2 * each, 1,
                           128 ** -0.5, 1, None, w.data_ptr() if weights else None, slots if weights else 0,
                           ws.data_ptr() if need else None, need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and fa.fa_get_device_status() == 0
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and (not weights or torch.equal(w, want[2]))
    assert (ws[need:] == 0xa5).all()
