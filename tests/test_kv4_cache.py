"""The 4-bit paged cache: appending and reading back, bit by bit against the format's
definition, and the refusals of its entry points."""
import ctypes
import math
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


# ------------------------------------------------------------------ host
BASE = 1 << 40


def cache(**kw):
    a = dict(pool=BASE, table=2 * BASE, lengths=3 * BASE, B=2, Hkv=4, D=128, group=64, page=64, pages=10, width=5)
    a.update(kw)
    return struct.pack("QQQ7i4x", *a.values())


def append(c=None, **kw):
    a = dict(k=4 * BASE, v=5 * BASE, k_t=512, k_h=128, v_t=512, v_h=128, cu=6 * BASE, total=7, pos=None, pos64=0,
             freq=None, rotary=0, inter=0, amp=1.0, w=None, sp=None, slots=0)
    a.update(kw)
    return fa.load_library().fa_kv4_append(cache() if c is None else c, *a.values(), None)


def read(c=None, **kw):
    a = dict(start=None, count=9, k=4 * BASE, v=5 * BASE)
    a.update(kw)
    return fa.load_library().fa_kv4_read(cache() if c is None else c, *a.values(), None)


def decode(c=None, **kw):
    a = dict(q=4 * BASE, o=5 * BASE, lse=6 * BASE, Hq=8, Tq=1, scale=0.1, causal=1, w=None, wo=None, slots=0, ws=None,
             n=0)
    a.update(kw)
    return fa.load_library().fa_kv4_decode(cache() if c is None else c, *a.values(), None)


def evict(c=None, **kw):
    a = dict(w=4 * BASE, sp=5 * BASE, slots=320, budget=64, recent=8, wo=6 * BASE, po=7 * BASE, lo=8 * BASE,
             src=9 * BASE, ws=None, n=0)
    a.update(kw)
    return fa.load_library().fa_kv4_evict(cache() if c is None else c, *a.values(), None)


@pytest.mark.parametrize("call", [append, read, decode, evict])
def test_cache_descriptions_are_refused(call):
    for kw, code in ((dict(pool=0), -1), (dict(table=0), -1), (dict(lengths=0), -1), (dict(B=0), -2), (dict(Hkv=0), -2),
                     (dict(width=0), -2), (dict(pages=0), -2), (dict(page=0), -2), (dict(page=24), -3), (dict(page=1 << 17, width=1), -3), (dict(D=96), -3),
                     (dict(group=128), -3), (dict(B=1 << 14, Hkv=8), -2), (dict(width=1 << 26), -2),
                     (dict(pool=BASE + 8), -4), (dict(table=2 * BASE + 2), -4), (dict(lengths=3 * BASE + 1), -4)):
        assert call(cache(**kw)) == code, kw


def test_append_refuses():
    assert append(k=None) == -1 and append(v=None) == -1 and append(cu=None) == -1
    assert append(total=0) == -2 and append(total=1 << 30) == -2 and append(w=8 * BASE, slots=0) == -2
    assert append(freq=7 * BASE, rotary=130) == -3 and append(freq=7 * BASE, rotary=3) == -3
    assert append(k=4 * BASE + 8) == -4 and append(k_t=516) == -4 and append(cu=6 * BASE + 2) == -4
    assert append(k_h=-128) == -8 and append(freq=7 * BASE, rotary=64, inter=2) == -8
    assert append(freq=7 * BASE, rotary=64, amp=math.inf) == -8 and append(pos64=3) == -8
    assert append(k=BASE + 64) == -8                                  # keys inside the pool
    assert append(w=8 * BASE, sp=8 * BASE, slots=64) == -8            # one buffer for both accounts
    assert append(w=3 * BASE, slots=64) == -8                         # weights over the lengths


def test_read_refuses():
    assert read(k=None) == -1 and read(count=0) == -2 and read(count=1 << 30) == -2
    assert read(k=4 * BASE + 8) == -4 and read(start=6 * BASE + 2) == -4
    assert read(v=4 * BASE) == -8 and read(k=BASE) == -8


def test_decode_refuses():
    assert decode(q=None) == -1 and decode(lse=None) == -1 and decode(w=7 * BASE, slots=320) == -1
    assert decode(Hq=6) == -2 and decode(Tq=0) == -2 and decode(wo=7 * BASE, slots=0) == -2
    assert decode(Tq=9) == -3 and decode(Hq=4 * 1025) == -3
    assert decode(q=4 * BASE + 2) == -4 and decode(wo=7 * BASE + 1, slots=320) == -4
    assert decode(causal=2) == -8 and decode(scale=math.nan) == -8
    assert decode(o=4 * BASE) == -8 and decode(o=BASE) == -8 and decode(wo=6 * BASE, slots=320) == -8
    lib = fa.load_library()
    assert lib.fa_kv4_decode_workspace(2, 6, 4, 1, 128, 320, 0) == -2
    assert lib.fa_kv4_decode_workspace(2, 8, 4, 1, 96, 320, 0) == -3
    assert lib.fa_kv4_decode_workspace(2, 8, 4, 1, 128, 300, 0) == -2


def test_evict_refuses():
    assert evict(w=None) == -1 and evict(src=None) == -1
    assert evict(slots=0) == -2 and evict(budget=0) == -2
    assert evict(recent=65) == -8 and evict(recent=-1) == -8
    assert evict(w=4 * BASE + 2) == -4
    assert evict(wo=4 * BASE) == -8 and evict(po=6 * BASE) == -8 and evict(lo=3 * BASE) == -8
    assert fa.load_library().fa_kv4_evict_workspace(0, 4, 64) == -2


def test_page_lookup_on_the_host():
    # the kernels' own lookup: a page outside the pool or past the table is refused
    lib = fa.load_library()
    table = (ctypes.c_int * 8)(3, 9, 10, -1, 0, 1, 2, 2 ** 31 - 1)
    size = 16 * (128 + 8 * 2)

    def at(b, h, slot):
        return lib.fa_kv4_block_offset(table, 4, 2, 128, 64, 32, 10, b, h, slot)

    for b, row in enumerate(([3, 9, 10, -1], [0, 1, 2, 2 ** 31 - 1])):
        for slot in range(0, 160):
            page = row[slot // 32] if slot < 128 else -1
            want = -13 if not 0 <= page < 10 else ((page * 2 + 1) * 2 + slot % 32 // 16) * size
            assert at(b, 1, slot) == want, (b, slot)
    assert at(-1, 0, 0) == -2 and at(0, 2, 0) == -2 and at(0, 0, -1) == -2


def test_pool_refuses():
    for kw in (dict(dim=96), dict(group=16), dict(page_size=40), dict(num_pages=0)):
        with pytest.raises(ValueError):
            fa.kv4_pool(**{"num_pages": 4, "kv_heads": 2, "dim": 64, "device": "cpu", **kw})
    with pytest.raises(ValueError):
        fa.kv4_read(fa.kv4_pool(4, 2, 64, device="cpu"), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_reference_format_reads_back_within_half_a_step():
    rng = np.random.default_rng(0)
    x = ref.bf16(rng.standard_normal((5, 64))).float().numpy()
    codes, s, m = ref.quantise(x, 32)
    back = codes.reshape(5, 2, 32) * s[..., None] + m[..., None]
    assert np.abs(back - x.reshape(5, 2, 32)).max() <= (s * (0.5 + 15 * 2.0 ** -8)).max()


# ------------------------------------------------------------------ GPU
def batch_append(lengths, new, heads, dim, group, page, seed, values=None, rotary=None, positions=None, strided=False,
                 **kw):
    """Appends through the entry point into a pool of noise; -> (pool before, pool after, want)."""
    c = ref.Batch(lengths, heads, dim, group, page, seed)
    before = c.pool.copy()
    total = sum(new)
    g = torch.Generator().manual_seed(seed)
    if values is None:
        k, v = ((torch.randn(total, heads, dim, generator=g) * 2).to(torch.bfloat16) for _ in range(2))
    else:
        k, v = values(total, heads, dim)
    if strided:
        both = torch.cat((k, v), 1).cuda()
        kd, vd = both[:, :heads], both[:, heads:]
    else:
        kd, vd = k.cuda(), v.cuda()
    pool, table, held = c.on()
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()
    fa.kv4_append(pool, kd, vd, table, held, cu, rotary=rotary, positions=positions, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    if rotary is not None:
        where = positions
        if where is None:
            where = torch.cat([torch.arange(n - m, n) for n, m in zip(lengths, new)]).cuda()
        k = fa.rope(kd.transpose(0, 1)[None], None, rotary, where, interleaved=kw.get("interleaved", False),
                    amplitude=kw.get("amplitude", 1.0))[0].transpose(0, 1).cpu()
    at = 0
    for b, (n, m) in enumerate(zip(lengths, new)):
        for i in range(m):
            ref.store(before, c.table, b, n - m + i, k[at].float().numpy(), v[at].float().numpy(), group)
            at += 1
    return pool.cpu().numpy(), before


FORMATS = [(128, 64), (128, 32), (64, 64), (64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("lengths,new,heads,page", [
    ([1], [1], 1, 16), ([37, 5, 0, 130], [37, 2, 0, 31], 3, 16), ([64, 65, 63], [1, 1, 1], 8, 64),
    ([100, 33], [0, 33], 2, 48)])
def test_append_writes_the_format(lengths, new, heads, page, dim, group):
    # every byte of the pool: the new tokens' records, and nothing else
    got, want = batch_append(lengths, new, heads, dim, group, page, seed=dim + len(lengths))
    assert np.array_equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
def test_append_of_strided_views(dim, group):
    got, want = batch_append([50, 20], [30, 20], 2, dim, group, 16, seed=3, strided=True)
    assert np.array_equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rotary,interleaved,far", [(64, False, 0), (64, True, 0), (20, False, 10 ** 6), (62, True, 7),
                                                    (2, False, 3)])
def test_append_rotates_as_rope_does(dim, rotary, interleaved, far):
    table = fa.rotary_frequencies(rotary, device="cuda")
    positions = torch.arange(41, device="cuda") * 3 + far if far else None
    got, want = batch_append([60, 12, 9], [25, 7, 9], 4, dim, 32, 32, seed=rotary, rotary=table,
                             positions=positions, interleaved=interleaved, amplitude=1.125)
    assert np.array_equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
def test_append_rounds_both_products_of_a_turn(dim):
    # pairs whose turned channel is a tie between two bf16 numbers when both products are rounded to
    # 32 bits, and is not when one of them goes into the sum as it is; the smallest of its group, so
    # that the cache holds it as the group's minimum, exactly
    table = fa.rotary_frequencies(64, device="cpu")
    to_bf16 = lambda x: ref.bf16(x).float().numpy()
    rng, hits = np.random.default_rng(11), []
    turns = table.numpy().view(np.uint64)
    for _ in range(4):
        n = 1 << 21
        pos, i = rng.integers(0, 1000, n), rng.integers(0, 32, n)
        a, b = (to_bf16(rng.standard_normal(n)) for _ in range(2))
        angle = (pos.astype(np.uint64) * turns[i]).astype(np.float64) * (2 * np.pi / 2.0 ** 64)
        c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        x, y = a * c, b * s
        u = x - y
        first = (a.astype(np.float64) * c - y).astype(np.float32)
        second = (x - b.astype(np.float64) * s).astype(np.float32)
        sign = np.where(u > 0, -1, 1).astype(np.float32)
        hit = (to_bf16(u) != to_bf16(first)) | (to_bf16(u) != to_bf16(second))
        hits += [z[hit] for z in (pos, i, a * sign, b * sign, to_bf16(u) * sign)]
    pos, i, a, b, u = (np.concatenate(hits[z::5]) for z in range(5))
    n = len(pos)
    assert n > 40
    k, at = torch.zeros(n, 1, dim), torch.arange(n)
    k[at, 0, i], k[at, 0, i + 32] = torch.from_numpy(a), torch.from_numpy(b)
    k = k.to(torch.bfloat16).cuda()
    pool = fa.kv4_pool(n // 16 + 1, 1, dim, page_size=16, group=32)
    pages = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda")[None]
    held, cu = (torch.tensor(z, dtype=torch.int32, device="cuda") for z in ([n], [0, n]))
    fa.kv4_append(pool, k, torch.zeros_like(k), pages, held, cu, rotary=table.cuda(), positions=torch.from_numpy(pos).cuda())
    got = fa.kv4_read(pool, pages, held)[0][0, 0].float().cpu().numpy()
    assert np.array_equal(got[np.arange(n), i], u)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64])
def test_append_of_hard_groups(group):
    # equal values, tiny and huge ranges, subnormals, infinities and NaN, ties on the grid
    def values(total, heads, dim):
        x = torch.zeros(total, heads, dim)
        x[0] = 3.0
        x[1] = torch.arange(heads * dim).view(heads, dim).float() % 16          # codes exactly
        x[2] = torch.arange(heads * dim).view(heads, dim).float() % 31 / 2      # half of them ties
        x[3] = torch.linspace(-3e38, 3e38, heads * dim).view(heads, dim)
        x[4] = torch.linspace(-1e-37, 1e-37, heads * dim).view(heads, dim)
        x[5] = torch.randn(heads, dim, generator=torch.Generator().manual_seed(1))
        x[5, 0, 3], x[5, 0, dim - 1], x[5, 1, 5] = math.inf, math.nan, -math.inf
        x[6] = 100.0 + torch.arange(heads * dim).view(heads, dim).float() % 2 * 0.5
        x[7] = torch.where(torch.arange(dim) % 7 == 0, 1e30, 1.0)
        x[8] = -0.0
        return x.to(torch.bfloat16), x.flip(0).to(torch.bfloat16)
    got, want = batch_append([11], [9], 2, 128, group, 16, seed=1, values=values)
    # a NaN scale may be any NaN; a zero minimum either zero
    parts = ref.sections(128, group)
    for i, (at, size) in enumerate(parts):
        x, y = got[..., at:at + 16 * size], want[..., at:at + 16 * size]
        if i % 2 == 0:
            assert np.array_equal(x, y)
        else:
            x, y = (torch.from_numpy(t.copy()).view(torch.bfloat16).float().numpy() for t in (x, y))
            assert np.array_equal(x, y, equal_nan=True)

@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("page", [16, 80])
def test_read_returns_what_the_codes_stand_for(dim, group, page):
    c = ref.Batch([1, 0, 97, 160], 3, dim, group, page, seed=dim + group)
    pool, table, held = c.on()
    for start, count in ((None, None), (torch.tensor([0, 0, 90, 31], dtype=torch.int32).cuda(), 29)):
        k, v = fa.kv4_read(pool, table, held, start=start, count=count)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == 0
        n = k.shape[2]
        assert n == (c.table.shape[1] * page if count is None else count)
        for b, length in enumerate(c.lengths):
            first = 0 if start is None else int(start[b])
            ks, km, vs, vm = c.loaded(b)
            for got, want in ((k[b], ks + km), (v[b], vs + vm)):
                full = np.zeros((3, n, dim))
                part = want[:, first:first + n]
                full[:, :part.shape[1]] = part
                # code * s is exact in fp32 (12 bits), one rounding of the sum, one to bf16
                assert torch.equal(got.cpu(), torch.from_numpy(full).float().to(torch.bfloat16))


@pytest.mark.gpu
def test_append_fills_the_accounts():
    lengths, new = [9, 40, 3], [2, 40, 0]
    c = ref.Batch(lengths, 2, 64, 64, 16, seed=0)
    pool, table, held = c.on()
    k = torch.randn(42, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 2, 42, 42], dtype=torch.int32).cuda()
    w = torch.full((3, 2, 44), 7.0, device="cuda")
    p = torch.full((3, 2, 44), -5, dtype=torch.int32, device="cuda")
    positions = torch.arange(1000, 1042, device="cuda")
    fa.kv4_append(pool, k, k, table, held, cu, positions=positions, weights=w, slot_positions=p)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    want_w, want_p = torch.full((3, 2, 44), 7.0), torch.full((3, 2, 44), -5, dtype=torch.int32)
    want_w[0, :, 7:9], want_w[1, :, :40] = 0, 0
    want_p[0, :, 7:9] = torch.arange(1000, 1002, dtype=torch.int32)
    want_p[1, :, :40] = torch.arange(1002, 1042, dtype=torch.int32)
    assert torch.equal(w.cpu(), want_w) and torch.equal(p.cpu(), want_p)


@pytest.mark.gpu
def test_rows_outside_the_sequences_are_not_used():
    c = ref.Batch([20, 20], 2, 64, 32, 16, seed=5)
    pool, table, held = c.on()
    k = torch.randn(30, 2, 64, device="cuda").to(torch.bfloat16)
    k[:4], k[24:] = math.nan, math.nan
    fa.kv4_append(pool, k, k, table, held, torch.tensor([4, 14, 24], dtype=torch.int32).cuda())
    got = fa.kv4_read(pool, table, held, start=torch.tensor([10, 10], dtype=torch.int32).cuda(), count=10)
    assert fa.fa_get_device_status() == 0
    assert all(torch.isfinite(t).all() for t in got)


@pytest.mark.gpu
def test_lengths_and_pages_that_do_not_fit_are_reported():
    # the kernels check every slot and page against the table and the pool (the lookup is
    # tested on the host above): nothing outside is touched, the rest is done
    lengths = [20, 40]
    c = ref.Batch(lengths, 2, 64, 64, 16, seed=2)
    pool, table, held = c.on()
    k = torch.randn(8, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
    before = pool.clone()
    for bad, status in ((torch.tensor([2, 40]), -11), (torch.tensor([-1, 40]), -11), (torch.tensor([20, 49]), -11)):
        pool.copy_(before)
        fa.kv4_append(pool, k, k, table, bad.int().cuda(), cu)
        assert fa.fa_get_device_status() == status
        assert fa.fa_get_device_status() == 0
    pool.copy_(before)          # accounts shorter than a sequence: its tokens are not stored
    fa.kv4_append(pool, k, k, table, held, cu, weights=torch.zeros(2, 2, 30, device="cuda"))
    assert fa.fa_get_device_status() == -11
    whole = before.clone()
    fa.kv4_append(whole, k, k, table, held, cu)
    at = table[0].tolist()[:2]
    assert torch.equal(pool[at], whole[at]) and torch.equal(pool[table[1, :3].long()], before[table[1, :3].long()])
    broken = table.clone()
    broken[0, 1] = c.pool.shape[0]
    pool.copy_(before)
    fa.kv4_append(pool, k, k, broken, held, cu)
    assert fa.fa_get_device_status() == -13
    kk, _ = fa.kv4_read(pool, broken, held)
    assert fa.fa_get_device_status() == -13
    assert not kk[0, :, 16:].any() and kk[1, :, :40].any()
    fa.kv4_read(pool, table, held, start=torch.tensor([-3, 0], dtype=torch.int32).cuda(), count=4)
    assert fa.fa_get_device_status() == -11


@pytest.mark.gpu
def test_python_entries_refuse():
    pool = fa.kv4_pool(8, 2, 64, page_size=16, group=32)
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    held = torch.zeros(2, dtype=torch.int32, device="cuda")
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 2, 48, device="cuda")
    p = torch.zeros(2, 2, 48, dtype=torch.int32, device="cuda")
    for bad in (lambda: fa.kv4_read(pool.float(), table, held), lambda: fa.kv4_read(pool, table.long(), held),
                lambda: fa.kv4_read(pool, table, held[:1]), lambda: fa.kv4_read(pool[..., :-16], table, held),
                lambda: fa.kv4_read(pool, table.cpu(), held), lambda: fa.kv4_append(pool, k.float(), k, table, held, cu),
                lambda: fa.kv4_append(pool, k[:, :1], k, table, held, cu),
                lambda: fa.kv4_append(pool, k, k[:3], table, held, cu),
                lambda: fa.kv4_append(pool, k, k, table, held, cu[:2]),
                lambda: fa.kv4_append(pool, k, k, table, held, cu, rotary=table),
                lambda: fa.kv4_append(pool, k, k, table, held, cu, weights=w[:, :, :40], slot_positions=p),
                lambda: fa.attention_decode_kv4(q.float(), pool, table, held),
                lambda: fa.attention_decode_kv4(q[:1], pool, table, held),
                lambda: fa.attention_decode_kv4(q, pool, table, held, weights=w.double()),
                lambda: fa.attention_decode_kv4(q, pool, table, held, lse=w),
                lambda: fa.kv4_evict(pool, table, held, w, p.float(), 4),
                lambda: fa.kv4_evict(pool, table, held, w[:, :1], p, 4)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fa.kv4_evict(pool, table, held, w, p, 0), lambda: fa.kv4_evict(pool, table, held, w, p, 4, 5),
                lambda: fa.attention_decode_kv4(q.expand(2, 4, 1, 64).repeat(1, 1, 9, 1), pool, table, held),
                lambda: fa.attention_decode_kv4(q[:, :3].contiguous(), pool, table, held),
                lambda: fa.kv4_read(pool, table, held, count=0)):
        with pytest.raises(fa.FAError):
            bad()


@pytest.mark.gpu
def test_pages_behind_the_first_four_gigabytes():
    # a pool of 5 GB, the sequences' pages at its end: append, read, decode and evict there
    heads, dim, group, page = 8, 128, 64, 64
    pages = 5 * 2 ** 30 // (heads * page * 144)
    pool = torch.empty(pages, heads, page // 16, 16 * 144, dtype=torch.uint8, device="cuda")
    width = 12
    rng = np.random.default_rng(0)
    table = torch.from_numpy((pages - 1 - rng.permutation(2 * width)).reshape(2, width).astype(np.int32)).cuda()
    assert int(table.min()) * heads * page * 144 > 2 ** 32
    held = torch.tensor([700, 300], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 700, 1000], dtype=torch.int32).cuda()
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn(1000, heads, dim, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, heads, 1, dim, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.rand(2, heads, 768, device="cuda", generator=g)
    p = torch.arange(768, dtype=torch.int32, device="cuda").expand(2, heads, 768).contiguous()

    def steps(pool, table):
        fa.kv4_append(pool, k, v, table, held, cu)
        out = [*fa.kv4_read(pool, table, held), *fa.attention_decode_kv4(q, pool, table, held)]
        got = fa.kv4_evict(pool, table, held, w, p, 200, 20)
        return out + [*got, *fa.kv4_read(pool, table, got[2], count=200)]

    small = fa.kv4_pool(2 * width, heads, dim, page_size=page, group=group)
    want = steps(small, torch.arange(2 * width, dtype=torch.int32, device="cuda").view(2, width))
    got = steps(pool, table)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("start", [None, [0, 0], [-3, 10]])
@pytest.mark.parametrize("bad", [49, -1, 20])
def test_reading_a_sequence_that_cannot_be_counts_it_as_empty(bad, start):
    # a length the table of 48 slots cannot hold, a negative one, a negative start: zeros, and a status
    c = ref.Batch([20, 40], 2, 64, 64, 16, seed=30)
    pool, table, held = c.on()
    if bad == 20 and (start is None or start[0] >= 0):
        return
    want = fa.kv4_read(pool, table, held)
    lengths = torch.tensor([bad, 40], dtype=torch.int32).cuda()
    first = None if start is None else torch.tensor(start, dtype=torch.int32).cuda()
    for x, y in zip(fa.kv4_read(pool, table, lengths, start=first, count=None if start is None else 30), want):
        assert not x[0].any()
        assert torch.equal(x[1], y[1] if start is None else y[1, :, start[1]:start[1] + 30])
    assert fa.fa_get_device_status() == -11
    assert fa.fa_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("length,slots", [(2, None), (-1, None), (50, None), (2 ** 31 - 1, None), (32, 30)])
def test_a_sequence_without_room_for_its_tokens_stores_none(length, slots):
    # fewer tokens than new ones, more than the table's 48 slots or than the accounts', by less than
    # the new tokens: the pool and the accounts stay as they are, the other sequence's tokens are stored
    c = ref.Batch([20, 29], 2, 64, 64, 16, seed=31, spare=1)
    c.table[0] = c.table[0][0], c.table[1][0], c.pool.shape[0] - 1       # three pages for each sequence
    c.table[1] = [x for x in range(c.pool.shape[0]) if x not in c.table[0].tolist()][:3]
    pool, table, _ = c.on()
    before = pool.clone()
    k = torch.randn(8, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
    alone = torch.tensor([4, 4, 8], dtype=torch.int32).cuda()             # the second sequence's tokens only
    new = lambda: (torch.full((2, 2, slots or 48), 7.0, device="cuda"),   # noqa: E731
                   torch.full((2, 2, slots or 48), -5, dtype=torch.int32, device="cuda"))
    held = torch.tensor([length, 29], dtype=torch.int32).cuda()
    want, accounts = new(), new()
    fa.kv4_append(pool, k, k, table, held, cu, weights=accounts[0], slot_positions=accounts[1])
    assert fa.fa_get_device_status() == -11
    fa.kv4_append(before, k, k, table, held, alone, weights=want[0], slot_positions=want[1])
    assert fa.fa_get_device_status() == 0
    assert torch.equal(pool, before) and torch.equal(accounts[0], want[0]) and torch.equal(accounts[1], want[1])
    assert (want[0][1, :, 25:29] == 0).all()


@pytest.mark.gpu
def test_accounts_of_positions_beyond_32_bits_are_reported():
    # they would come back wrapped, the newest token as the oldest; the keys' own rotation takes them
    c = ref.Batch([6], 1, 64, 64, 16, seed=32)
    pool, table, held = c.on()
    k = torch.randn(6, 1, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 6], dtype=torch.int32).cuda()
    positions = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, 2 ** 40, -2 ** 31, -2 ** 31 - 1], device="cuda")
    freq = fa.rotary_frequencies(64, device="cuda")
    p = torch.zeros(1, 1, 16, dtype=torch.int32, device="cuda")
    fa.kv4_append(pool, k, k, table, held, cu, rotary=freq, positions=positions)
    assert fa.fa_get_device_status() == 0
    want = pool.clone()
    fa.kv4_append(pool, k, k, table, held, cu, rotary=freq, positions=positions, slot_positions=p)
    assert fa.fa_get_device_status() == -11
    assert p[0, 0, :6].tolist() == [0] + [2 ** 31 - 1] * 3 + [-2 ** 31] * 2 and torch.equal(pool, want)
    fa.kv4_append(pool, k, k, table, held, cu, rotary=freq, positions=positions.clamp(-2 ** 31, 2 ** 31 - 1), slot_positions=p)
    assert fa.fa_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("total,heads,strides", [(1, 2, (133, 64, 1)), (5, 1, (64, 3, 1)), (1, 1, (7, 13, 1))])
def test_append_takes_any_stride_of_a_single_token_or_head(total, heads, strides):
    g = torch.Generator().manual_seed(33)
    flat = torch.randn(2 * total * heads * 64 + 256, generator=g).to(torch.bfloat16).cuda()
    k, v = (flat[at:].as_strided((total, heads, 64), strides) for at in (0, 128))
    held, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([total], [0, total]))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    pools = [fa.kv4_pool(1, heads, 64, page_size=16, group=32) for _ in range(2)]
    freq = fa.rotary_frequencies(20, device="cuda")
    fa.kv4_append(pools[0], k, v, table, held, cu, rotary=freq)
    fa.kv4_append(pools[1], k.contiguous().view(-1).view(total, heads, 64).clone(), v.clone(memory_format=torch.contiguous_format),
                  table, held, cu, rotary=freq)
    assert fa.fa_get_device_status() == 0
    assert pools[0].any() and torch.equal(*pools)


@pytest.mark.gpu
def test_numbers_beyond_32_bits_are_refused():
    # a C int would hold their low 32 bits: recent = 2^32 would protect nothing
    pool = fa.kv4_pool(4, 1, 64, page_size=16, group=32)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    held, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([60], [0, 1]))
    w, p = torch.rand(1, 1, 64, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda")[None, None]
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(2 ** 32 + 1, 1, 64)
    for bad in (lambda: fa.kv4_evict(pool, table, held, w, p, 8, 2 ** 32), lambda: fa.kv4_evict(pool, table, held, w, p, 2 ** 32 + 8),
                lambda: fa.kv4_evict(pool, table, held, w, p, 8, -2 ** 32), lambda: fa.kv4_read(pool, table, held, count=2 ** 32 + 8),
                lambda: fa.kv4_append(pool, k, k, table, held, cu)):
        with pytest.raises(ValueError):
            bad()
