"""Joining the pieces of a cut batch: what the joining kernel reads, of batches whose cut uses every CTA
that there is and leaves whole units behind the cut ones, by the plan restated on the host, by what the kernels
leave in a workspace, and by the debug library, which checks each unit's pieces against the room for them."""
import ctypes
import os
import random

import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as kv4
from tests import split_ref as plan
from tests.cross_ref import check, reference
from tests.test_kv4_tree import check as check_tree
from tests.test_kv4_tree import trees

PKG = os.path.dirname(os.path.abspath(fa.__file__))

# (lengths, query heads, kv heads, rows, D): every item in use on 152 SMs, units of one piece last
CROSS = [([14000, 200], 8, 8, 64, 64), ([303 * 128, 0], 1, 1, 1, 128), ([606 * 128, 100], 1, 1, 1, 64),
         ([14000, 200], 16, 8, 32, 128), ([5000, 9000, 77, 3000], 4, 4, 20, 64)]
TREES = [([14200, 0], 4, 4, 47, 64, 32), ([453 * 128, 0], 1, 1, 8, 128, 64), ([9000, 40, 300], 4, 2, 40, 128, 64)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from online_softmax_05_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def debug():
    """The debug library, with the product's argument types."""
    lib, like = ctypes.CDLL(os.path.join(PKG, "libfa_debug.so")), fa.load_library()
    for name in ("fa_cross_fwd", "fa_cross_fwd_workspace", "fa_kv4_tree", "fa_kv4_tree_workspace", "fa_get_device_status"):
        getattr(lib, name).argtypes = getattr(like, name).argtypes
        getattr(lib, name).restype = getattr(like, name).restype
    return lib


def tiles(lengths):
    return [plan.ceil(n, 128) for n in lengths]


# ------------------------------------------------------------------ the plan (no GPU)

@pytest.mark.parametrize("sms", [152, 148, 7])
def test_no_piece_that_is_read_lies_behind_the_room_for_them(sms):
    rng = random.Random(sms)
    for _ in range(300):
        B, heads = rng.choice([1, 2, 3, 8, 31, 32, 33, 128, 129, 300, 512, 513]), rng.choice([1, 2, 8])
        most = rng.choice([1, 128, 129, 1000, 14000, 80000])
        lengths = [rng.choice([0, 1, rng.randint(0, most), most]) for _ in range(B)]
        for p in (plan.cross_plan(B, heads, heads, rng.choice([1, 64, 300]), most, sms)[0],
                  plan.tree_plan(B, heads, heads, rng.choice([1, 64]), plan.ceil(most, 16) * 16, sms)[0]):
            units = plan.units_of(p, tiles(lengths))
            assert sum(n for _, n in units.values()) <= p.items
            read = plan.joined(units)
            assert all(r.start >= 0 and r.stop <= p.room for r in read)
            taken = [i for r in read for i in r]
            assert len(taken) == len(set(taken))          # no two units share a piece


def test_whole_units_behind_the_cut_ones_name_a_piece_past_the_room():
    """What the cases below are made of: such an entry is not to be read through."""
    for p, lengths in [(plan.cross_plan(2, *s[1:4], max(s[0]), 152)[0], s[0]) for s in CROSS[:4]] + \
                      [(plan.tree_plan(2, *s[1:4], plan.ceil(max(s[0]), 16) * 16, 152)[0], s[0]) for s in TREES[:2]]:
        units = plan.units_of(p, tiles(lengths))
        assert sum(n for _, n in units.values()) == p.items >= 16 * p.units  # eight warps join a row
        assert any(part == p.room and n == 1 for part, n in units.values())
        assert all(r.stop <= p.room for r in plan.joined(units))


# ------------------------------------------------------------------ the kernels

def table_of(workspace, p, rows, dim):
    """[unit] (first piece, pieces) as the cutting kernel left them."""
    at = p.room * rows * (dim + 1) * 4
    return [tuple(x) for x in workspace[at:at + 8 * p.units].cpu().numpy().view(np.int32).reshape(-1, 2).tolist()]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def exact_workspace(need):
    """A buffer whose first `need` bytes are the workspace; behind it, numbers that would be seen as pieces'."""
    return torch.empty(need // 4 + 1024, dtype=torch.float32, device="cuda").fill_(3e38).view(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CROSS, ids=[str(c[0]) for c in CROSS])
def test_cross_attention(case, debug):
    from online_softmax_05_gb300 import cross as x
    lengths, hq, hkv, rows, dim = case
    B, Tk = len(lengths), max(lengths)
    g = torch.Generator().manual_seed(rows + dim)
    q, k, v = (torch.randn(B, h, t, dim, generator=g).to(torch.bfloat16).cuda()
               for h, t in ((hq, rows), (hkv, Tk), (hkv, Tk)))
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    p, unit_rows = plan.cross_plan(B, hq, hkv, rows, Tk, sms())
    want = reference(q, k, v, lengths)
    stream = torch.cuda.current_stream().cuda_stream
    for lib in (debug, fa.load_library()):
        need = lib.fa_cross_fwd_workspace(B, hq, hkv, rows, Tk, dim)
        assert need == p.room * unit_rows * (dim + 1) * 4 + 8 * p.units
        ws = exact_workspace(need)
        out, lse = torch.empty_like(q), torch.empty(B, hq, rows, device="cuda")
        args = [x._shape(q, k, n)[0]] + [x._packed(t) for t in (q, k, v, out)] + [None, lse.data_ptr(), dim ** -0.5]
        assert lib.fa_cross_fwd(*args, ws.data_ptr(), need, stream) == 0
        assert lib.fa_get_device_status(stream) == 0
        check("o", out, want)
        check("lse", lse, want)
        units = plan.units_of(p, tiles(lengths))
        assert table_of(ws, p, unit_rows, dim) == [units[u] for u in range(p.units)]
        assert (ws[need:].view(torch.float32) == 3e38).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", TREES, ids=[str(c[0]) for c in TREES])
def test_trees(case, debug):
    from online_softmax_05_gb300.kv4 import _cache
    lengths, hq, hkv, n, dim, group = case
    B = len(lengths)
    c = kv4.Batch(lengths, hkv, dim, group, 16, seed=n)
    parents = trees(B, n, seed=n)
    q = c.queries(hq, n)
    pool, table, held = c.on()
    slots = table.shape[1] * 16
    p, unit_rows = plan.tree_plan(B, hq, hkv, n, slots, sms())
    stream = torch.cuda.current_stream().cuda_stream
    qd, pd = q.cuda(), torch.from_numpy(parents).cuda()
    packed = _cache(pool, table, held)[0]
    for lib in (debug, fa.load_library()):
        need = lib.fa_kv4_tree_workspace(B, hq, hkv, n, dim, slots)
        assert need == p.room * unit_rows * (dim + 1) * 4 + 8 * p.units
        ws = exact_workspace(need)
        o, lse = torch.empty_like(qd), torch.empty(B, hq, n, device="cuda")
        assert lib.fa_kv4_tree(packed, qd.data_ptr(), pd.data_ptr(), o.data_ptr(), lse.data_ptr(), hq, n, dim ** -0.5,
                               ws.data_ptr(), need, stream) == 0
        assert lib.fa_get_device_status(stream) == 0
        check_tree(c, q, parents, o, lse)
        units = plan.units_of(p, tiles(lengths))
        assert table_of(ws, p, unit_rows, dim) == [units[u] for u in range(p.units)]
        assert (ws[need:].view(torch.float32) == 3e38).all()
