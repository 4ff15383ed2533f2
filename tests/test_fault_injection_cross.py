"""Failure detection of cross attention's few-rows kernel and of the tree kernel, without a GPU fault.

A host-side test hook keeps one tile from the first CTA:
  mode 4  the few-rows kernel's load warp skips its first K tile copy;
  mode 5  the tree kernel's unpacking warps keep their first tile of keys to themselves.
The waits that need it run out after 100 ms, the CTA records FA_ERR_DEVICE_TIMEOUT, drains its copies and
matrix instructions in flight, frees its tensor memory and exits.  The context stays usable: the status word is
cleared by the read, and the same call again, and one with CTAs on every SM, give what they should."""
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as ref
from tests.cross_ref import check, reference
from tests.test_cross import ints, tensors
from tests.test_fault_injection import _inject
from tests.test_kv4_tree import run, trees


@pytest.fixture(scope="module")
def lib():
    from online_softmax_05_gb300 import build
    build.build()
    return fa.load_library()


def timed_out(lib, mode, call):
    assert fa.fa_get_device_status() == 0
    _inject(lib, mode, call)
    assert fa.fa_get_device_status() == -7
    assert fa.fa_get_device_status() == 0   # the status word was cleared


def test_other_modes_are_refused(lib):
    assert lib.fa_debug_inject(6) == -8 and lib.fa_debug_inject(-1) == -8
    assert lib.fa_debug_inject(5) == 0 and lib.fa_debug_inject(0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("B,heads,Tk", [(1, 2, 100), (2, 2, 3000), (40, 8, 700)], ids=["one_tile", "cut", "whole"])
def test_few_rows(lib, B, heads, Tk, dim):
    q, k, v, _ = tensors((B, heads, heads, 5, Tk, dim), seed=B)
    n = ints([Tk - b for b in range(B)])
    timed_out(lib, 4, lambda: fa.attention_forward_cross(q, k, v, n))
    o, lse = fa.attention_forward_cross(q, k, v, n)
    assert fa.fa_get_device_status() == 0
    want = reference(q, k, v, n)
    check("o", o, want)
    check("lse", lse, want)
    q, k, v, _ = tensors((20, 16, 16, 3, 260, dim), seed=1)     # 320 CTAs, two on each SM
    o, lse = fa.attention_forward_cross(q, k, v)
    assert fa.fa_get_device_status() == 0
    check("o", o, reference(q, k, v))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("lengths", [[90], [5000, 700], [300, 1000, 260] * 9], ids=["one_tile", "cut", "whole"])
@pytest.mark.parametrize("wide", [False, True])
def test_trees(lib, lengths, dim, group, wide):
    """wide: keys whose scales leave fp16's range go as two tiles."""
    c = ref.Batch(lengths, 8, dim, group, 16, seed=len(lengths), gain=2.0 ** 20 if wide else 1.0)
    parents = trees(len(lengths), 12, seed=3)
    q, (pool, table, held) = c.queries(16, 12), c.on()
    on = torch.from_numpy(parents).cuda()
    timed_out(lib, 5, lambda: fa.attention_tree_kv4(q.cuda(), pool, table, held, on))
    run(c, 16, parents, std=2.0 ** -20 if wide else 1.0)
    c = ref.Batch([150] * 20, 8, dim, group, 16, seed=2)        # 160 CTAs
    run(c, 16, trees(20, 12, seed=4))
