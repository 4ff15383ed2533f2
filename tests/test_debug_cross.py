"""Cross attention, trees, accepting and keeping through the debug library: no check of a run-time index
fails, and its results are the product library's, bit for bit."""
import ctypes
import os

import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as ref
from tests.test_abi import declared_functions
from tests.test_cross import ints, tensors
from tests.test_kv4_tree import trees


@pytest.fixture
def both(monkeypatch):
    """both(fn): fn()'s results from the product library and from the debug library."""
    from online_softmax_05_gb300 import build
    build.build()
    product = fa.load_library()
    debug = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "libfa_debug.so"))
    for name in declared_functions():
        getattr(debug, name).argtypes = getattr(product, name).argtypes
        getattr(debug, name).restype = getattr(product, name).restype

    def run(fn):
        got = []
        for lib in (product, debug):
            monkeypatch.setattr(fa, "_lib", lib)
            got.append(fn())
            assert fa.fa_get_device_status() == 0
        assert fa.load_library().fa_debug_checks_enabled() == 1
        monkeypatch.setattr(fa, "_lib", product)
        assert len(got[0]) == len(got[1]) and all(torch.equal(a, b) for a, b in zip(*got))
    return run


@pytest.mark.gpu
@pytest.mark.parametrize("shape,lengths", [
    ((1, 2, 1, 1, 1, 64), None), ((2, 4, 2, 5, 129, 128), [0, 129]), ((3, 4, 4, 3, 3000, 64), [3000, 1, 0]),
    ((1, 2, 2, 300, 700, 128), [650]), ((40, 8, 8, 2, 500, 64), list(range(0, 500, 13))[:39] + [500]),
    ((3, 26, 26, 300, 260, 128), [260, 0, 129]), ((2, 30, 15, 700, 200, 64), [200, 130])])
def test_cross_attention(both, shape, lengths, deterministic_backward):
    q, k, v, do = tensors(shape, seed=sum(shape))
    n = ints(lengths)

    def call():
        assert fa.load_library().fa_set_deterministic(1) == 0
        rest = torch.empty_like(q)
        o, lse = fa.attention_forward_cross(q, k, v, n, rest=rest)
        return (o, lse, rest) + fa.attention_backward_cross(q, k, v, o, lse, do, n, rest=rest)
    both(call)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,group,page", [(64, 32, 16), (64, 64, 48), (128, 32, 64), (128, 64, 16)])
@pytest.mark.parametrize("lengths", [[40], [5000, 0, 700], [300] * 25])
def test_trees_and_keeping(both, dim, group, page, lengths):
    n, B = 24, len(lengths)
    c = ref.Batch(lengths, 8, dim, group, page, seed=B)
    q, parents = c.queries(16, n).cuda(), torch.from_numpy(trees(B, n, seed=B)).cuda()
    rng = np.random.default_rng(B)
    tokens, picks = (torch.from_numpy(x).cuda() for x in rng.integers(0, 3, (2, B, n)))

    def call():
        pool, table, held = c.on()
        o, lse = fa.attention_tree_kv4(q, pool, table, held, parents)
        path, counts, follow = fa.tree_accept(parents, tokens, picks)
        new = fa.kv4_keep(pool, table, held, path)
        return o, lse, path, counts, follow, new, pool
    both(call)
