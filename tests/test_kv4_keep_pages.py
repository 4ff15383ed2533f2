"""Keeping a path some of whose pages the table does not name: what is left out is left out as a whole, the
codes of a place together with its accounts."""
import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as ref
from tests.test_kv4_keep import copy_token


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_05_gb300 import build
    build.build()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("page_at,left_out", [(3, [1, 2]), (2, [0, 1, 2])])
def test_a_place_without_a_page_keeps_its_accounts(page_at, left_out, bad):
    """Slots 44 to 51 hold the tree, pages 16: the path's places 2, 4 and 7 lie in slots 46, 48 and 51."""
    c = ref.Batch([40, 52], 2, 64, 32, 16, seed=4)
    path = [2, 4, 7, -1, -1, -1, -1, -1]
    rng = np.random.default_rng(4)
    weights = rng.random((2, 2, 64)).astype(np.float32)
    where = rng.integers(0, 1 << 20, (2, 2, 64)).astype(np.int32)
    pool, table, held = c.on()
    table[1, page_at] = bad
    w, p = torch.from_numpy(weights).cuda(), torch.from_numpy(where).cuda()
    new = fa.kv4_keep(pool, table, held, torch.tensor([path, path], dtype=torch.int32, device="cuda"), weights=w,
                      slot_positions=p)
    assert fa.fa_get_device_status() == -13
    assert new.tolist() == [35, 47]
    want, want_w, want_p = c.pool.copy(), weights.copy(), where.copy()
    for b, n in ((0, 40), (1, 52)):
        for i, j in enumerate(path[:3]):
            if b == 1 and i in left_out:
                continue
            copy_token(c, want, b, n - 8 + j, n - 8 + i)
            want_w[b, :, n - 8 + i] = weights[b, :, n - 8 + j]
            want_p[b, :, n - 8 + i] = where[b, :, n - 8 + j]
    assert np.array_equal(pool.cpu().numpy(), want)
    assert np.array_equal(w.cpu().numpy(), want_w) and np.array_equal(p.cpu().numpy(), want_p)
