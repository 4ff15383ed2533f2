"""The largest numbers of keys: windows of one buffer may overlap, so that 2^31 of them fit the memory."""
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests.test_cross import NO_DEVICE, backward, forward, shape_of, view


@pytest.fixture(scope="module", autouse=True)
def built():
    from online_softmax_05_gb300 import build
    build.build()


def test_keys_that_do_not_round_up_to_tiles_are_refused():
    if torch.cuda.is_available():
        pytest.skip("good arguments would launch on made-up addresses")
    last = (1 << 31) - 128
    windows = dict(k=view(1 << 40, t=8), v=view(1 << 41, t=8))
    assert forward(shape=shape_of(1, 1, 1, 3, last), **windows) in NO_DEVICE
    for n in (last + 1, (1 << 31) - 1):
        assert forward(shape=shape_of(1, 1, 1, 3, n), **windows) == -2
        assert backward(shape=shape_of(1, 1, 1, 3, n), **windows) == -2
    # the limit is one of a sequence's keys
    assert forward(shape=shape_of(2, 1, 1, 3, (1 << 30) - 1), **windows) in NO_DEVICE
    lib = fa.load_library()
    for query in (lib.fa_cross_fwd_workspace, lib.fa_cross_bwd_workspace):
        assert query(1, 1, 1, 3, last, 64) in NO_DEVICE and query(1, 1, 1, 3, last + 1, 64) == -2


@pytest.mark.gpu
def test_the_most_keys():
    """2^31 - 128 keys, 8 elements apart: the last of them takes all the weight, or (scale 0) each the same."""
    n = (1 << 31) - 128
    size = 8 * (n - 1) + 64
    k, v = (torch.zeros(size, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[-64:] = 1.0
    v[-64:] = torch.arange(64, device="cuda") - 32.0
    keys, values = (torch.as_strided(x, (1, 1, n, 64), (size, size, 8, 1)) for x in (k, v))
    # scores of the last keys: 320, 280, 240 and so on, as windows share the ones
    q = torch.full((1, 1, 2, 64), 40.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_forward_cross(q, keys, values)
    assert fa.fa_get_device_status() == 0
    # the others' weights are e^-40, e^-80 and so on, of values up to 32: 64 e^-40 < 2^-51 off, and the rest exact
    assert (o.double() - v[-64:].double()).abs().max() <= 2.0 ** -51
    assert (lse - 320.0).abs().max() <= 320 * 2.0 ** -20
    o, lse = fa.attention_forward_cross(q, keys, values, scale=0.0)
    assert fa.fa_get_device_status() == 0
    assert o.abs().max() <= 2.0 ** -20
    assert (lse.double() - torch.tensor(n).double().log()).abs().max() <= 22 * 2.0 ** -20
    del k, v, keys, values
    torch.cuda.empty_cache()  # 69 GB that no other test wants
