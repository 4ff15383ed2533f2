"""How ragged batches are cut over CTAs: extremes of the lengths, many sequences, long next to
short, through the operators that are cut this way."""
import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests import kv4_ref as ref
from tests.cross_ref import check, reference
from tests.test_kv4_tree import run, trees


@pytest.fixture(scope="module", autouse=True)
def built():
    from online_softmax_05_gb300 import build
    build.build()


def cross(lengths, heads, rows, Tk, seed, dim=64):
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    q, k, v = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
               for s in ((B, heads, rows, dim), (B, heads, Tk, dim), (B, heads, Tk, dim)))
    o, lse = fa.attention_forward_cross(q, k, v, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert fa.fa_get_device_status() == 0
    want = reference(q, k, v, lengths)
    check("o", o, want)
    check("lse", lse, want)
    return q, k, v, o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("heads,rows", [(1, 1), (3, 5), (1, 128), (2, 130)])
@pytest.mark.parametrize("lengths", [
    [4000], [0], [1], [128], [129],
    [0] * 31 + [4000], [1] * 32, list(range(0, 4000, 130)),      # up to 32 sequences: sorted
    [1] * 32 + [4000], [0] * 40, list(range(3000, 3000 + 33)),   # more
    [5] * 127 + [3999], [5] * 128 + [3999], [0] * 200,           # the chunk is searched for up to 128
    [3] * 511 + [900], [3] * 512 + [900],                        # cut up to 512
])
def test_lengths(lengths, heads, rows):
    cross(lengths, heads, rows, 4000, seed=len(lengths) + heads)


@pytest.mark.gpu
@pytest.mark.parametrize("count", [1, 20, 33, 150])
def test_many_heads_and_one_long_sequence(count):
    """Many units: only the long one is cut, whatever its place."""
    rng = np.random.default_rng(count)
    lengths = rng.integers(0, 200, count).tolist()
    lengths[count // 2] = 9000
    cross(lengths, 12, 3, 9000, seed=count)


@pytest.mark.gpu
@pytest.mark.parametrize("count,heads,n", [(1, 1, 3), (1, 1, 64), (40, 2, 5), (150, 1, 2), (70, 4, 9)])
def test_trees(count, heads, n):
    rng = np.random.default_rng(count)
    lengths = (rng.integers(0, 2, count) * rng.integers(n, 300, count)).tolist()
    lengths[count // 3] = 5000
    c = ref.Batch(lengths, heads, 64, 32, 16, seed=count)
    run(c, 2 * heads, trees(count, n, seed=count))


@pytest.mark.gpu
def test_pieces_are_joined_alike_at_any_cut():
    """A sequence's result does not go by the batch that it lies in, up to the cut's rounding: O
    to bf16's step, the log-sum-exp to fp32's sums."""
    q, k, v, o, lse = cross([3000] + [700] * 9, 2, 4, 3000, seed=5)
    one, l1 = fa.attention_forward_cross(q[:1].contiguous(), k[:1].contiguous(), v[:1].contiguous())
    assert (one.float() - o[:1].float()).abs().max() <= 2.0 ** -6 * o[:1].float().abs().max()
    assert (l1 - lse[:1]).abs().max() <= 1e-5


@pytest.mark.gpu
def test_a_workspace_of_exactly_the_size_asked_for():
    """Nothing behind it is written: the library's own call with a workspace inside a larger buffer."""
    from online_softmax_05_gb300 import cross as x
    lib = fa.load_library()
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
               for s in ((3, 4, 5, 64), (3, 2, 2500, 64), (3, 2, 2500, 64)))
    n = torch.tensor([2500, 0, 1300], dtype=torch.int32, device="cuda")
    want, _ = fa.attention_forward_cross(q, k, v, n)
    need = lib.fa_cross_fwd_workspace(3, 4, 2, 5, 2500, 64)
    assert need > 0
    buffer = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 4, 5, device="cuda")
    packed, _, _, _ = x._shape(q, k, n)
    args = [packed] + [x._packed(t) for t in (q, k, v, out)] + [None, lse.data_ptr(), 64 ** -0.5]
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.fa_cross_fwd(*args, buffer.data_ptr(), need - 1, stream) == -10
    assert lib.fa_cross_fwd(*args, buffer.data_ptr() + 4, need, stream) == -4
    assert lib.fa_cross_fwd(*args, buffer.data_ptr(), need, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (buffer[need:] == 77).all()
    assert lib.fa_cross_fwd(*args, None, 0, stream) == 0  # taken by the library
    torch.cuda.synchronize()
    assert torch.equal(out, want)
