"""cross_attention copies what the kernels cannot take as it lies: views off 16-byte alignment, odd strides."""
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests.cross_ref import check, reference
from tests.test_cross import ints, tensors


def off_alignment(x, by=1):
    """A contiguous copy of x, `by` elements into its buffer."""
    buffer = torch.empty(x.numel() + 8, dtype=x.dtype, device=x.device)
    view = buffer[by:by + x.numel()].view(x.shape)
    view.copy_(x)
    return view


def odd_rows(x):
    """x with rows D + 1 elements apart."""
    wide = torch.empty(*x.shape[:-1], x.shape[-1] + 1, dtype=x.dtype, device=x.device)
    wide[..., :-1] = x
    return wide[..., :-1]


@pytest.mark.parametrize("shape", [(2, 3, 5, 64), (1, 1, 1, 64), (2, 5, 64)])
def test_a_copy_fits(shape):
    from online_softmax_05_gb300.cross import _fits, _laid_out
    x = torch.randn(shape).to(torch.bfloat16)
    four = x.unsqueeze(1) if x.dim() == 3 else x
    for y in (off_alignment(x), off_alignment(x, 7), odd_rows(off_alignment(x)), x[:1].expand(shape)):
        got = _laid_out(y, "x")
        assert _fits(got) and torch.equal(got, y.unsqueeze(1) if y.dim() == 3 else y)
    assert _laid_out(four, "x") is four                       # what fits is taken as it lies


@pytest.mark.gpu
@pytest.mark.parametrize("change", [off_alignment, odd_rows])
@pytest.mark.parametrize("rows", [3, 130])
def test_values_and_gradients(rows, change):
    q, k, v, do = tensors((2, 4, 2, rows, 150, 64), seed=rows)
    n = ints([150, 33])
    leaves = [change(x).detach().requires_grad_() for x in (q, k, v)]
    o = fa.cross_attention(*leaves, n)
    grads = torch.autograd.grad(o, leaves, change(do))
    ref = reference(q, k, v, [150, 33], do=do)
    for name, got in zip(("o", "dq", "dk", "dv"), (o, *grads)):
        check(name, got, ref)
    with pytest.raises(ValueError):                           # the call that takes tensors as they lie
        fa.attention_forward_cross(leaves[0].detach(), k, v, n)
