"""Cross attention by the kernels of whole query tiles: shapes with enough heads that the few-rows kernel is
not taken, tiles that have no partner, sequences of one key tile and of none, more sequences than are sorted;
and what O's rounding took off (`rest`), of both kernels."""
import pytest
import torch

import online_softmax_05_gb300 as fa
from tests.cross_ref import check, reference
from tests.test_cross import ints, tensors


@pytest.fixture(scope="module", autouse=True)
def built():
    from online_softmax_05_gb300 import build
    build.build()


def pairs_of(shape):
    """Items of the kernel of whole tiles; with fewer than half the SMs the few-rows kernel is taken."""
    B, Hq, Hkv, Tq, _, _ = shape
    each = Hq // Hkv
    return B * Hq // 2 * -(-Tq // 128) if each % 2 == 0 else B * Hq * -(-Tq // 256)


WHOLE = [
    ((6, 13, 13, 260, 400, 64), [0, 1, 128, 129, 256, 383]),       # three tiles: the last has no partner
    ((6, 13, 13, 260, 400, 128), [127, 255, 257, 384, 385, 400]),
    ((6, 13, 13, 384, 128, 128), None),                            # one key tile: half of a split item has none
    ((4, 12, 4, 513, 130, 64), [130, 0, 1, 129]),                  # odd groups, five tiles
    ((3, 36, 12, 257, 300, 128), [300, 77, 256]),
    ((2, 26, 13, 700, 200, 128), [200, 130]),                      # even groups: pairs of heads
    ((1, 80, 80, 129, 513, 64), [500]),
    ((256, 1, 1, 258, 140, 64), "many"),                           # as many sequences as are sorted
    ((257, 1, 1, 258, 140, 128), "many"),                          # and one more
]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["plain", "fused"])
@pytest.mark.parametrize("shape,lengths", WHOLE, ids=[str(s) for s, _ in WHOLE])
def test_forward_and_backward(shape, lengths, layout):
    B, Hq, Hkv, Tq, Tk, _ = shape
    assert 2 * pairs_of(shape) > 152 and Hq // Hkv * Tq > 128
    if lengths == "many":
        lengths = [(37 * b + 5) % (Tk + 1) for b in range(B)]
    q, k, v, do = tensors(shape, layout, seed=sum(shape))
    n = ints(lengths)
    rest = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_forward_cross(q, k, v, n, rest=rest)
    assert (rest.abs() <= 2.0 ** -8 * o.abs()).all()
    dq, dk, dv = fa.attention_backward_cross(q, k, v, o, lse, do, n, rest=rest)
    assert fa.fa_get_device_status() == 0
    ref = reference(q, k, v, lengths, do=do)
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got, ref)
    for b, length in enumerate(lengths or []):
        assert not dk[b, :, length:].any() and not dv[b, :, length:].any()
        if length == 0:
            assert not o[b].any() and not rest[b].any() and not dq[b].any() and (lse[b] == -torch.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape,lengths", [
    ((3, 26, 13, 300, 700, 64), [700, 130, 401]),      # pairs of heads
    ((3, 26, 26, 300, 700, 128), [700, 130, 401]),     # pairs of tiles and lone ones
    ((3, 26, 26, 500, 400, 64), None),
    ((2, 4, 2, 3, 9000, 128), [9000, 300]),            # few rows, cut and joined
    ((2, 2, 2, 2, 9000, 64), [9000, 300]),             # joined by eight warps a row
    ((64, 4, 4, 5, 400, 64), None),                    # few rows, nothing cut
])
def test_the_rest_is_what_rounding_took_off(shape, lengths):
    """Values around 1: rounding O takes off 2^-9 / sqrt(3) of 1 or so, evenly spread.  P's own roundings, of weights
    between 0.5 and 1, are as large and as evenly spread, but n of them are averaged: they leave 1 / sqrt(n)
    of that, at most 0.09 here, and the rest's rounding 2^-8.  A quarter is three times as much.  The gradient
    of the queries goes by D, whose error is O's times the mean of the keys, 1."""
    q, k, v, do = tensors(shape, seed=sum(shape))
    q, k, v = q * 0.3, (k * 0.3 + 1.0).to(torch.bfloat16), (v * 0.05 + 1.0).to(torch.bfloat16)
    n = ints(lengths)
    plain, lse = fa.attention_forward_cross(q, k, v, n)
    rest = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse2 = fa.attention_forward_cross(q, k, v, n, rest=rest)
    assert torch.equal(o, plain) and torch.equal(lse, lse2)
    ref = reference(q, k, v, lengths, do=do)
    exact = ref["o"][0].cuda()
    for b in range(shape[0]):
        for h in range(shape[1]):
            left = (o[b, h].double() + rest[b, h].double() - exact[b, h]).norm()
            assert left < 0.25 * (o[b, h].double() - exact[b, h]).norm(), (b, h)
    off = []
    for r in (None, rest):
        dq, dk, dv = fa.attention_backward_cross(q, k, v, o, lse, do, n, rest=r)
        for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
            check(name, got, ref)
        off.append((dq.double().cpu() - ref["dq"][0]).norm())
    assert off[1] < 0.5 * off[0]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 4, 2, 5, 3000, 64), (3, 26, 26, 300, 500, 128)])
def test_captured_with_the_librarys_own_workspaces(shape):
    """Workspaces that the library takes inside a capture are the graph's: two graphs replayed in turn."""
    from online_softmax_05_gb300 import cross as x
    lib = fa.load_library()
    B, Hq, Hkv, Tq, Tk, D = shape
    q, k, v, do = tensors(shape, seed=3)
    lengths = [Tk - 7 * b for b in range(B)]
    n = ints(lengths)
    o, lse = fa.attention_forward_cross(q, k, v, n)
    want = (o, lse) + fa.attention_backward_cross(q, k, v, o, lse, do, n)
    graphs, outs = [], []
    for _ in range(2):
        out = [torch.empty_like(t) for t in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            stream = torch.cuda.current_stream().cuda_stream
            packed = x._shape(q, k, n)[0]
            p = [x._packed(t) for t in (q, k, v, out[0], do, *out[2:])]
            assert lib.fa_cross_fwd(packed, *p[:4], None, out[1].data_ptr(), D ** -0.5, None, 0, stream) == 0
            assert lib.fa_cross_bwd(packed, *p[:4], None, p[4], out[1].data_ptr(), *p[5:], D ** -0.5, None, 0, stream) == 0
        graphs.append(graph)
        outs.append(out)
    for _ in range(2):
        for graph, out in zip(graphs, outs):
            for t in out:
                t.fill_(3.0)
            graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
