"""Cross attention: queries of one sequence over the keys of another, forward and
backward, against the definition in 64 bits; lengths, layouts, refusals."""
import struct
import threading

import pytest
import torch

import online_softmax_05_gb300 as fa

from tests.cross_ref import check, reference


@pytest.fixture(scope="module", autouse=True)
def built():
    from online_softmax_05_gb300 import build
    build.build()


def tensors(shape, layout="plain", seed=0, device="cuda", qk=1.0):
    """q, k, v, do of (B, Hq, Hkv, Tq, Tk, D) in bf16."""
    B, Hq, Hkv, Tq, Tk, D = shape
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    if layout == "plain":
        q, k, v = normal(B, Hq, Tq, D) * qk, normal(B, Hkv, Tk, D) * qk, normal(B, Hkv, Tk, D)
        q, k, v = (x.to(torch.bfloat16).to(device) for x in (q, k, v))
    elif layout == "tokens":  # heads behind tokens
        q, k, v = (normal(B, n, h, D).to(torch.bfloat16).to(device).transpose(1, 2)
                   for n, h in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv)))
    else:  # keys and values side by side behind tokens, queries between others' channels, sequences innermost but one
        q = normal(Tq, B, Hq, 3 * D).to(torch.bfloat16).to(device)[..., D:2 * D].permute(1, 2, 0, 3)
        kv = normal(B, Tk, 2, Hkv, D).to(torch.bfloat16).to(device).permute(2, 0, 3, 1, 4)
        k, v = kv[0], kv[1]
    do = normal(B, Hq, Tq, D).to(torch.bfloat16).to(device)
    return q, k, v, do


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


SHAPES = [
    ((1, 1, 1, 1, 1, 64), None),
    ((1, 2, 1, 1, 2, 128), [1]),
    ((2, 4, 2, 5, 129, 64), [0, 129]),
    ((3, 2, 2, 130, 300, 128), [1, 300, 128]),
    ((2, 8, 1, 257, 127, 128), [127, 64]),
    ((1, 3, 1, 127, 257, 64), None),
    ((2, 2, 2, 300, 1, 128), None),
    ((4, 6, 2, 33, 515, 64), [0, 513, 512, 1]),
    ((2, 16, 4, 1, 1000, 128), [1000, 257]),
    ((3, 32, 8, 9, 700, 64), [699, 3, 385]),
    ((1, 7, 1, 64, 4096, 128), None),
    ((2, 20, 20, 129, 513, 128), [513, 384]),      # enough items for pairs of query tiles
    ((4, 10, 10, 200, 513, 64), [513, 0, 200, 384]),  # dq summed in place
    ((2, 64, 32, 260, 400, 64), [130, 400]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["plain", "tokens", "fused"])
@pytest.mark.parametrize("shape,lengths", SHAPES)
def test_forward_and_backward(shape, lengths, layout):
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
            assert not o[b].any() and not dq[b].any() and (lse[b] == -torch.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
@pytest.mark.parametrize("rows", [3, 200])
def test_scales(scale, rows):
    q, k, v, do = tensors((2, 2, 2, rows, 211, 64), seed=4)
    o, lse = fa.attention_forward_cross(q, k, v, ints([211, 40]), scale=scale)
    grads = fa.attention_backward_cross(q, k, v, o, lse, do, ints([211, 40]), scale=scale)
    ref = reference(q, k, v, [211, 40], scale=scale, do=do)
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        check(name, got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads,dim", [(1, 2, 64), (40, 2, 128), (300, 2, 64), (300, 20, 128), (200, 40, 64)])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3.3895313892515355e38])
def test_what_lies_past_a_length_is_not_used(rows, heads, dim, junk):
    lengths = [300, 129, 0, 1, 256]
    q, k, v, do = tensors((5, heads, heads, rows, 300, dim), seed=8)
    n = ints(lengths)
    for b, length in enumerate(lengths):
        k[b, :, length:] = 0
        v[b, :, length:] = 0
    o, lse = fa.attention_forward_cross(q, k, v, n)
    want = (o, lse) + fa.attention_backward_cross(q, k, v, o, lse, do, n)
    for b, length in enumerate(lengths):
        k[b, :, length:] = junk
        v[b, :, length:] = junk
    o, lse = fa.attention_forward_cross(q, k, v, n)
    got = (o, lse) + fa.attention_backward_cross(q, k, v, o, lse, do, n)
    fused = fa.load_library().fa_bwd_sums_dq_in_place(5, heads, 300, dim)  # dq's sums vary in their order
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), got, want):
        if name == "dq" and fused:
            assert torch.isfinite(a).all() and (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
        else:
            assert torch.equal(a, b), name


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 150])
def test_a_nan_query_stays_in_its_row(rows):
    q, k, v, _ = tensors((1, 2, 1, rows, 200, 64), seed=9)
    o, lse = fa.attention_forward_cross(q, k, v)
    q[0, 1, 1, 5] = float("nan")
    o2, lse2 = fa.attention_forward_cross(q, k, v)
    assert o2[0, 1, 1].isnan().all() and lse2[0, 1, 1].isnan()
    o2[0, 1, 1], lse2[0, 1, 1] = o[0, 1, 1], lse[0, 1, 1]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 70, 140])
def test_large_scores(rows):
    """Scores of hundreds: one key takes all, and nothing overflows."""
    q, k, v, do = tensors((1, 2, 2, rows, 300, 128), seed=10, qk=6.0)
    o, lse = fa.attention_forward_cross(q, k, v)
    grads = fa.attention_backward_cross(q, k, v, o, lse, do)
    ref = reference(q, k, v, do=do)
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        check(name, got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [4, 260])
def test_given_outputs_and_what_lies_around_them(rows):
    shape = (2, 4, 2, rows, 130, 64)
    q, k, v, do = tensors(shape, seed=11)
    n = ints([77, 0])
    o, lse = fa.attention_forward_cross(q, k, v, n)
    grads = fa.attention_backward_cross(q, k, v, o, lse, do, n)

    def hole(like):  # a tensor inside a larger one, tokens, heads and channels around it
        B, H, T, D = like.shape
        whole = torch.full((B, T + 3, H + 1, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[:, 1:T + 1, :H, :D].transpose(1, 2)

    whole, out = hole(o)
    o2, _ = fa.attention_forward_cross(q, k, v, n, out=out, lse=torch.empty_like(lse))
    assert o2 is out and torch.equal(o2, o)
    out.fill_(7.0)
    assert (whole == 7.0).all()
    holes = [hole(g) for g in grads]
    fa.attention_backward_cross(q, k, v, o, lse, do, n, dq=holes[0][1], dk=holes[1][1], dv=holes[2][1])
    for (whole, out), g in zip(holes, grads):
        assert torch.equal(out, g)
        out.fill_(7.0)
        assert (whole == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 140])
def test_bad_lengths_are_recorded_and_count_as_none(rows):
    q, k, v, do = tensors((3, 2, 2, rows, 150, 64), seed=12)
    o, lse = fa.attention_forward_cross(q, k, v, ints([151, -1, 150]))
    assert fa.fa_get_device_status() == -11
    assert not o[:2].any() and (lse[:2] == -torch.inf).all()
    dq, dk, dv = fa.attention_backward_cross(q, k, v, o, lse, do, ints([151, -1, 150]))
    assert fa.fa_get_device_status() == -11
    assert not dq[:2].any() and not dk[:2].any() and not dv[:2].any()
    want, _ = fa.attention_forward_cross(q[2:], k[2:], v[2:])
    assert torch.equal(o[2:], want)


@pytest.mark.gpu
def test_autograd():
    """Gradients through cross_attention: grouped heads, lengths, layouts, broadcasts."""
    q, k, v, do = tensors((2, 6, 2, 70, 190, 64), "tokens", seed=13)
    n = ints([190, 101])
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = fa.cross_attention(*leaves, n)
    assert o.stride() == q.stride()
    grads = torch.autograd.grad(o, leaves, do)
    ref = reference(q, k, v, [190, 101], do=do)
    for name, got in zip(("o", "dq", "dk", "dv"), (o, *grads)):
        check(name, got, ref)
    # one source for a batch of two: its gradients are summed, from a gradient without strides
    k1, v1 = (x[:1].detach().contiguous().requires_grad_() for x in (k, v))
    o = fa.cross_attention(leaves[0], k1.expand(2, -1, -1, -1), v1.expand(2, -1, -1, -1))
    dk1, dv1 = torch.autograd.grad(o.float().sum(), (k1, v1))
    ref = reference(q, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1), do=torch.ones_like(q))
    for got, name in ((dk1, "dk"), (dv1, "dv")):
        value, bound = ref[name]
        value, bound = value.sum(0, keepdim=True), bound.sum(0, keepdim=True)
        bound = bound + 2.0 ** -8 * (value.abs() + bound)  # the sum is rounded again
        assert ((got.double().cpu() - value).abs() <= bound).all()
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(fa.cross_attention(*leaves).float().square().sum(), leaves[0], create_graph=True)
        g.sum().backward()


@pytest.mark.gpu
def test_the_rest_makes_dq_exact_where_keys_have_a_mean():
    """An error of D reaches dQ times the weighted mean of the keys, here 20 times their spread.  O's
    rounding is off by 2^-9 of 1 or so, which the rest removes but for P's own rounding, averaged over
    400 keys: 2^-9 / 20."""
    q, k, v, do = tensors((1, 2, 2, 150, 400, 64), seed=20)
    q = q * 0.1
    k, v = ((x * 0.05 + 1.0).to(torch.bfloat16) for x in (k, v))
    o0, lse = fa.attention_forward_cross(q, k, v)
    rest = torch.empty_like(q)
    o, _ = fa.attention_forward_cross(q, k, v, rest=rest)
    assert torch.equal(o, o0)
    ref = reference(q, k, v, do=do)
    exact = ref["o"][0].cuda()
    assert ((o.double() + rest.double() - exact).norm() < 0.2 * (o.double() - exact).norm())
    off = [(fa.attention_backward_cross(q, k, v, o, lse, do, rest=r)[0].double().cpu() - ref["dq"][0]).norm()
           for r in (None, rest)]
    assert off[1] < 0.5 * off[0]


@pytest.mark.gpu
def test_gradients_against_differences():
    """The loss along the gradients' own direction: its difference is their squared length."""
    q, k, v, do = tensors((2, 2, 1, 40, 90, 64), seed=14)
    lengths = [90, 33]
    o, lse = fa.attention_forward_cross(q, k, v, ints(lengths))
    grads = [g.double().cpu() for g in fa.attention_backward_cross(q, k, v, o, lse, do, ints(lengths))]

    def loss(step):
        x = [t.double().cpu() + step * g for t, g in zip((q, k, v), grads)]
        return (reference(*x, lengths)["o"][0] * do.double().cpu()).sum()

    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    # central differences are off by h^2; each gradient by 3 U of its norm at most (rounded P or dS, D, the result)
    length = sum((g ** 2).sum() for g in grads)
    assert abs(slope - length) <= 3 * 2.0 ** -8 * length


@pytest.mark.gpu
def test_one_head_form():
    q, k, v, do = tensors((2, 1, 1, 50, 80, 64), seed=15)
    a = [x[:, 0].detach().requires_grad_() for x in (q, k, v)]
    b = [x.detach().requires_grad_() for x in (q, k, v)]
    oa, ob = fa.cross_attention(*a), fa.cross_attention(*b)
    assert torch.equal(oa, ob[:, 0])
    for x, y in zip(torch.autograd.grad(oa, a, do[:, 0]), torch.autograd.grad(ob, b, do)):
        assert torch.equal(x, y[:, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("heads,same", [(4, False), (40, True)])
def test_equals_plain_attention_where_both_apply(heads, same):
    """As many queries as keys, all there: what the other entry points give, bitwise where the
    same forward kernel runs (with few heads this one cuts the keys)."""
    q, k, v, do = tensors((2, heads, heads // 2, 300, 300, 128), seed=16)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    stream, shape = torch.cuda.current_stream(), (2, heads, heads // 2, 300, 128)
    assert fa.fa_fwd_gqa(q, k, v, o, lse, *shape, 128 ** -0.5, 0, stream) == 0
    grads = [torch.empty_like(x) for x in (q, k, v)]
    assert fa.fa_bwd_gqa(q, k, v, o, do, lse, *grads, *shape, 128 ** -0.5, 0, stream) == 0
    o2, lse2 = fa.attention_forward_cross(q, k, v)
    grads2 = fa.attention_backward_cross(q, k, v, o2, lse2, do)
    ref = None if same else reference(q, k, v, do=do)
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads), (o2, lse2, *grads2)):
        if same:
            assert torch.equal(a, b), name
        else:
            check(name, a, ref)
            check(name, b, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads", [(2, 4), (300, 20)])
def test_streams_and_graphs(rows, heads):
    q, k, v, do = tensors((2, heads, heads, rows, 260, 128), seed=17)
    n = ints([260, 100])
    o, lse = fa.attention_forward_cross(q, k, v, n)
    want = (o, lse) + fa.attention_backward_cross(q, k, v, o, lse, do, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = fa.attention_forward_cross(q, k, v, n, stream=side)
    got = (o2, lse2) + fa.attention_backward_cross(q, k, v, o2, lse2, do, n, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = fa.attention_forward_cross(q, k, v, n)
        held = (o3, lse3) + fa.attention_backward_cross(q, k, v, o3, lse3, do, n)
    for lengths in ([260, 100], [0, 259]):
        n.copy_(ints(lengths))
        graph.replay()
        o, lse = fa.attention_forward_cross(q, k, v, n)
        want = (o, lse) + fa.attention_backward_cross(q, k, v, o, lse, do, n)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads,dim", [(3, 2, 128), (300, 20, 64), (300, 20, 128)])
def test_strides_beyond_32_bits(rows, heads, dim, deterministic_backward):
    """Sequences 2^31 + 64 elements apart, inputs and outputs; the results are those of tensors side by side."""
    q, k, v, do = tensors((2, heads, heads, rows, 260, dim), seed=19)
    n = ints([260, 131])
    far = (1 << 31) + 64

    def apart(*given):
        """Copies of tensors, in one buffer one behind the other, their sequences far apart."""
        sizes = [x[0].numel() for x in given]
        assert sum(sizes) <= 1 << 22
        buffer = torch.empty(far + (1 << 22), dtype=torch.bfloat16, device="cuda")
        out, at = [], 0
        for x, size in zip(given, sizes):
            _, h, t, d = x.shape
            out.append(torch.as_strided(buffer, x.shape, (far, t * d, d, 1), at))
            out[-1].copy_(x)
            at += size
        return out

    o, lse = fa.attention_forward_cross(q, k, v, n)
    grads = fa.attention_backward_cross(q, k, v, o, lse, do, n)
    q2, k2, v2, do2 = apart(q, k, v, do)
    o2, lse2 = fa.attention_forward_cross(q2, k2, v2, n, out=apart(torch.zeros_like(q))[0])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    outs = [apart(torch.zeros_like(x))[0] for x in (q, k, v)]
    fa.attention_backward_cross(q2, k2, v2, o2, lse2, do2, n, dq=outs[0], dk=outs[1], dv=outs[2])
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads", [(2, 4), (300, 20)])
def test_a_captured_training_pass(rows, heads):
    """Forward and backward under autograd in one graph; the graphs of the passes before are gone by then."""
    q, k, v, do = tensors((2, heads, heads, rows, 260, 128), seed=18)
    n = ints([260, 100])
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]

    def step():
        o = fa.cross_attention(*leaves, n)
        return (o.detach(),) + torch.autograd.grad(o, leaves, do)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for lengths, gain in (([260, 100], 1.0), ([0, 259], 0.5)):
        n.copy_(ints(lengths))
        with torch.no_grad():
            leaves[0].copy_(q * gain)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 200])
def test_calls_from_a_thread_that_has_used_no_gpu(rows):
    """Tensor maps are made in a thread whose first call this is."""
    q, k, v, do = tensors((1, 2, 2, rows, 130, 64), seed=19)
    o, lse = fa.attention_forward_cross(q, k, v)
    want = (o, lse) + fa.attention_backward_cross(q, k, v, o, lse, do)
    plain = fa.attention_forward(q, q, q)
    outs = [torch.empty_like(x) for x in want + plain]
    torch.cuda.synchronize()
    main, failed = torch.cuda.current_stream(), []

    def call(fn, *args, **given):
        try:
            fn(*args, stream=main, **given)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    for fn, args, given in ((fa.attention_forward_cross, (q, k, v), dict(out=outs[0], lse=outs[1])),
                            (fa.attention_backward_cross, (q, k, v, o, lse, do), dict(dq=outs[2], dk=outs[3], dv=outs[4])),
                            (fa.attention_forward, (q, q, q), dict(out=outs[5], lse=outs[6]))):
        thread = threading.Thread(target=call, args=(fn, *args), kwargs=given)
        thread.start()
        thread.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(torch.equal(a, b) for a, b in zip(outs, want + plain))


@pytest.mark.gpu
def test_two_calls_at_once():
    q, k, v, do = tensors((3, 8, 8, 200, 400, 64), seed=18)
    streams = [torch.cuda.Stream() for _ in range(3)]
    want = []
    for b in range(3):
        o, lse = fa.attention_forward_cross(q[b:b + 1], k[b:b + 1], v[b:b + 1])
        want.append((o, lse) + fa.attention_backward_cross(q[b:b + 1], k[b:b + 1], v[b:b + 1], o, lse, do[b:b + 1]))
    torch.cuda.synchronize()
    got = [None] * 3
    for _ in range(3):
        for b, s in enumerate(streams):
            x = q[b:b + 1], k[b:b + 1], v[b:b + 1]
            o, lse = fa.attention_forward_cross(*x, stream=s)
            got[b] = (o, lse) + fa.attention_backward_cross(*x, o, lse, do[b:b + 1], stream=s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


# ------------------------------------------------------------------ refusals (no GPU)

def shape_of(B=2, Hq=4, Hkv=2, Tq=3, Tk=5, D=64, lengths=0):
    return struct.pack("6iQ", B, Hq, Hkv, Tq, Tk, D, lengths)


def view(at, b=4096, h=512, t=64):
    return struct.pack("Q3q", at, b, h, t)


BASE = 1 << 20


def forward(shape=None, q=None, k=None, v=None, o=None, lse=BASE * 9, scale=0.1, rest=None):
    lib = fa.load_library()
    return lib.fa_cross_fwd(shape or shape_of(), q or view(BASE), k or view(2 * BASE), v or view(3 * BASE),
                            o or view(4 * BASE), rest, lse, scale, None, 0, None)


def backward(shape=None, scale=0.1, lse=BASE * 9, workspace=None, size=0, rest=None, **x):
    lib = fa.load_library()
    at = {n: x.get(n) or view((i + 1) * BASE) for i, n in enumerate(("q", "k", "v", "o", "do", "dq", "dk", "dv"))}
    return lib.fa_cross_bwd(shape or shape_of(), at["q"], at["k"], at["v"], at["o"], rest, at["do"], lse, at["dq"], at["dk"],
                            at["dv"], scale, workspace, size, None)


NO_DEVICE = (-5, -9)  # every argument was good: the device is looked for next


def test_refusals_of_the_c_abi():
    if torch.cuda.is_available():
        pytest.skip("good arguments would launch on made-up addresses")
    assert forward() in NO_DEVICE and backward() in NO_DEVICE
    for call in (forward, backward):
        assert call(lse=None) == -1
        assert call(q=view(0)) == -1
        assert call(shape=shape_of(Hq=3)) == -2
        for name in ("B", "Hq", "Hkv", "Tq", "Tk"):
            assert call(shape=shape_of(**{name: 0})) == -2
            assert call(shape=shape_of(**{name: -4})) == -2
        assert call(shape=shape_of(Tq=1 << 30)) == -2
        assert call(shape=shape_of(Tk=1 << 30)) == -2
        assert call(shape=shape_of(D=96)) == -3
        assert call(scale=float("inf")) == -8
        assert call(scale=float("nan")) == -8
        assert call(lse=BASE * 9 + 4) == -4
        assert call(shape=shape_of(lengths=BASE * 11 + 2)) == -4
        assert call(k=view(2 * BASE + 8)) == -4
        assert call(k=view(2 * BASE, t=68)) == -4          # no multiple of 8
        assert call(k=view(2 * BASE, h=0)) == -8           # a broadcast
        assert call(v=view(3 * BASE, t=-64)) == -8
        assert call(v=view(3 * BASE, b=1 << 38)) == -2
        assert call(o=view(BASE)) == (-8 if call is forward else call())
    assert forward(rest=10 * BASE + 8) == -4 and backward(rest=10 * BASE + 8) == -4
    assert forward(rest=4 * BASE) == -8 and forward(rest=BASE) == -8 and backward(rest=8 * BASE) == -8
    assert forward(o=view(4 * BASE, b=64)) == -8           # rows that share elements
    assert forward(o=view(2 * BASE)) == -8
    assert forward(lse=BASE + 64) == -8
    assert forward(shape=shape_of(lengths=4 * BASE)) == -8
    assert backward(dk=view(8 * BASE + 1024)) == -8        # dk inside dv
    assert backward(dq=view(BASE)) == -8
    assert backward(dv=view(9 * BASE)) == -8
    assert backward(dq=view(6 * BASE, t=0)) == -8
    # dimensions of one may have any stride
    assert forward(shape=shape_of(B=1, Tq=1), q=view(BASE, b=-3, t=0)) in NO_DEVICE


def test_workspace_query_refuses():
    lib = fa.load_library()
    for query in (lib.fa_cross_fwd_workspace, lib.fa_cross_bwd_workspace):
        assert query(0, 1, 1, 1, 1, 64) == -2
        assert query(1, 3, 2, 1, 1, 64) == -2
        assert query(1, 2, 2, 1, 1, 32) == -3


def test_cpu_tensors_are_refused():
    q, k, v, do = tensors((1, 2, 2, 3, 4, 64), device="cpu")
    with pytest.raises(ValueError):
        fa.cross_attention(q, k, v)
    with pytest.raises(ValueError):
        fa.attention_forward_cross(q, k, v)
    with pytest.raises(ValueError):
        fa.attention_backward_cross(q, k, v, q, do[..., 0].float(), do)


@pytest.mark.gpu
def test_refusals_of_the_python_entry_points():
    q, k, v, do = tensors((2, 4, 2, 3, 5, 64))
    o, lse = fa.attention_forward_cross(q, k, v)
    bad = [
        dict(q=q.float()), dict(k=k.half()), dict(v=v[:, :, :4]), dict(k=k[:1]), dict(v=v.cpu()),
        dict(q=q[:, :3]), dict(q=q[0]), dict(k=k.expand(2, 2, 5, 64)[..., ::2]),
        dict(key_lengths=torch.tensor([5, 5])), dict(key_lengths=ints([5])), dict(key_lengths=ints([5, 5]).cpu()),
        dict(out=torch.empty_like(q, dtype=torch.float32)), dict(out=torch.empty_like(k)),
        dict(lse=torch.empty(2, 4, 4, device="cuda")), dict(k=k[:, :1].expand(-1, 2, -1, -1)),
    ]
    for x in bad:
        with pytest.raises(ValueError):
            fa.attention_forward_cross(**{**dict(q=q, k=k, v=v), **x})
    for x in (dict(o=o.float()), dict(lse=lse[:, :2]), dict(do=do[:, :2]), dict(dk=torch.empty_like(q)), dict(rest=torch.empty_like(o)[:1]),
              dict(dv=torch.empty_like(v, dtype=torch.float16))):
        with pytest.raises(ValueError):
            fa.attention_backward_cross(**{**dict(q=q, k=k, v=v, o=o, lse=lse, do=do), **x})
    with pytest.raises(fa.FAError):
        fa.attention_forward_cross(q, k, v, out=q)
    with pytest.raises(fa.FAError):
        fa.attention_backward_cross(q, k, v, o, lse, do, dk=torch.empty_like(k), dv=k)
    with pytest.raises(fa.FAError):
        fa.attention_forward_cross(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous())
    with pytest.raises(fa.FAError):
        fa.attention_forward_cross(q[:, :, :0], k, v)
