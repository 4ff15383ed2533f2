"""Rotary positions (fa_rope) against the formula in 64 bits, angles as exact whole
numbers, every element; gradients against the formula's and against differences.

Tolerance of an element: half a step of its type, and for the fp32 arithmetic
2^-22 a (|x1| + |x2|): cosine and sine are rounded to fp32 (2^-24), and so are their
products with the amplitude, those with x1 and x2, and the sum."""
import math

import numpy as np
import pytest
import torch

import online_softmax_05_gb300 as fa

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_05_gb300 import build
    build.build()
    fa.load_library()


def turned(x, table, positions, interleaved, amplitude, inverse=False):
    """x (B, H, T, D) float64, positions (B, T) ints -> the rotation, and |x1| + |x2| of each channel's pair."""
    words = [int(w) for w in table.tolist()]
    angle = np.array([[[(int(p) * w) % 2 ** 64 / 2.0 ** 64 for w in words] for p in row] for row in positions])
    c, s = np.cos(2 * np.pi * angle)[:, None] * amplitude, np.sin(2 * np.pi * angle)[:, None] * amplitude
    if inverse:
        s = -s
    r = 2 * len(words)
    one, two = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, size = x.copy(), np.zeros_like(x)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    size[..., one] = size[..., two] = np.abs(x[..., one]) + np.abs(x[..., two])
    return y, size * amplitude


def check(got, want, size, dtype):
    got = got.detach().cpu().double().numpy()
    tol = HALF[dtype] * np.abs(want) + size * 2.0 ** -22 + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


def fused(B, T, Hq, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda().transpose(1, 2)
    return x[:, :Hq], x[:, Hq:Hq + Hkv]


def test_frequencies_follow_their_formulas():
    def radians(**kw):
        t = fa.rotary_frequencies(64, device="cpu", **kw)
        return t.double().numpy() / 2.0 ** 64 * 2 * math.pi
    i = np.arange(32)
    plain = 10000.0 ** (-i / 32)
    assert np.allclose(radians(), plain, rtol=1e-12)
    assert np.allclose(radians(scaling="linear", factor=4), plain / 4, rtol=1e-12)
    stretched = radians(scaling="base", factor=8)
    assert np.allclose(stretched[[0, -1]], [1.0, plain[-1] / 8], rtol=1e-12)
    parts = radians(scaling="parts", factor=8, original_length=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(parts[turns > 32], plain[turns > 32], rtol=1e-12)
    assert np.allclose(parts[turns < 1], plain[turns < 1] / 8, rtol=1e-12)
    between = (turns > 1) & (turns < 32)
    assert ((parts < plain) & (parts > plain / 8))[between].all() and between.any()
    own = np.linspace(-2.0, 3.0, 32)   # negative ones wrap
    t = fa.rotary_frequencies(64, frequencies=own, device="cpu")
    assert np.allclose([int(w) / 2.0 ** 64 * 2 * math.pi for w in t], own, atol=1e-12)
    assert fa.rotary_amplitude(1.0) == 1.0 and math.isclose(fa.rotary_amplitude(8.0), 0.1 * math.log(8) + 1)


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(scaling="other"), dict(factor=0.0),
                                dict(scaling="parts"), dict(frequencies=[1.0]), dict(base=-1.0),
                                dict(rotary_dim=2, scaling="base", factor=2.0),
                                dict(scaling="parts", original_length=64, low_turns=4.0, high_turns=4.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        fa.rotary_frequencies(**{"rotary_dim": 64, "device": "cpu", **kw})


def test_rope_refuses_cpu_tensors():
    x = torch.zeros(1, 1, 4, 64)
    with pytest.raises(ValueError):
        fa.rope(x, x, fa.rotary_frequencies(64, device="cpu"))


BASE = 1 << 40


def c_rope(lib_args=None, tensors=None, **kw):
    from online_softmax_05_gb300.rotary import _pack_tensor
    t = dict(inp=BASE, out=2 * BASE, heads=4, in_b=4096, in_t=64, in_h=1024, out_b=4096, out_t=64, out_h=1024)
    t2 = dict(t, inp=3 * BASE, out=4 * BASE)
    t.update(tensors or {})
    a = dict(n=1, pos=None, pos64=0, freq=5 * BASE, B=2, T=16, D=64, rotary=64, inter=0, amp=1.0, inverse=0, dtype=0)
    a.update(kw)
    packed = b"".join(_pack_tensor(*x.values()) for x in (t, t2))
    return fa.load_library().fa_rope(packed if a.get("tensors", 1) else None, a["n"], a["pos"], a["pos64"], 0,
                                     a["freq"], a["B"], a["T"], a["D"], a["rotary"], a["inter"], a["amp"],
                                     a["inverse"], a["dtype"], None)


def test_c_entry_refuses():
    assert c_rope(freq=None) == -1
    assert c_rope(tensors=dict(inp=0)) == -1
    assert c_rope(B=0) == -2 and c_rope(T=0) == -2 and c_rope(D=2048, rotary=64) == -2
    assert c_rope(tensors=dict(heads=0)) == -2
    assert c_rope(B=1 << 16, T=1 << 16) == -2
    assert c_rope(rotary=63) == -3 and c_rope(rotary=66) == -3 and c_rope(rotary=0) == -3 and c_rope(dtype=3) == -3
    assert c_rope(freq=5 * BASE + 4) == -4 and c_rope(tensors=dict(inp=BASE + 1)) == -4
    assert c_rope(pos=BASE * 6 + 4, pos64=1) == -4
    assert c_rope(amp=float("nan")) == -8 and c_rope(inter=2) == -8 and c_rope(n=3) == -8
    assert c_rope(tensors=dict(in_t=-64)) == -8
    assert c_rope(tensors=dict(out_h=0)) == -8                      # heads written on top of each other
    assert c_rope(tensors=dict(out=BASE + 64)) == -8                # output inside the input
    assert c_rope(tensors=dict(out=BASE, out_t=128)) == -8          # in place with other strides
    assert c_rope(tensors=dict(out=4 * BASE), n=2) == -8            # both tensors to one output
    assert c_rope(tensors=dict(out=3 * BASE), n=2) == -8            # one tensor's output in the other's input


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rotary", [
    (2, 5, 3, 1, 64, 64), (1, 1, 1, 1, 128, 128), (3, 17, 8, 2, 128, 64), (2, 33, 9, 3, 64, 20), (1, 7, 5, 5, 80, 62),
    (2, 3, 2, 1, 33, 2), (1, 300, 12, 4, 96, 96), (2, 9, 40, 1, 256, 32), (1, 2, 2, 2, 2, 2),
    (2, 19, 4, 2, 128, 126), (2, 19, 4, 2, 128, 20), (1, 5, 3, 3, 72, 22), (1, 5, 3, 3, 66, 12), (3, 4, 2, 2, 68, 44),
    (1, 6, 2, 1, 1024, 1022)])
def test_rope_matches_the_formula(B, T, Hq, Hkv, D, rotary, interleaved, dtype):
    q, k = fused(B, T, Hq, Hkv, D, dtype, seed=B * T + D)
    table = fa.rotary_frequencies(rotary, device="cuda")
    positions = torch.randint(-50, 1 << 20, (B, T), dtype=torch.int32, device="cuda",
                              generator=torch.Generator("cuda").manual_seed(1))
    got = fa.rope(q, k, table, positions, interleaved=interleaved, amplitude=1.25)
    for x, y in zip((q, k), got):
        assert y.is_contiguous() and y.shape == x.shape and y.dtype == dtype
        want, size = turned(x.cpu().double().numpy(), table, positions.tolist(), interleaved, 1.25)
        check(y, want, size, dtype)
        assert torch.equal(y[..., rotary:], x[..., rotary:])


@pytest.mark.gpu
@pytest.mark.parametrize("positions", [[0, 1, 2, 3], [2 ** 31 - 1, 2 ** 24 + 1, 999983, 123456789],
                                       [-1, -2 ** 31, -77, 5], [2 ** 40 + 3, -2 ** 50, 2 ** 62, 10 ** 12]])
def test_far_positions_keep_their_angle(positions):
    q = torch.randn(1, 2, 4, 128, generator=torch.Generator().manual_seed(3)).cuda()
    table = fa.rotary_frequencies(128, device="cuda")
    dtype = torch.int64 if max(map(abs, positions)) >= 2 ** 31 + 1 else torch.int32
    y = fa.rope(q, None, table, torch.tensor(positions, dtype=dtype, device="cuda"))
    want, size = turned(q.cpu().double().numpy(), table, [positions], False, 1.0)
    check(y, want, size, torch.float32)


@pytest.mark.gpu
def test_default_positions_shared_positions_and_layouts_agree():
    q, k = fused(2, 21, 4, 2, 64, torch.bfloat16, 5)
    table = fa.rotary_frequencies(64, device="cuda")
    a = fa.rope(q, k, table)
    for positions in (torch.arange(21, device="cuda"), torch.arange(21, dtype=torch.int32, device="cuda").expand(2, 21),
                      torch.arange(42, device="cuda").reshape(1, 42)[:, :21]):
        b = fa.rope(q.contiguous(), k.contiguous(), table, positions)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    alone = fa.rope(k, None, table)
    assert torch.equal(alone, a[1])
    # unaligned rows take the narrow path and give the same bits
    shifted = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    shifted.copy_(q)
    assert torch.equal(fa.rope(shifted, None, table), a[0])


@pytest.mark.gpu
def test_in_place_on_views_of_one_projection():
    B, T, Hq, Hkv, D = 2, 19, 6, 2, 128
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    keep = x.clone()
    q, k = x.transpose(1, 2)[:, :Hq], x.transpose(1, 2)[:, Hq:Hq + Hkv]
    table = fa.rotary_frequencies(96, device="cuda")
    want = fa.rope(q, k, table)
    got = fa.rope(q, k, table, out=(q, k))
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(x[:, :, Hq + Hkv:], keep[:, :, Hq + Hkv:])
    with pytest.raises(fa.FAError):
        fa.rope(q, k, table, out=(q, q[:, :Hkv]))
    with pytest.raises(fa.FAError):                 # broadcast heads cannot be written
        fa.rope(q, None, table, out=torch.zeros(B, 1, T, D, dtype=torch.bfloat16, device="cuda").expand(B, Hq, T, D))


@pytest.mark.gpu
def test_python_entry_refuses():
    q, k = fused(1, 4, 2, 1, 64, torch.bfloat16, 5)
    table = fa.rotary_frequencies(64, device="cuda")
    for bad in (lambda: fa.rope(q.double(), k.double(), table), lambda: fa.rope(q, k.float(), table),
                lambda: fa.rope(q[0], k[0], table), lambda: fa.rope(q.transpose(2, 3), None, table),
                lambda: fa.rope(q, k, table.int()), lambda: fa.rope(q, k, fa.rotary_frequencies(66, device="cuda")),
                lambda: fa.rope(q, k, table, torch.arange(5, device="cuda")),
                lambda: fa.rope(q, k, table, torch.arange(4.0, device="cuda")),
                lambda: fa.rope(q, k, table, torch.arange(4)), lambda: fa.rope(q, k, table, out=(q,)),
                lambda: fa.rope(q, k[..., :32], table), lambda: fa.rope(q.clone().requires_grad_(), k, table, out=(q, k))):
        with pytest.raises(ValueError):
            bad()
    empty = fa.rope(q[:, :, :0], k[:, :, :0], table)
    assert empty[0].shape == (1, 2, 0, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(dtype, interleaved):
    B, T, Hq, Hkv, D = 2, 13, 4, 2, 64
    q, k = (t.detach().requires_grad_() for t in fused(B, T, Hq, Hkv, D, dtype, 9))
    table = fa.rotary_frequencies(48, device="cuda")
    positions = torch.randint(0, 4096, (B, T), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    yq, yk = fa.rope(q, k, table, positions, interleaved=interleaved, amplitude=0.75)
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk), retain_graph=True)
    for g, d in ((gq, dq), (gk, dk)):
        want, size = turned(g.cpu().double().numpy(), table, positions.tolist(), interleaved, 0.75, inverse=True)
        check(d, want, size, dtype)
    # broadcast and transposed gradients, and one input alone
    assert torch.equal(torch.autograd.grad(yk.sum(), k, retain_graph=True)[0],
                       fa.rope(torch.ones_like(yk), None, table, positions, interleaved=interleaved, amplitude=0.75,
                               inverse=True))
    turned_g = gq.transpose(2, 3).contiguous().transpose(2, 3)
    assert torch.equal(torch.autograd.grad(yq, q, turned_g, retain_graph=True)[0], dq)


@pytest.mark.gpu
def test_gradient_against_differences_and_twice():
    # linear in x: a central difference is exact up to rounding, so a wide step is taken
    x = torch.randn(1, 2, 3, 16, generator=torch.Generator().manual_seed(4)).cuda().requires_grad_()
    table = fa.rotary_frequencies(12, device="cuda")
    g = torch.randn(1, 2, 3, 16, generator=torch.Generator().manual_seed(5)).cuda().requires_grad_()
    y = fa.rope(x, None, table)
    (dx,) = torch.autograd.grad(y, x, g, create_graph=True)
    with torch.no_grad():
        for i in range(0, x.numel(), 5):
            e = torch.zeros_like(x).view(-1)
            e[i] = 1.0
            e = e.view(x.shape)
            num = ((fa.rope(x + e, None, table) - fa.rope(x - e, None, table)).double() / 2 * g.double()).sum()
            # at most 32 elements of the pair move; each rounding 2^-22 of values below 6
            assert abs(float(num) - float(dx.view(-1)[i])) <= 2.0 ** -22 * 6 * float(g.abs().sum())
    (back,) = torch.autograd.grad(dx, g, torch.ones_like(dx))
    assert torch.equal(back, fa.rope(torch.ones_like(x), None, table).detach())


@pytest.mark.gpu
@pytest.mark.parametrize("dims", [4, 3])
def test_flash_attention_rotates_and_its_gradients_go_through(dims):
    B, H, T, D = 2, 2, 150, 64
    g = torch.Generator().manual_seed(6)
    shape = (B, H, T, D) if dims == 4 else (B, T, D)
    q, k, v = (torch.randn(shape, generator=g).to(torch.bfloat16).cuda().requires_grad_() for _ in range(3))
    do = torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
    table = fa.rotary_frequencies(D, device="cuda")
    o = fa.flash_attention(q, k, v, causal=True, rotary=table)
    grads = torch.autograd.grad(o, (q, k, v), do)
    up = (lambda t: t) if dims == 4 else (lambda t: t.unsqueeze(1))
    q2, k2 = (t.detach() for t in fa.rope(up(q), up(k), table))
    o2, lse = fa.attention_forward(q2, k2, up(v).contiguous(), causal=True)
    assert torch.equal(up(o), o2)
    dq2, dk2, dv2 = fa.attention_backward(q2, k2, up(v).contiguous(), o2, lse, up(do).contiguous(), causal=True)
    dq, dk = fa.rope(dq2, dk2, table, inverse=True)
    for a, b in zip(grads, (dq, dk, dv2)):
        assert torch.equal(up(a), b)


@pytest.mark.gpu
def test_streams_and_graph():
    q, k = fused(2, 64, 4, 2, 128, torch.bfloat16, 11)
    table = fa.rotary_frequencies(128, device="cuda")
    want = fa.rope(q, k, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.rope(q, k, table, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qs, ks = q.clone(), k.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = fa.rope(qs, ks, table)
    qs.copy_(q.flip(2))
    ks.copy_(k.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    want = fa.rope(q.flip(2), k.flip(2), table)
    assert torch.equal(cap[0], want[0]) and torch.equal(cap[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 1])
def test_a_tensor_without_heads_leaves_the_other(empty):
    q, k = fused(2, 9, 3, 2, 64, torch.bfloat16, 12)
    table = fa.rotary_frequencies(64, device="cuda")
    x = [t.detach().contiguous() for t in (q, k)]
    x[empty] = x[empty][:, :0]
    full = x[1 - empty]
    want = fa.rope(full, None, table)
    torch.full((4, *full.shape), 9.0, dtype=full.dtype, device="cuda")      # what a result not written would hold
    got = fa.rope(*x, table)
    assert got[empty].shape == x[empty].shape and torch.equal(got[1 - empty], want)
    leaves = [t.requires_grad_() for t in x]
    out = fa.rope(*leaves, table)
    torch.full((4, *full.shape), 9.0, dtype=full.dtype, device="cuda")
    grads = torch.autograd.grad(out, leaves, [torch.ones_like(t) for t in out])
    assert grads[empty].shape == x[empty].shape
    assert torch.equal(grads[1 - empty], fa.rope(torch.ones_like(want), None, table, inverse=True))


def test_outputs_whose_rows_share_elements_are_refused():
    # each stride covers a row by itself, but batch 1 lies on rows 1 .. of batch 0, or rows on heads
    assert c_rope(tensors=dict(heads=1, out_b=64, out_t=64)) == -8
    assert c_rope(tensors=dict(out_t=64, out_h=64)) == -8
    assert c_rope(tensors=dict(out_t=64, out_h=960)) == -8          # the last row on the next head's first
    assert c_rope(tensors=dict(out_b=2048, out_t=64, out_h=1024)) == -8
    assert c_rope(tensors=dict(out_t=256, out_h=64, out_b=16 * 256 - 1)) == -8
    assert c_rope(tensors=dict(inp=BASE, out=BASE, in_t=64, in_h=64, out_t=64, out_h=64)) == -8      # in place


@pytest.mark.gpu
@pytest.mark.parametrize("order", [(0, 1, 2, 3), (0, 2, 1, 3), (1, 0, 2, 3), (2, 1, 0, 3)])
def test_outputs_of_any_order_of_dimensions(order):
    q, k = fused(2, 9, 3, 2, 64, torch.bfloat16, 13)
    table = fa.rotary_frequencies(64, device="cuda")
    want = fa.rope(q, k, table)
    back = [order.index(i) for i in range(4)]
    out = tuple(torch.zeros([t.shape[i] for i in order], dtype=t.dtype, device="cuda").permute(back) for t in (q, k))
    got = fa.rope(q, k, table, out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # dimensions of one element take any stride
    one = torch.zeros(1, 1, 9, 64, dtype=q.dtype, device="cuda").as_strided((1, 1, 9, 64), (1, 2, 64, 1))
    assert torch.equal(fa.rope(q[:1, :1], None, table, out=one), want[0][:1, :1])


@pytest.mark.gpu
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_raise(grad):
    # never a result without its tangent, which would be a derivative of zero
    import torch.autograd.forward_ad as fwd
    q, k = (t.detach().clone() for t in fused(1, 8, 2, 1, 64, torch.bfloat16, 14))
    v = torch.zeros_like(q)
    table = fa.rotary_frequencies(64, device="cuda")
    with fwd.dual_level(), torch.set_grad_enabled(grad):
        for x in ((fwd.make_dual(q, torch.ones_like(q)), k), (q, fwd.make_dual(k, torch.ones_like(k)))):
            with pytest.raises(RuntimeError):
                fa.rope(*x, table)
            with pytest.raises(ValueError):
                fa.rope(*x, table, out=(q.clone(), k.clone()))
        with pytest.raises(RuntimeError):
            fa.flash_attention(fwd.make_dual(q, torch.ones_like(q)), q, v, rotary=table)
        assert fa.rope(q, k, table)[0].shape == q.shape
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: fa.rope(x, k, table)[0], (q,), (torch.ones_like(q),))


@pytest.mark.gpu
def test_more_rows_than_32_bits_count_are_refused():
    q = torch.zeros(1, 1, 1, 2, dtype=torch.bfloat16, device="cuda")
    table = fa.rotary_frequencies(2, device="cuda")
    for shape in ((1, 1, 2 ** 32 + 1, 2), (2 ** 16, 1, 2 ** 16, 2)):
        with pytest.raises(ValueError):
            fa.rope(q.expand(shape), None, table)


@pytest.mark.gpu
def test_gradients_that_saved_what_is_rotated_in_place_raise():
    q, k = (t.detach().contiguous() for t in fused(1, 8, 2, 1, 64, torch.float32, 15))
    table = fa.rotary_frequencies(64, device="cuda")
    x = torch.ones_like(q).requires_grad_()
    y = x * q                       # saves q
    fa.rope(q, k, table, out=(q, k))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        z = q.clone()
        assert torch.equal(fa.rope(z, None, table, out=z), fa.rope(q, None, table))


@pytest.mark.parametrize("kw", [dict(positions=torch.arange(4)), dict(interleaved=True), dict(amplitude=1.5)])
def test_flash_attention_refuses_a_rotation_without_its_table(kw):
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rotary"):
        fa.flash_attention(x, x, x, **kw)


def test_own_frequencies_have_no_base_to_scale():
    own = [0.5, 0.25]
    with pytest.raises(ValueError, match="base"):
        fa.rotary_frequencies(4, scaling="base", factor=2.0, frequencies=own, device="cpu")
    half = fa.rotary_frequencies(4, scaling="linear", factor=2.0, frequencies=own, device="cpu")
    assert torch.equal(half, fa.rotary_frequencies(4, frequencies=[0.25, 0.125], device="cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(160000, 0), (70001, 100001)])
def test_more_heads_than_a_grid_has_rows(Hq, Hkv):
    q, k = (torch.randn(1, h, 1, 2, generator=torch.Generator().manual_seed(16)).cuda() for h in (Hq, Hkv))
    table = fa.rotary_frequencies(2, device="cuda")
    where = torch.tensor([5], device="cuda")
    got = fa.rope(q, k, table, where)
    for x, y in zip((q, k), got):
        assert torch.equal(y, torch.cat([fa.rope(part, None, table, where) for part in x.split(60000, 1)], 1))
