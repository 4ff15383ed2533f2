"""Cross attention in 64 bits, for the tests, with a bound for each element of what the kernels may be off.

The kernels round P and dS to bf16 before their products and every result to bf16
once; a rounding is off by at most U = 2^-8 of the value.  Scores, statistics and
sums are fp32: a score is off by D 2^-24 of the sum of its products' magnitudes at
most, for which (and for the exponential and the logarithm) the bounds take 2^-18."""
import torch

U = 2.0 ** -8
F = 2.0 ** -18


def reference(q, k, v, key_lengths=None, scale=None, do=None):
    """{name: (value, bound)} of o, lse and, with do, dq, dk, dv; tensors (B, H, T, D) of any type."""
    q, k, v = (x.detach().double().cpu() for x in (q, k, v))
    B, Hq, Tq, D = q.shape
    Hkv, Tk = k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    each = Hq // Hkv
    lengths = [Tk] * B if key_lengths is None else [int(n) for n in key_lengths]
    here = torch.arange(Tk) < torch.tensor(lengths)[:, None]                     # (B, Tk)
    k, v = (torch.where(here[:, None, :, None], x, 0.0) for x in (k, v))         # whatever lies behind
    k, v = (x.repeat_interleave(each, 1) for x in (k, v))
    s = torch.where(here[:, None, None], q @ k.mT * scale, -torch.inf)
    size = (q.abs() @ k.abs().mT * abs(scale)).amax(-1, keepdim=True)            # of a row's scores
    lse = torch.logsumexp(s, -1)
    p = (s - lse[..., None].nan_to_num(neginf=0.0)).exp()
    near = F * (1 + size)                                                        # relative error of P before it is rounded
    o = p @ v
    bo = (U + 2 * near) * (p @ v.abs()) + U * o.abs()
    out = {"o": (o, bo), "lse": (lse, near[..., 0] + F * lse.abs().nan_to_num(posinf=0.0))}
    if do is None:
        return out
    do = do.detach().double().cpu()

    def heads(x):                                                                # a group's heads summed
        return x.unflatten(1, (Hkv, each)).sum(2)

    dv, bdv = heads(p.mT @ do), heads((p * (U + 2 * near)).mT @ do.abs())
    dp = do @ v.mT
    d = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - d)
    bd = (do.abs() * bo).sum(-1, keepdim=True)                                   # D is taken from the stored O
    e = U * ds.abs() + p * bd + p * (2 * near) * (do.abs() @ v.abs().mT + (do.abs() * o.abs()).sum(-1, keepdim=True))
    e = e * (1 + U)                                                              # those of rounded values
    dq, bdq = ds @ k * scale, e @ k.abs() * abs(scale)
    dk, bdk = heads(ds.mT @ q * scale), heads(e.mT @ q.abs() * abs(scale))
    for name, x, b in (("dq", dq, bdq), ("dk", dk, bdk), ("dv", dv, bdv)):
        out[name] = (x, b + U * (x.abs() + b))
    return out


def check(name, got, ref):
    """Whether every element of `got` lies within its bound of the reference."""
    value, bound = ref[name]
    got = got.detach().double().cpu()
    assert got.shape == value.shape, name
    finite = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got), finite), f"{name}: other elements are finite"
    assert torch.equal(got[~finite], value[~finite]), name
    off = (got - value).abs()[finite] - bound[finite] - 1e-30
    assert off.numel() == 0 or off.max() <= 0, f"{name}: {off.max():.3g} beyond its bound"
