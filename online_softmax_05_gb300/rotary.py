"""Rotary positions for the attention entry points: frequency tables, the
rotation of queries and keys (``fa_rope``), and its gradient under autograd."""
from __future__ import annotations

import math
import struct

from . import FA_OK, FAError, _c_int, _launch_on, _lock, _raw_stream, load_library

__all__ = ["rope", "rotary_frequencies", "rotary_amplitude"]

_DTYPES: dict = {}
_rope_cls = None
_forward_ad = None
_pack_tensor = struct.Struct("9q").pack


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, low_turns: float = 1.0, high_turns: float = 32.0,
                       frequencies=None, device="cuda"):
    """The table ``rope`` and ``kv4_append`` take: int64 (rotary_dim / 2,), turns
    per position in units of 2^-64.

    Pair i turns by base^(-2 i / rotary_dim) radians per position.  ``scaling``
    stretches a context by ``factor``:
      ``"linear"``  every frequency divided by factor
      ``"base"``    base multiplied by factor^(rotary_dim / (rotary_dim - 2)), so
                    that the slowest pair is divided by factor and the fastest kept
      ``"parts"``   by the turns a pair makes in ``original_length`` positions:
                    fewer than low_turns divided by factor, more than high_turns
                    kept, a linear mix between; use rotary_amplitude(factor) with it
    ``frequencies`` (radians per position, rotary_dim / 2 of them) replaces the
    formula; "linear" and "parts" apply to it."""
    import torch
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    if not (factor > 0 and math.isfinite(factor) and base > 0 and math.isfinite(base)):
        raise ValueError("base and factor must be positive and finite")
    if frequencies is not None:
        f = [float(x) for x in frequencies]
        if len(f) != rotary_dim // 2 or not all(math.isfinite(x) for x in f):
            raise ValueError("frequencies must be rotary_dim / 2 finite numbers")
        if scaling == "base":
            raise ValueError("scaling 'base' is for the formula, which frequencies replaces")
    else:
        if scaling == "base":
            if rotary_dim == 2:
                raise ValueError("scaling 'base' needs a rotary_dim above 2")
            base = base * factor ** (rotary_dim / (rotary_dim - 2))
        f = [base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":
        if not original_length or original_length < 1 or not high_turns > low_turns:
            raise ValueError("scaling 'parts' needs original_length, and high_turns above low_turns")
        keep = [min(1.0, max(0.0, (original_length * x / (2 * math.pi) - low_turns) / (high_turns - low_turns)))
                for x in f]
        f = [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)]
    words = [round(x / (2 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for x in f]
    return torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64, device=device)


def rotary_amplitude(factor: float) -> float:
    """The amplitude that goes with scaling 'parts': 0.1 ln(factor) + 1 (1 for factors up to 1)."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _positions(positions, batch, rows, dev):
    """(pointer, is 64-bit, batch stride) of a positions tensor (rows,) or (batch, rows)."""
    import torch
    if positions is None:
        return None, 0, 0
    dtype, shape, stride = positions.dtype, positions.shape, positions.stride()
    if (dtype is not torch.int32 and dtype is not torch.int64) or positions.get_device() != dev:
        raise ValueError("positions must be an int32 or int64 tensor on the device of the others")
    if len(shape) == 2 and (shape[0] == batch or shape[0] == 1):
        step = stride[0] if shape[0] > 1 else 0
    elif len(shape) == 1:
        step = 0
    else:
        raise ValueError("positions must be (T,) or (B, T)")
    if shape[-1] != rows or (rows > 1 and stride[-1] != 1):
        raise ValueError("positions must hold T consecutive values per row")
    return positions.data_ptr(), int(dtype is torch.int64), step


def _check_table(table, dim, dev):
    import torch
    if table.dtype is not torch.int64 or table.dim() != 1 or not table.is_contiguous() or table.get_device() != dev:
        raise ValueError("the frequency table must be a contiguous 1-D int64 tensor on the device of the others")
    rotary = 2 * table.shape[0]
    if rotary < 2 or rotary > dim:
        raise ValueError("the frequency table must hold 1 .. D/2 entries")
    return rotary


def _rope(tensors, table, positions, interleaved, amplitude, inverse, outs):
    """fa_rope on the current stream; tensors: one or two (B, H, T, D)."""
    import torch
    if not _DTYPES:
        _DTYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    first = tensors[0]
    dev, dtype, shape = first.get_device(), first.dtype, first.shape
    code = _DTYPES.get(dtype)
    if len(shape) != 4 or code is None or dev < 0:
        raise ValueError("rope takes (B, H, T, D) CUDA tensors of one type: bf16, fp16 or fp32")
    B, _, T, D = shape
    _c_int(B * T, "the number of rows of a head")
    packed, results, count = b"", (), 0
    for i, t in enumerate(tensors):
        if i:
            shape = t.shape
            if t.dtype is not dtype or t.get_device() != dev or len(shape) != 4:
                raise ValueError("rope takes (B, H, T, D) CUDA tensors of one type: bf16, fp16 or fp32")
            if shape[0] != B or shape[2] != T or shape[3] != D:
                raise ValueError("rope's tensors may differ in their heads only")
        sb, sh, st, sc = t.stride()
        if sc != 1 and D > 1:
            raise ValueError("the channels of rope's tensors must be contiguous")
        H = shape[1]
        if outs is None:
            o = torch.empty(shape, dtype=dtype, device=t.device)
            ob, oh, ot = H * T * D, T * D, D
        else:
            o = outs[i]
            if o.shape != shape or o.dtype is not dtype or o.get_device() != dev or (o.stride(3) != 1 and D > 1):
                raise ValueError("out must match rope's input in shape, type and device, with contiguous channels")
            ob, oh, ot, _ = o.stride()
        results += (o,)
        if H:
            packed += _pack_tensor(t.data_ptr(), o.data_ptr(), H, sb, st, sh, ob, ot, oh)
            count += 1
    rotary = _check_table(table, D, dev)
    pos, pos64, pos_b = _positions(positions, B, T, dev)
    if B * T * count:
        rc = load_library().fa_rope(packed, count, pos, pos64, pos_b, table.data_ptr(), B, T, D, rotary,
                                    interleaved, amplitude, inverse, code, _raw_stream(dev))
        if rc != FA_OK:
            raise FAError(rc, "fa_rope")
    return results


def _make_rope_class():
    import torch

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, table, positions, interleaved, amplitude, inverse):
            ctx.save_for_backward(table, positions)
            ctx.args = interleaved, amplitude, inverse
            got = _rope((q,) if k is None else (q, k), table, positions, interleaved, amplitude, inverse, None)
            return got if k is not None else got[0]

        @staticmethod
        def backward(ctx, *grads):
            table, positions = ctx.saved_tensors
            interleaved, amplitude, inverse = ctx.args
            want = [i for i, g in enumerate(grads) if ctx.needs_input_grad[i] and g is not None]
            given = [grads[i] if grads[i].stride(3) == 1 or grads[i].shape[3] == 1 else grads[i].contiguous()
                     for i in want]
            turned = []
            if given:
                # the inverse turn, itself differentiable
                turned = _rope_any(given, table, positions, interleaved, amplitude, 1 - inverse)
            full = [None, None]
            for i, g in zip(want, turned):
                full[i] = g
            return full[0], full[1], None, None, None, None, None

    return Rope


def _has_tangent(tensors):
    """Whether a tensor carries a forward-mode derivative."""
    global _forward_ad
    if _forward_ad is None:
        from torch.autograd import forward_ad as _forward_ad
    if getattr(_forward_ad, "_current_level", 0) < 0:  # no forward mode at all: a microsecond saved
        return False
    return any(_forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _rope_any(tensors, table, positions, interleaved, amplitude, inverse):
    """_rope, through autograd where a tensor wants it (which refuses forward mode)."""
    import torch
    if (torch.is_grad_enabled() and (tensors[0].requires_grad or tensors[-1].requires_grad)) or _has_tangent(tensors):
        global _rope_cls
        if _rope_cls is None:
            cls = _make_rope_class()
            with _lock:
                _rope_cls = _rope_cls or cls
        k = tensors[1] if len(tensors) > 1 else None
        got = _rope_cls.apply(tensors[0], k, table, positions, interleaved, amplitude, inverse)
        return got if k is not None else (got,)
    return _rope(tensors, table, positions, interleaved, amplitude, inverse, None)


def rope(q, k, table, positions=None, interleaved: bool = False, amplitude: float = 1.0, inverse: bool = False,
         out=None, stream=None):
    """Rotated copies of queries (B, Hq, T, D) and keys (B, Hkv, T, D), one launch.

    bf16, fp16 or fp32 CUDA tensors with contiguous channels and any other
    strides (views of a fused projection, say); the results are contiguous, as
    the attention entry points want them.  ``k`` may be None: then one tensor is
    returned.  ``table``: from rotary_frequencies, its 2 * len(table) channels
    are rotated and the others copied.  ``positions``: int32 or int64 (T,) or
    (B, T), 0 .. T-1 if None.  ``interleaved``: pairs (2i, 2i + 1) instead of
    (i, i + R/2).  ``inverse`` turns back.  ``out``: tensors (a tuple if k is
    given) to write to, which may be the inputs; not under autograd.
    Differentiable in q and k, any number of times; forward-mode derivatives raise."""
    tensors = (q,) if k is None else (q, k)
    if out is None:
        got = _launch_on(q, stream, _rope_any, tensors, table, positions, 1 if interleaved else 0, amplitude,
                         1 if inverse else 0)
    else:
        outs = (out,) if k is None else tuple(out)
        if len(outs) != len(tensors):
            raise ValueError("out must hold a tensor for each input")
        import torch
        if torch.is_grad_enabled() and any(t.requires_grad for t in tensors + outs) or _has_tangent(tensors + outs):
            raise ValueError("out cannot be given under autograd")
        got = _launch_on(q, stream, _rope, tensors, table, positions, 1 if interleaved else 0, amplitude,
                         1 if inverse else 0, outs)
        for t in outs:  # as torch's own in-place operations: a gradient that saved the old values raises
            if not t.is_inference():
                torch.autograd.graph.increment_version(t)
    return got if k is not None else got[0]
