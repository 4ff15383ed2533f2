"""Cross attention: queries of one sequence over the keys and values of another
(``fa_cross_*``, described in ``include/fa.h``)."""
from __future__ import annotations

import math
import struct
import threading

from . import FA_OK, FAError, _launch_on, _raw_stream, load_library

__all__ = ["attention_forward_cross", "attention_backward_cross", "cross_attention"]

_pack_shape = struct.Struct("6iQ").pack
_pack_tensor = struct.Struct("Q3q").pack
_lock = threading.Lock()
_autograd_cls = None
_forward_bytes: dict = {}


def _fits(t) -> bool:
    """Whether the kernels take the tensor by its strides."""
    b, h, s, c = t.stride()
    if c != 1 or t.data_ptr() & 15:
        return False
    if b > 0 and h > 0 and s > 0 and not (b | h | s) & 7:
        return True
    B, H, T, _ = t.shape  # a dimension of one may have any stride
    return ((B == 1 or (b > 0 and not b & 7)) and (H == 1 or (h > 0 and not h & 7))
            and (T == 1 or (s > 0 and not s & 7)))


def _tensor(t, name, shape, dev) -> bytes:
    import torch
    if not (t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == dev and dev >= 0):
        raise ValueError(f"{name} must be a bf16 CUDA tensor {tuple(shape)} on the device of the others")
    if not _fits(t):
        raise ValueError(f"{name} must have contiguous channels, 16-byte alignment and strides that are positive "
                         "multiples of 8")
    return _packed(t)


def _packed(t) -> bytes:
    b, h, s, _ = t.stride()
    return _pack_tensor(t.data_ptr(), b, h, s)


def _shape(q, k, key_lengths):
    """(packed fa_cross_shape, query shape, key shape, device index)"""
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be (B, H, T, D) tensors")
    dev = q.get_device()
    B, Hq, Tq, D = q.shape
    _, Hkv, Tk, _ = k.shape
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    if key_lengths is not None and not (key_lengths.dtype is torch.int32 and key_lengths.shape == (B,)
                                        and key_lengths.is_contiguous() and key_lengths.get_device() == dev):
        raise ValueError("key_lengths must be a contiguous int32 (B,) tensor on the device of q")
    if max(B, Hq, Hkv, Tq, Tk) >= 1 << 31:
        raise ValueError("a dimension is out of range")
    packed = _pack_shape(B, Hq, Hkv, Tq, Tk, D, 0 if key_lengths is None else key_lengths.data_ptr())
    return packed, (B, Hq, Tq, D), (B, Hkv, Tk, D), dev


def _check_lse(lse, shape, dev):
    import torch
    if not (lse.dtype is torch.float32 and lse.shape == shape and lse.is_contiguous() and lse.get_device() == dev):
        raise ValueError("lse must be a contiguous float32 (B, H, T) tensor on the device of q")


def _rest(rest, shape, dev):
    import torch
    if rest is None:
        return None
    if not (rest.dtype is torch.bfloat16 and rest.shape == shape and rest.is_contiguous() and rest.get_device() == dev):
        raise ValueError("rest must be a contiguous bf16 (B, H, T, D) tensor on the device of q")
    return rest.data_ptr()


def _forward(q, k, v, key_lengths, scale, out, lse, rest):
    import torch
    packed, rows, keys, dev = _shape(q, k, key_lengths)
    qp, kp, vp = _tensor(q, "q", rows, dev), _tensor(k, "k", keys, dev), _tensor(v, "v", keys, dev)
    if out is None:
        out = torch.empty_like(q)
        op = _packed(out)
    else:
        op = _tensor(out, "out", rows, dev)
    if lse is None:
        lse = torch.empty(rows[:3], device=q.device, dtype=torch.float32)
    else:
        _check_lse(lse, rows[:3], dev)
    lib = load_library()
    key = rows, keys, dev
    need = _forward_bytes.get(key)
    if need is None:
        need = lib.fa_cross_fwd_workspace(rows[0], rows[1], keys[1], rows[2], keys[2], rows[3])
        if need < 0:
            raise FAError(need, "fa_cross_fwd_workspace")
        if len(_forward_bytes) > 4096:
            _forward_bytes.clear()
        _forward_bytes[key] = need
    workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    rc = lib.fa_cross_fwd(packed, qp, kp, vp, op, _rest(rest, rows, dev), lse.data_ptr(),
                          1.0 / math.sqrt(rows[3]) if scale is None else scale,
                          workspace.data_ptr() if need else None, need, _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_cross_fwd")
    return out, lse


def attention_forward_cross(q, k, v, key_lengths=None, scale: float | None = None, out=None, lse=None, rest=None,
                            stream=None):
    """O and LSE of q (B, Hq, Tq, D) over k, v (B, Hkv, Tk, D), every query over its sequence's
    keys below ``key_lengths[b]`` (int32 CUDA tensor; None: all Tk).

    bf16 tensors with contiguous channels and any other strides that are multiples of 8 (heads
    behind tokens, views of a fused projection); Hq is a multiple of Hkv.  What lies past a length
    is not used, NaN included; a sequence without keys gives 0 and -infinity.  The output lies in
    memory as q does.

    ``rest``, a contiguous bf16 (B, Hq, Tq, D) tensor, receives what rounding O to bf16 took off;
    given to the backward it makes dQ more exact (cross_attention does so)."""
    return _launch_on(q, stream, _forward, q, k, v, key_lengths, scale, out, lse, rest)


def _backward(q, k, v, o, lse, do, key_lengths, scale, rest, dq, dk, dv):
    import torch
    packed, rows, keys, dev = _shape(q, k, key_lengths)
    tensors = [_tensor(q, "q", rows, dev), _tensor(k, "k", keys, dev), _tensor(v, "v", keys, dev),
               _tensor(o, "o", rows, dev)]
    do_view = _tensor(do, "do", rows, dev)
    _check_lse(lse, rows[:3], dev)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    grads = [_tensor(dq, "dq", rows, dev), _tensor(dk, "dk", keys, dev), _tensor(dv, "dv", keys, dev)]
    lib = load_library()
    need = lib.fa_cross_bwd_workspace(rows[0], rows[1], keys[1], rows[2], keys[2], rows[3])
    if need < 0:
        raise FAError(need, "fa_cross_bwd_workspace")
    workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib.fa_cross_bwd(packed, *tensors, _rest(rest, rows, dev), do_view, lse.data_ptr(), *grads,
                          1.0 / math.sqrt(rows[3]) if scale is None else scale, workspace.data_ptr(), need,
                          _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_cross_bwd")
    return dq, dk, dv


def attention_backward_cross(q, k, v, o, lse, do, key_lengths=None, scale: float | None = None, rest=None, dq=None,
                             dk=None, dv=None, stream=None):
    """dQ, dK, dV for attention_forward_cross (o, lse and ``rest`` are its results); tensors by their
    strides as there.  dK and dV sum over the query heads of a group and are 0 past a length."""
    return _launch_on(q, stream, _backward, q, k, v, o, lse, do, key_lengths, scale, rest, dq, dk, dv)


def _laid_out(t, name):
    """(B, H, T, D) of a (B, H, T, D) or (B, T, D) tensor, copied if the kernels cannot take its strides or address."""
    import torch
    if t.dim() == 3:
        t = t.unsqueeze(1)
    elif t.dim() != 4:
        raise ValueError(f"{name} must be (B, H, T, D) or (B, T, D)")
    if _fits(t):
        return t
    # contiguous() returns a tensor that is already contiguous, whatever its address
    return t.clone(memory_format=torch.contiguous_format)


def _make_autograd_class():
    import torch
    from torch.autograd.function import once_differentiable

    class CrossAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, key_lengths, scale):
            q4, k4, v4 = (_laid_out(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
            rest = torch.empty(q4.shape, dtype=q4.dtype, device=q4.device) if any(ctx.needs_input_grad) else None
            o, lse = attention_forward_cross(q4, k4, v4, key_lengths, scale, rest=rest)
            ctx.save_for_backward(q4, k4, v4, o, lse, rest, key_lengths)
            ctx.scale, ctx.dims = scale, (q.dim(), k.dim(), v.dim())
            return o.squeeze(1) if q.dim() == 3 else o

        @staticmethod
        @once_differentiable
        def backward(ctx, grad_o):
            q, k, v, o, lse, rest, key_lengths = ctx.saved_tensors
            grads = attention_backward_cross(q, k, v, o, lse, _laid_out(grad_o, "grad of o"), key_lengths, ctx.scale, rest)
            return tuple(g.squeeze(1) if n == 3 else g for g, n in zip(grads, ctx.dims)) + (None, None)

    return CrossAttention


def cross_attention(q, k, v, key_lengths=None, scale: float | None = None):
    """O = softmax(q k^T * scale) v with keys of another sequence, differentiable once.

    q (B, Hq, Tq, D) and k, v (B, Hkv, Tk, D), or (B, T, D) as one head; Hq a multiple of Hkv.
    ``key_lengths`` (int32 CUDA tensor (B,)) are the keys there; scale defaults to 1/sqrt(D).
    See attention_forward_cross; what the kernels cannot take (a broadcast, a view off 16-byte alignment) is copied.
    A pass captured into a CUDA graph wants leaves that no eager autograd graph still holds: torch would
    join that graph's stream to the capture, and fails."""
    global _autograd_cls
    if _autograd_cls is None:
        with _lock:
            if _autograd_cls is None:
                _autograd_cls = _make_autograd_class()
    return _autograd_cls.apply(q, k, v, key_lengths, scale)
