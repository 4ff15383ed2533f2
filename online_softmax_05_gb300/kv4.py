"""The 4-bit paged key/value cache: appending, reading back, decoding over it
and evicting from it (``fa_kv4_*``; the layout is described in ``include/fa.h``).

A cache is a pool of pages (``kv4_pool``), a table of each sequence's pages and
the sequences' lengths, all held by the caller."""
from __future__ import annotations

import math
import struct

from . import FA_OK, FAError, _c_int, _launch_on, _raw_stream, load_library
from .rotary import _check_table, _positions

__all__ = ["kv4_pool", "kv4_append", "kv4_read", "attention_decode_kv4", "kv4_evict"]

# (D, group) by the bytes of a 16-token block: no two agree
_FORMATS = {16 * (d + 8 * d // g): (d, g) for d in (64, 128) for g in (32, 64)}
_pack_cache = struct.Struct("QQQ7i4x").pack
_decode_bytes: dict = {}


def kv4_pool(num_pages: int, kv_heads: int, dim: int, page_size: int = 64, group: int = 64, device="cuda"):
    """A pool of empty pages: uint8 (num_pages, kv_heads, page_size / 16, block bytes).

    dim 64 or 128; page_size a multiple of 16; group (32 or 64): channels that
    share a scale.  A token takes dim + 8 dim / group bytes per head, keys and
    values together."""
    import torch
    if dim not in (64, 128) or group not in (32, 64):
        raise ValueError("dim must be 64 or 128 and group 32 or 64")
    if page_size < 16 or page_size > 65536 or page_size % 16 or num_pages < 1 or kv_heads < 1:
        raise ValueError("page_size must be a multiple of 16 up to 65536, num_pages and kv_heads at least 1")
    return torch.zeros(num_pages, kv_heads, page_size // 16, 16 * (dim + 8 * dim // group), dtype=torch.uint8,
                       device=device)


def _cache(pool, block_table, lengths):
    """(packed fa_kv4_cache, B, Hkv, D, slots per sequence, device index)"""
    import torch
    dev, shape, i32 = pool.get_device(), pool.shape, torch.int32
    fmt = _FORMATS.get(shape[3]) if len(shape) == 4 else None
    if fmt is None or dev < 0 or pool.dtype is not torch.uint8 or shape[2] < 1 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous uint8 CUDA tensor from kv4_pool")
    table_shape = block_table.shape
    if not (block_table.dtype is i32 and len(table_shape) == 2 and block_table.is_contiguous()
            and block_table.get_device() == dev):
        raise ValueError("block_table must be a contiguous int32 (B, pages) tensor on the pool's device")
    B, width = table_shape
    if not (lengths.dtype is i32 and lengths.shape == (B,) and lengths.is_contiguous() and lengths.get_device() == dev):
        raise ValueError("lengths must be a contiguous int32 (B,) tensor on the pool's device")
    num_pages, heads, blocks, _ = shape
    packed = _pack_cache(pool.data_ptr(), block_table.data_ptr(), lengths.data_ptr(), B, heads, fmt[0], fmt[1],
                         blocks * 16, num_pages, width)
    return packed, B, heads, fmt[0], width * blocks * 16, dev


def _account(t, name, dtype, B, heads, dev, like=None):
    """A (B, heads, slots) tensor that goes with the cache."""
    if not (t.dtype == dtype and t.dim() == 3 and t.is_contiguous() and t.get_device() == dev
            and t.shape[0] == B and t.shape[1] == heads and (like is None or t.shape == like.shape)):
        raise ValueError(f"{name} must be a contiguous {dtype} (B, kv heads, slots) tensor on the pool's device")


def _append(pool, k, v, block_table, lengths, cu_new, rotary, positions, interleaved, amplitude, weights,
            slot_positions):
    import torch
    packed, B, heads, D, _, dev = _cache(pool, block_table, lengths)
    for t, n in ((k, "k"), (v, "v")):
        if not (t.dtype == torch.bfloat16 and t.dim() == 3 and t.get_device() == dev and t.shape[1] == heads
                and t.shape[2] == D and t.stride(2) == 1 and t.shape[0] == k.shape[0]):
            raise ValueError(f"{n} must be a (tokens, kv heads, D) bf16 tensor on the pool's device, channels contiguous")
    if not (cu_new.dtype == torch.int32 and cu_new.is_contiguous() and cu_new.shape == (B + 1,)
            and cu_new.get_device() == dev):
        raise ValueError("cu_new must be a contiguous int32 (B + 1,) tensor on the pool's device")
    total = _c_int(k.shape[0], "the number of tokens")
    table = turned = None
    if rotary is not None:
        turned = _check_table(rotary, D, dev)
        table = rotary.data_ptr()
    pos, pos64, _ = _positions(positions, 1, total, dev)
    slots = 0
    for t, n, dtype in ((weights, "weights", torch.float32), (slot_positions, "slot_positions", torch.int32)):
        if t is not None:
            _account(t, n, dtype, B, heads, dev, weights)
            slots = t.shape[2]
    if total:
        rc = load_library().fa_kv4_append(
            packed, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0), v.stride(1), cu_new.data_ptr(),
            total, pos, pos64, table, turned or 0, interleaved, amplitude,
            None if weights is None else weights.data_ptr(),
            None if slot_positions is None else slot_positions.data_ptr(), slots, _raw_stream(dev))
        if rc != FA_OK:
            raise FAError(rc, "fa_kv4_append")


def kv4_append(pool, k, v, block_table, lengths, cu_new, rotary=None, positions=None, interleaved: bool = False,
               amplitude: float = 1.0, weights=None, slot_positions=None, stream=None):
    """Writes new tokens to the cache, quantised to 4 bits.

    k, v: packed (tokens, kv heads, D) bf16, contiguous channels; ``cu_new``
    int32 (B + 1,) delimits each sequence's tokens.  ``lengths`` counts them
    already: they go to the last slots.  With ``rotary`` (a table from
    rotary_frequencies) the keys are rotated first, at ``positions`` (one per
    token; the slot if None), with the same result as ``rope`` before.
    ``weights`` and ``slot_positions`` (float32 / int32 (B, kv heads, slots)), kept
    for kv4_evict, get 0 and the position at the new slots (positions within int32)."""
    _launch_on(pool, stream, _append, pool, k, v, block_table, lengths, cu_new, rotary, positions,
               int(bool(interleaved)), float(amplitude), weights, slot_positions)


def _read(pool, block_table, lengths, start, count):
    import torch
    packed, B, heads, D, slots, dev = _cache(pool, block_table, lengths)
    if start is not None and not (start.dtype == torch.int32 and start.shape == (B,) and start.is_contiguous()
                                  and start.get_device() == dev):
        raise ValueError("start must be a contiguous int32 (B,) tensor on the pool's device")
    count = _c_int(slots if count is None else int(count), "count")
    k = torch.empty((B, heads, count, D), dtype=torch.bfloat16, device=pool.device)
    v = torch.empty_like(k)
    rc = load_library().fa_kv4_read(packed, None if start is None else start.data_ptr(), count, k.data_ptr(),
                                    v.data_ptr(), _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv4_read")
    return k, v


def kv4_read(pool, block_table, lengths, start=None, count: int | None = None, stream=None):
    """Keys and values (B, kv heads, count, D) in bf16 that the cache stands for, from
    slot ``start[b]`` (0 if None) on; zeros behind a sequence's length.  count: every
    slot of the table if None.  The layout is attention_decode's."""
    return _launch_on(pool, stream, _read, pool, block_table, lengths, start, count)


def _decode(q, pool, block_table, lengths, causal, scale, weights, weights_out, out, lse):
    import torch
    packed, B, heads, D, slots, dev = _cache(pool, block_table, lengths)
    shape = q.shape
    if not (q.dtype is torch.bfloat16 and len(shape) == 4 and q.is_contiguous() and q.get_device() == dev
            and shape[0] == B and shape[3] == D):
        raise ValueError("q must be a contiguous (B, H, T, D) bf16 tensor on the pool's device")
    _, Hq, Tq, _ = shape
    if out is None:
        out = torch.empty_like(q)
    elif not (out.dtype == torch.bfloat16 and out.shape == q.shape and out.is_contiguous() and out.get_device() == dev):
        raise ValueError("out must be like q")
    if lse is None:
        lse = torch.empty((B, Hq, Tq), device=q.device, dtype=torch.float32)
    elif not (lse.dtype == torch.float32 and lse.shape == (B, Hq, Tq) and lse.is_contiguous()
              and lse.get_device() == dev):
        raise ValueError("lse must be a contiguous float32 (B, H, T) tensor on the pool's device")
    w_in = w_out = None
    w_slots = 0
    if weights is not None:
        _account(weights, "weights", torch.float32, B, heads, dev)
        w_in, w_slots = weights.data_ptr(), weights.shape[2]
        if weights_out is None:
            weights_out = weights
    if weights_out is not None:
        _account(weights_out, "weights_out", torch.float32, B, heads, dev, weights)
        w_out, w_slots = weights_out.data_ptr(), weights_out.shape[2]
    lib = load_library()
    key = B, Hq, heads, Tq, D, slots, w_out is not None, dev
    need = _decode_bytes.get(key)
    if need is None:
        need = lib.fa_kv4_decode_workspace(B, Hq, heads, Tq, D, slots, int(w_out is not None))
        if need < 0:
            raise FAError(need, "fa_kv4_decode_workspace")
        if len(_decode_bytes) > 4096:
            _decode_bytes.clear()
        _decode_bytes[key] = need
    workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    rc = lib.fa_kv4_decode(packed, q.data_ptr(), out.data_ptr(), lse.data_ptr(), Hq, Tq,
                           1.0 / math.sqrt(D) if scale is None else scale, causal, w_in, w_out, w_slots,
                           workspace.data_ptr() if need else None, need, _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv4_decode")
    return (out, lse) if w_out is None else (out, lse, weights_out)


def attention_decode_kv4(q, pool, block_table, lengths, causal: bool = True, scale: float | None = None, weights=None,
                         weights_out=None, out=None, lse=None, stream=None):
    """O (B, H, Tq, D) and LSE (B, H, Tq) of q (B, H, Tq, D), Tq <= 8, over the 4-bit cache.

    H is a multiple of the pool's kv heads (grouped queries).  causal: the queries
    are the sequence's last Tq tokens and each sees up to itself; otherwise all see
    everything.  With ``weights`` (float32 (B, kv heads, slots)) every slot's
    attention weight, summed over the queries, is added to it, in place or to
    ``weights_out``, which is returned third (``weights_out`` alone: a first account)."""
    return _launch_on(pool, stream, _decode, q, pool, block_table, lengths, int(bool(causal)), scale, weights,
                      weights_out, out, lse)


def _evict(pool, block_table, lengths, weights, slot_positions, budget, recent):
    import torch
    packed, B, heads, _, _, dev = _cache(pool, block_table, lengths)
    _account(weights, "weights", torch.float32, B, heads, dev)
    _account(slot_positions, "slot_positions", torch.int32, B, heads, dev, weights)
    new_weights, new_positions = torch.empty_like(weights), torch.empty_like(slot_positions)
    new_lengths = torch.empty_like(lengths)
    lib = load_library()
    need = lib.fa_kv4_evict_workspace(B, heads, budget)
    if need < 0:
        raise FAError(need, "fa_kv4_evict_workspace")
    source = torch.empty(B, heads, budget, dtype=torch.int32, device=pool.device)
    workspace = torch.empty(max(16, need), dtype=torch.uint8, device=pool.device)
    rc = lib.fa_kv4_evict(packed, weights.data_ptr(), slot_positions.data_ptr(), weights.shape[2], budget, recent,
                          new_weights.data_ptr(), new_positions.data_ptr(), new_lengths.data_ptr(),
                          source.data_ptr(), workspace.data_ptr(), workspace.shape[0], _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv4_evict")
    return new_weights, new_positions, new_lengths, source


def kv4_evict(pool, block_table, lengths, weights, slot_positions, budget: int, recent: int = 0, stream=None):
    """Evicts every sequence down to ``budget`` tokens, each kv head by itself: the
    ``recent`` newest stay, and the ones with the largest accumulated weights.

    The pages must not be shared with other sequences (a common prefix, say).  Moves
    what has to move inside the pool and returns (weights, slot_positions,
    lengths, source) to go on with: the accounts after the eviction (0 and -1 behind
    the new length), min(length, budget), and the slot each kept token came from,
    int32 (B, kv heads, budget)."""
    return _launch_on(pool, stream, _evict, pool, block_table, lengths, weights, slot_positions,
                      _c_int(int(budget), "budget"), _c_int(int(recent), "recent"))
