"""Trees of drafted tokens over the 4-bit cache: attention, which tokens stand, and
keeping those (``fa_kv4_tree``, ``fa_tree_accept``, ``fa_kv4_keep`` in ``include/fa.h``).

A tree takes the last N slots of a sequence; ``parents`` (int32 (B, N)) holds each
place's parent, below it, or -1 behind the context; any other value marks a place without
a token."""
from __future__ import annotations

import math

from . import FA_OK, FAError, _launch_on, _raw_stream, load_library
from .kv4 import _account, _cache

__all__ = ["attention_tree_kv4", "tree_accept", "kv4_keep"]


_workspace_bytes: dict = {}


def _check_parents(parents, B, N, dev):
    import torch
    if not (parents.dtype is torch.int32 and parents.shape == (B, N) and parents.is_contiguous()
            and parents.get_device() == dev):
        raise ValueError("parents must be a contiguous int32 (B, N) tensor on the same device")


def _attention(q, pool, block_table, lengths, parents, scale, out, lse):
    import torch
    packed, B, heads, D, slots, dev = _cache(pool, block_table, lengths)
    shape = q.shape
    if not (q.dtype is torch.bfloat16 and len(shape) == 4 and q.is_contiguous() and q.get_device() == dev
            and shape[0] == B and shape[3] == D):
        raise ValueError("q must be a contiguous (B, H, N, D) bf16 tensor on the pool's device")
    _, Hq, N, _ = shape
    _check_parents(parents, B, N, dev)
    if out is None:
        out = torch.empty_like(q)
    elif not (out.dtype is torch.bfloat16 and out.shape == shape and out.is_contiguous() and out.get_device() == dev):
        raise ValueError("out must be like q")
    if lse is None:
        lse = torch.empty((B, Hq, N), device=q.device, dtype=torch.float32)
    elif not (lse.dtype is torch.float32 and lse.shape == (B, Hq, N) and lse.is_contiguous()
              and lse.get_device() == dev):
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor on the pool's device")
    lib = load_library()
    key = B, Hq, heads, N, D, slots, dev
    need = _workspace_bytes.get(key)
    if need is None:
        need = lib.fa_kv4_tree_workspace(B, Hq, heads, N, D, slots)
        if need < 0:
            raise FAError(need, "fa_kv4_tree_workspace")
        if len(_workspace_bytes) > 4096:
            _workspace_bytes.clear()
        _workspace_bytes[key] = need
    workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    rc = lib.fa_kv4_tree(packed, q.data_ptr(), parents.data_ptr(), out.data_ptr(), lse.data_ptr(), Hq, N,
                         1.0 / math.sqrt(D) if scale is None else scale, workspace.data_ptr() if need else None, need,
                         _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv4_tree")
    return out, lse


def attention_tree_kv4(q, pool, block_table, lengths, parents, scale: float | None = None, out=None, lse=None,
                       stream=None):
    """O (B, H, N, D) and LSE (B, H, N) of q (B, H, N, D) for a tree of N <= 64 drafted tokens over the 4-bit cache.

    ``lengths`` counts the tree's N places, the sequence's last slots (kv4_append writes them).  Each
    place sees the context, its ancestors and itself; one without a token gives 0 and -infinity.
    H is a multiple of the pool's kv heads.  A chain (parents -1, 0, 1, ...) is causal decoding, with
    weights and values rounded to bf16.  No attention weights are accumulated for kv4_evict."""
    return _launch_on(pool, stream, _attention, q, pool, block_table, lengths, parents, scale, out, lse)


def _accept(parents, tokens, picks, first):
    import torch
    if parents.dim() != 2:
        raise ValueError("parents must be a contiguous int32 (B, N) tensor")
    B, N = parents.shape
    dev = parents.get_device()
    _check_parents(parents, B, N, dev)
    kind, shape, device = tokens.dtype, parents.shape, parents.device
    if kind is not torch.int64 and kind is not torch.int32:
        raise ValueError("tokens must be int32 or int64")
    if not (tokens.shape == shape and tokens.is_contiguous() and tokens.get_device() == dev):
        raise ValueError("tokens must be a contiguous (B, N) tensor on the same device")
    if not (picks.dtype is kind and picks.shape == shape and picks.is_contiguous() and picks.get_device() == dev):
        raise ValueError("picks must be a contiguous (B, N) tensor of the tokens' type on the same device")
    if first is not None and not (first.dtype is kind and first.shape == (B,) and first.is_contiguous()
                                  and first.get_device() == dev):
        raise ValueError("first must be a contiguous (B,) tensor of the tokens' type on the same device")
    path = torch.empty_like(parents)
    counts = torch.empty(B, dtype=torch.int32, device=device)
    follow = torch.empty(B, dtype=kind, device=device)
    rc = load_library().fa_tree_accept(parents.data_ptr(), tokens.data_ptr(), picks.data_ptr(),
                                       None if first is None else first.data_ptr(), kind is torch.int64, B, N,
                                       path.data_ptr(), counts.data_ptr(), follow.data_ptr(), _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_tree_accept")
    return path, counts, follow


def tree_accept(parents, tokens, picks, first=None, stream=None):
    """(path, counts, next): the longest way from a root on which every token is the model's pick behind the one before.

    tokens, picks: int32 or int64 (B, N), what was drafted at each place and what the model picks
    behind it; ``first`` (B,): its pick behind the context (None: every root stands).  path int32 (B, N):
    the places of that way, -1 behind them (of equally long ones, the one that ends lowest); counts
    int32 (B,); next (B,): the model's pick behind the last of them (``first``, or -1, where there is none)."""
    return _launch_on(parents, stream, _accept, parents, tokens, picks, first)


def _keep(pool, block_table, lengths, path, weights, slot_positions):
    import torch
    packed, B, heads, _, _, dev = _cache(pool, block_table, lengths)
    if not (path.dtype is torch.int32 and path.dim() == 2 and path.shape[0] == B and path.is_contiguous()
            and path.get_device() == dev):
        raise ValueError("path must be a contiguous int32 (B, N) tensor on the pool's device")
    slots = 0
    for t, n, dtype in ((weights, "weights", torch.float32), (slot_positions, "slot_positions", torch.int32)):
        if t is not None:
            _account(t, n, dtype, B, heads, dev, weights)
            slots = t.shape[2]
    new_lengths = torch.empty_like(lengths)
    rc = load_library().fa_kv4_keep(packed, path.data_ptr(), path.shape[1], new_lengths.data_ptr(),
                                    None if weights is None else weights.data_ptr(),
                                    None if slot_positions is None else slot_positions.data_ptr(), slots, _raw_stream(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv4_keep")
    return new_lengths


def kv4_keep(pool, block_table, lengths, path, weights=None, slot_positions=None, stream=None):
    """Keeps a path of each sequence's tree in the cache and drops the rest; returns the new lengths.

    path: int32 (B, N), rising places of the last N slots up to the first -1 (tree_accept's, say).  Their
    keys and values move to the first of those slots, and so do ``weights`` and ``slot_positions``
    (float32 / int32 (B, kv heads, slots), kept for kv4_evict) in place.  A place whose page the table does not
    name is left out (recorded).  The pages of the last N slots must be the sequence's own."""
    return _launch_on(pool, stream, _keep, pool, block_table, lengths, path, weights, slot_positions)
