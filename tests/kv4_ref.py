"""The 4-bit cache and the operators over it in numpy, for the tests: the format
from its definition (one channel at a time by its nibble), attention in 64 bits."""
import math

import numpy as np
import torch


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def quantise(x, group):
    """codes (..., D) and (s, m) (..., D / group) float32 of float32 values that are bf16 numbers."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)       # NaN propagates
        span = hi - lo
        s = bf16(span / np.float32(15)).float().numpy()
        bad = ~np.isfinite(span)
        s = np.where(s < 2.0 ** -100, np.float32(0), s)
        q = np.rint((g - lo[..., None]) / s[..., None])
        flat = bad | (s == 0)
        codes = np.where(flat[..., None], 0, np.clip(np.nan_to_num(q, nan=0.0, posinf=15.0), 0, 15)).astype(np.uint8)
    nan = np.float32(np.nan)
    return codes.reshape(x.shape), np.where(bad, nan, s), np.where(bad, nan, lo)


def nibble_of(dim):
    """Nibble of each key channel and of each value channel in its row."""
    key = [8 * ((c % 32) // 8 * (dim // 32) + c // 32) + c % 8 for c in range(dim)]
    value = [4 * ((c % 32) // 4 * (dim // 32) + c // 32) + c % 4 for c in range(dim)]
    return key, value


def record(k, v, group):
    """The key and value rows of one token and head: codes and scales as bytes."""
    out = []
    for x, nibble in zip((k, v), nibble_of(k.shape[-1])):
        codes, s, m = quantise(x, group)
        row = np.zeros(x.shape[-1] // 2, np.uint8)
        for c, n in enumerate(nibble):
            row[n // 2] |= codes[c] << (4 * (n % 2))
        pairs = torch.stack((bf16(s), bf16(m)), -1).view(torch.uint8).numpy().reshape(-1)
        out += [row, pairs]
    return out


def sections(dim, group):
    """(start, bytes of a row) of the four parts of a block."""
    row, scale = dim // 2, dim // group * 4
    at, out = 0, []
    for size in (row, scale, row, scale):
        out.append((at, size))
        at += 16 * size
    return out


def store(pool, table, b, slot, k, v, group):
    """Writes one token (heads, D) into a numpy pool."""
    page_size = pool.shape[2] * 16
    page, block, r = table[b][slot // page_size], slot % page_size // 16, slot % 16
    for h in range(pool.shape[1]):
        for (at, size), data in zip(sections(k.shape[-1], group), record(k[h], v[h], group)):
            pool[page, h, block, at + r * size:at + (r + 1) * size] = data


def load(pool, table, b, length, dim, group):
    """(codes * s, m) of keys and values of a sequence: four float64 arrays (heads, length, D):
    key product, key minimum, value product, value minimum."""
    page_size = pool.shape[2] * 16
    slots = np.arange(length)
    pages = np.asarray(table)[b][slots // page_size] if length else slots
    blocks = pool[pages, :, slots % page_size // 16].transpose(1, 0, 2)      # (heads, length, bytes)
    r, c = slots % 16, np.arange(dim)
    parts = sections(dim, group)
    out = []
    for i, nibble in zip((0, 2), nibble_of(dim)):
        n = np.array(nibble)
        (at, size), (sat, ssize) = parts[i], parts[i + 1]
        idx = at + r[:, None] * size + n // 2
        codes = np.take_along_axis(blocks, np.broadcast_to(idx, (blocks.shape[0], length, dim)), 2)
        codes = codes >> (4 * (n % 2)).astype(np.uint8) & 15
        pair = sat + r[:, None] * ssize + c // group * 4
        byte = [np.take_along_axis(blocks, np.broadcast_to(pair + j, codes.shape), 2).astype(np.uint32)
                for j in range(4)]
        s = (byte[0] << 16 | byte[1] << 24).view(np.float32).astype(np.float64)
        m = (byte[2] << 16 | byte[3] << 24).view(np.float32).astype(np.float64)
        out += [s * codes, m]
    return out


def attend(q, loaded, scale, causal):
    """o, lse, p of q (Hq, Tq, D) over loaded keys and values, and what the tolerances
    go by: the largest |terms| of a score, and the weighted |terms| of the outputs."""
    ks, km, vs, vm = loaded
    heads, length, dim = ks.shape
    hq, tq, _ = q.shape
    q = q.reshape(heads, -1, tq, dim)
    s = np.einsum("hgid,htd->hgit", q, ks + km) * scale
    size = np.einsum("hgid,htd->hgit", np.abs(q), np.abs(ks) + np.abs(km)) * abs(scale)
    if causal:
        hidden = np.arange(length)[None] > length - tq + np.arange(tq)[:, None]
        s = np.where(hidden, -np.inf, s)
        size = np.where(hidden, 0.0, size)
    with np.errstate(all="ignore"):
        top = s.max(-1, keepdims=True) if length else np.full(s.shape[:-1] + (1,), -np.inf)
        e = np.where(np.isneginf(s), 0.0, np.exp(s - np.where(np.isfinite(top), top, 0.0)))
        total = e.sum(-1, keepdims=True)
        p = np.where(total > 0, e / total, 0.0)
        lse = np.where(total > 0, top + np.log(total), -np.inf)[..., 0]
    o = np.einsum("hgit,htd->hgid", p, vs + vm)
    weighed = np.einsum("hgit,htd->hgid", p, np.abs(vs) + np.abs(vm))
    most = size.max(-1) if length else np.zeros(s.shape[:-1])
    flat = lambda x: x.reshape(hq, tq, *x.shape[3:])  # noqa: E731
    return flat(o), flat(lse), p.sum((1, 2)), flat(most), flat(weighed)


# Tolerances of the decoding kernel, from its arithmetic:
# a score is a sum of products of bf16 queries (exact in fp16 when scaled by a
#   power of two) with codes, accumulated in fp32 by chained matrix instructions,
#   then scaled and offset in fp32: at most 16 roundings of 2^-23 of the sum of
#   the absolute terms, so 2^-19 of it;
# a weight p = 2^(s - m) carries that error (times 2, numerator and sum) and
#   2^-21 for the exponential and the sum;
# a weight times a scale is rounded to fp16 (2^-11 relative) before the second
#   matrix product, the output to bf16 (2^-8 relative).
def score_tol(most):
    return most * 2.0 ** -19


def o_tol(o, most, weighed):
    return np.abs(o) * 2.0 ** -8 + weighed * (2.0 ** -11 + 2.0 ** -20 + 2 * score_tol(most)[..., None]) + 2.0 ** -126


def lse_tol(lse, most):
    return score_tol(most) + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))


class Batch:
    """Sequences of random keys and values in a numpy pool, pages in shuffled order."""

    def __init__(self, lengths, heads, dim, group, page, seed, spare=0, gain=1.0):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lengths]
        width = max(1, max(need)) + spare
        order = rng.permutation(sum(need) + 2)
        self.table = np.full((len(lengths), width), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lengths, self.heads, self.dim, self.group, self.page = list(lengths), heads, dim, group, page
        self.rng = rng
        blocks = (sum(need) + 2, heads, page // 16)
        # random codes everywhere, NaN scales where no token lies
        self.pool = np.zeros((*blocks, 16 * (dim + 8 * dim // group)), np.uint8)
        parts = sections(dim, group)
        for at, size in parts[::2]:
            self.pool[..., at:at + 16 * size] = rng.integers(0, 256, (*blocks, 16 * size), dtype=np.uint8)
        live = np.zeros((*blocks, 16), bool)
        for b, n in enumerate(lengths):
            slots = np.arange(n)
            live[self.table[b][slots // page], :, slots % page // 16, slots % 16] = True
        for at, size in parts[1::2]:
            s = bf16(rng.uniform(0.2, 0.4, (*blocks, 16, size // 4)) * gain)
            m = bf16(rng.uniform(-3.0, -1.5, (*blocks, 16, size // 4)) * gain)
            pairs = torch.stack((s, m), -1)
            pairs[~torch.from_numpy(live)] = math.nan
            self.pool[..., at:at + 16 * size] = pairs.view(torch.uint8).numpy().reshape(*blocks, 16 * size)

    def queries(self, hq, tq, std=1.0):
        return bf16(self.rng.standard_normal((len(self.lengths), hq, tq, self.dim)) * std)

    def loaded(self, b):
        return load(self.pool, self.table, b, self.lengths[b], self.dim, self.group)

    def on(self, device="cuda"):
        return (torch.from_numpy(self.pool).to(device), torch.from_numpy(self.table).to(device),
                torch.tensor(self.lengths, dtype=torch.int32, device=device))
