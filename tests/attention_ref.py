"""Plain float64 implementations of the attention operators, and bounds of their errors."""
from __future__ import annotations

import math

import torch

# Half a step of a type, relative; and half a step of its smallest numbers, absolute.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def rope(x, positions, frequencies, interleaved=False, scale=1.0):
    """(values, bound): [T, heads, D] in float64, angles in float64."""
    n = len(frequencies)
    x64 = x.double()
    angle = (positions.double()[:, None] * frequencies.double().to(x.device))[:, None]
    r = x64[..., :2 * n]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :n], r[..., n:])
    y0, y1 = (a * angle.cos() - b * angle.sin()) * scale, (a * angle.sin() + b * angle.cos()) * scale
    size = (a.abs() + b.abs()) * abs(scale)
    put = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat((p, q), -1))
    y, size = put(y0, y1), put(size, size)
    # one rounding at the end; before it the angle (2^-23 of a radian: 2^-33 turns and f32's
    # half step of half a turn, 2^-24 pi), cos and sin (2 ulp each), their product with the scale,
    # two products and a sum (f32): together below 2^-20 of the operands
    bound = y.abs() * HALF[x.dtype] + size * 2.0 ** -20 + TINY[x.dtype]
    rest = x64[..., 2 * n:]
    return torch.cat((y, rest), -1), torch.cat((bound, torch.zeros_like(rest)), -1)


def plan(offsets, lengths, page_table, page_size, pages, tokens):
    """(positions, slots) as lists, sequence by sequence."""
    positions, slots = [-1] * tokens, [-1] * tokens
    for b, length in enumerate(lengths):
        lo, hi = offsets[b], offsets[b + 1]
        length = min(max(length, 0), len(page_table[b]) * page_size)
        for t in range(lo, hi):
            p = length - (hi - t)
            if p < 0:
                continue
            positions[t] = p
            page = page_table[b][p // page_size]
            if 0 <= page < pages:
                slots[t] = page * page_size + p % page_size
    return positions, slots


def gather(cache, table, length):
    """[kv_heads, length, D] of one sequence in float64; pages outside the cache are zeros."""
    pages, kv_heads, page_size, D = cache.shape
    p = torch.arange(length, device=cache.device)
    page = table.long()[p // page_size] if length else p
    good = (page >= 0) & (page < pages)
    rows = cache[page.clamp(0, pages - 1), :, p % page_size].double()
    return torch.where(good[:, None, None], rows, 0.0).transpose(0, 1)


def attention(q, k_cache, v_cache, offsets, lengths, page_table, scale, window=0):
    """(values, bound), float64 [T, heads, D]; NaN in rows of no sequence."""
    T, heads, D = q.shape
    kv_heads, page_size = k_cache.shape[1:3]
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    bound = torch.full_like(out, math.nan)
    half, tiny = HALF[q.dtype], TINY[q.dtype]
    for b, length in enumerate(lengths):
        lo, hi = offsets[b], offsets[b + 1]
        if lo == hi:
            continue
        length = min(max(length, 0), page_table.shape[1] * page_size)
        k, v = gather(k_cache, page_table[b], length), gather(v_cache, page_table[b], length)
        at = length - (hi - lo) + torch.arange(hi - lo, device=q.device)[:, None]
        j = torch.arange(length, device=q.device)
        seen = (j <= at) & ((j > at - window) if window else True)
        for h in range(heads):
            kv = h * kv_heads // heads
            qh = q[lo:hi, h].double()
            s = torch.where(seen, qh @ k[kv].T * scale, -math.inf)
            top = s.amax(1, keepdim=True) if length else torch.full((hi - lo, 1), -math.inf, device=q.device)
            w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total == 0, 1.0, total)
            # key by key where a weight is 0: what is not seen has no part in the sum
            fine = torch.isfinite(v[kv]).all() and torch.isfinite(s[seen]).all()

            def weighted(x):
                return w @ x if fine else torch.stack([w[i][seen[i]] @ x[seen[i]] for i in range(hi - lo)])
            o, size = weighted(v[kv]), weighted(v[kv].abs())
            # Scores in f32: D products and their sum, each step within 2^-23 of the sum of
            # magnitudes; a weight is off by twice that (its own and the sum's).
            mag = (qh.abs() @ torch.where(torch.isfinite(k[kv]), k[kv].abs(), 0.0).T * scale)
            mag = torch.where(seen, mag, 0.0).amax(1, keepdim=True) if length else torch.zeros_like(top)
            rel = 2 * (D + 8) * 2.0 ** -23 * mag
            # The weights' rounding to the type (relative, and its smallest numbers' half step times
            # |v| over a sum of at least 1), the sums of `length` products in f32, 2^-19 for the
            # exponentials, factors and divisions of a few passes; the rounding at the end.
            rel = rel + half + (length / 8 + 64) * 2.0 ** -23 + 2.0 ** -19
            most = v[kv].abs().nan_to_num(0.0, 0.0, 0.0).sum(0)[None] if length else 0.0
            out[lo:hi, h] = o
            bound[lo:hi, h] = rel * size + o.abs() * half + tiny * (1 + most)
    return out, bound
