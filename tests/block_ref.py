"""Plain float64 implementations of the block operators, from their formulas:
microscaled 4-bit floating point, grouped products, routing, norms.  Shares no
code with the package."""
from __future__ import annotations

import torch

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e2m1_index(a):
    """Index in GRID nearest to |a|, ties to the even index, saturating."""
    a = a.abs()
    i = torch.zeros_like(a, dtype=torch.int64)
    for j in range(7):
        mid = (GRID[j] + GRID[j + 1]) / 2
        i = torch.where((a > mid) | ((a == mid) & (j % 2 == 1)), torch.full_like(i, j + 1), i)
    return i


def e4m3_value(byte):
    b = byte.to(torch.float64)
    e, m = torch.floor(b / 8), b % 8
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    return torch.where(byte == 127, torch.full_like(v, torch.nan), v)


def e4m3_byte(v):
    """Nearest non-negative E4M3 value's byte, ties to even, saturating at 448."""
    grid = e4m3_value(torch.arange(127, device=v.device))
    i = torch.searchsorted(grid, v.to(torch.float64).clamp(max=448.0).contiguous()).clamp(1, 126)
    lo, hi = grid[i - 1], grid[i]
    mid = (lo + hi) / 2
    up = (v > mid) | ((v == mid) & (i % 2 == 0))
    return torch.where(up, i, i - 1)


def scale_value(byte, fmt, g):
    if fmt == MX:
        v = torch.exp2(byte.to(torch.float64) - 127)
        return torch.where(byte == 255, torch.full_like(v, torch.nan), v)
    return e4m3_value(byte) * g


def quantize(x, fmt, g=1.0):
    """(codes 0..15, scale bytes) of x [..., K], computed with the documented f32
    steps: products and the reciprocal correctly rounded to f32."""
    f32 = lambda t: t.to(torch.float32)     # noqa: E731
    b = f32(x).reshape(*x.shape[:-1], -1, BLOCK[fmt])
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(bad, torch.zeros_like(b), b)
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == MX:
        e = torch.frexp(amax.double()).exponent - 1 - 2
        byte = torch.where(amax > 0, (e + 127).clamp(min=0), torch.zeros_like(e)).long()
        r = b.double() * torch.exp2(127.0 - byte.double())
    else:
        byte = e4m3_byte(f32(amax.double() * f32(torch.tensor(1 / (6 * g), dtype=torch.float64)).double()).double())
        s = f32(e4m3_value(byte) * float(torch.tensor(g, dtype=torch.float32)))
        inv = torch.where(s >= 2.0 ** -126, f32(1.0 / s.double()), torch.zeros_like(s))
        r = f32(b.double() * inv.double()).double()
    code = e2m1_index(r) + 8 * torch.signbit(r)
    byte = torch.where(bad, torch.full_like(byte, 255 if fmt == MX else 127), byte)
    code = torch.where(bad, torch.zeros_like(code), code)
    return code.reshape(x.shape), byte.squeeze(-1)


def unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def scale_at(tiles, rows, n):
    """Scale bytes [rows, n] out of the 512-byte blocks, by the documented address."""
    r = torch.arange(rows, device=tiles.device)[:, None]
    j = torch.arange(n, device=tiles.device)[None]
    flat = tiles.reshape(-1)
    at = 512 * ((r // 128) * tiles.shape[-2] + j // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + j % 4
    return flat[at].long()


def values(packed, tiles, fmt, g=1.0):
    """The float64 matrix of packed codes [rows, K/2] and scale blocks."""
    rows, K = packed.shape[0], packed.shape[1] * 2
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=packed.device)
    s = scale_value(scale_at(tiles, rows, K // BLOCK[fmt]), fmt, g)
    v = grid[unpack(packed).long()].reshape(rows, -1, BLOCK[fmt]) * s[..., None]
    return v.reshape(rows, K)


def hold(x, fmt, g=1.0):
    """x (float64) rounded to the format in exact arithmetic."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK[fmt])
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == MX:
        s = torch.where(amax > 0, torch.exp2((torch.frexp(amax).exponent - 3.0).clamp(min=-127)), torch.ones_like(amax))
    else:
        s = e4m3_value(e4m3_byte(amax / (6 * g))) * g
    r = torch.where(s > 0, b / s, torch.zeros_like(b))
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    return (grid[e2m1_index(r)] * torch.sign(r) * s).reshape(x.shape)


def half_ulp(v, dtype):
    """Half the spacing of `dtype` around v (float64)."""
    bits, low = (8, -126) if dtype == torch.bfloat16 else (11, -14)
    e = (torch.frexp(v.abs()).exponent - 1).clamp(min=low).double()
    return torch.exp2(e - bits)


def sum_bound(absolute, K):
    """Bound on an f32 sum of K exact products whose magnitudes add up to
    `absolute`, in any order and with the tensor core's truncating additions
    (at most 2^-22 of the running sum each, one per 16 products)."""
    return absolute * (K / 16 + 2) * 2.0 ** -22


def route(logits, k, sigmoid=False, renormalize=True, scale=1.0):
    """(ids, weights, offsets, slots, order)."""
    x = logits.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, -torch.inf), x)
    ids = torch.argsort(-x, dim=1, stable=True)[:, :k]
    if sigmoid:
        p = torch.sigmoid(x)
    else:
        peak = x.amax(1, keepdim=True)
        p = torch.where(x == peak, torch.ones_like(x), torch.exp(x - peak))
        p = torch.where(peak == -torch.inf, torch.zeros_like(p), p)
        if not renormalize:
            total = p.sum(1, keepdim=True)
            p = torch.where(total > 0, p / total, p)
    w = p.gather(1, ids)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.bincount(flat, minlength=logits.shape[1])
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    return ids, w * scale, offsets, slots.reshape(ids.shape), order


def rms(v, w, eps):
    n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return n if w is None else n * w
