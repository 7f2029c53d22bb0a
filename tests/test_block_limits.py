"""The block operators at their limits: many experts and choices, and matrices whose
offsets pass 32 bits."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import block_ref as ref
from tests.test_block_large import check_grouped_linear, experts
from tests.test_block_ops import BF16, SCALE, check, dev, formats, held, moe_reference, randn, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@formats
@pytest.mark.parametrize("T,E,k,H,I", [(1, 40, 17, 96, 64), (7, 64, 32, 256, 32), (30, 12, 9, 288, 96), (3, 1024, 8, 64, 32)])
def test_many_choices_and_experts(dev, fmt, T, E, k, H, I):  # noqa: F811
    """More choices than the weighted sum has in flight, as many experts as there may be."""
    mlp, vgu, vd, _ = experts(E, H, I, fmt)
    x, res = randn(T, T, H), randn(T + 2, T, H)
    r = ops.moe_route(randn(T + 1, T, E, dt=torch.float32), k)
    y = mlp(x, r, res)
    ops.qsw_check_device_errors()
    want, bound = moe_reference(x, r, k, vgu, vd, fmt, BF16, res)
    check(y, want, bound)


@formats
def test_a_thousand_groups(dev, fmt):  # noqa: F811
    check_grouped_linear(dev, fmt, [(7 * e) % 4 * (e % 3) + (200 if e == 700 else 0) for e in range(1024)], 136, 96)


# Past 2^32 bytes, or 2^31 elements: rows are checked against calls on few rows.

def some_rows(rows):
    return torch.tensor([0, 1, rows // 3, rows // 2 + 77, rows - 129, rows - 2, rows - 1], device="cuda")


def bits(rows, n, seed=0):
    """Random bf16 values of moderate size, made in place (randn would need four times the memory)."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.empty(rows, n, dtype=BF16, device="cuda")
    for part in x.split(1 << 16):
        part.normal_(generator=g)
    return x


@formats
def test_quantize_past_32_bits(dev, fmt):  # noqa: F811
    rows, K = 310_000, 14336
    x, at = bits(rows, K), some_rows(310_000)
    codes, scales = ops.fp4_quantize(x, fmt, scale=SCALE[fmt])
    out = ops.fp4_dequantize(codes, scales, fmt, scale=SCALE[fmt])
    want = ops.fp4_dequantize(*ops.fp4_quantize(x[at], fmt, scale=SCALE[fmt]), fmt, scale=SCALE[fmt])
    assert torch.equal(out[at], want)
    assert torch.equal(codes[at], ops.fp4_quantize(x[at], fmt, scale=SCALE[fmt])[0])


@formats
def test_linear_past_32_bits(dev, fmt):  # noqa: F811
    M, N, K = 140_001, 16400, 96
    x, at = bits(M, K), some_rows(M)
    w, ws, wg, vals = weight(3, 1, N, K, fmt)
    y = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    ops.qsw_check_device_errors()
    a = held(x[at].contiguous(), fmt)
    want = a @ vals[0].T
    check(y[at], want, ref.half_ulp(want, BF16) * (1 + 2.0 ** -8) + ref.sum_bound(a.abs() @ vals[0].abs().T, K) + 2.0 ** -26)


@formats
def test_expert_mlp_past_32_bits(dev, fmt):  # noqa: F811
    """9.4 GB of expert rows; every token checked against the same tokens in smaller batches."""
    T, E, k, H, I = 143_000, 9, 8, 2048, 32
    mlp, _, _, _ = experts(E, H, I, fmt)
    x, logits = bits(T, H), randn(2, T, E, dt=torch.float32)
    y = mlp(x, ops.moe_route(logits, k))
    ops.qsw_check_device_errors()
    for lo in range(0, T, 30_000):
        hi = min(lo + 30_000, T)
        assert torch.equal(y[lo:hi], mlp(x[lo:hi], ops.moe_route(logits[lo:hi], k))), lo


def test_norms_past_32_bits(dev):  # noqa: F811
    rows, H = 540_000, 4096
    h, y, w = bits(rows, H), bits(rows, H, 1), randn(3, H)
    gate = bits(rows // 2, H, 2)
    out, n = ops.post_norm(h, y, w, gate=gate, scale=0.5, next_weight=w)
    alone = ops.rms_norm(h, w)
    for lo in range(0, rows, 60_000):
        s, g = slice(lo, lo + 60_000), gate[lo // 2:(lo + 60_000) // 2]
        a, b = ops.post_norm(h[s], y[s], w, gate=g, scale=0.5, next_weight=w)
        assert torch.equal(out[s], a) and torch.equal(n[s], b)
        assert torch.equal(alone[s], ops.rms_norm(h[s], w))
