"""The block operators at the sizes of long prompts, where the kernels loop, stream and
share tiles differently than for the small cases of test_block_ops.py."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import block_ref as ref
from tests.test_block_ops import (BF16, F16, SCALE, check, dev, dtypes, formats, held, moe_reference,  # noqa: F401
                                  randn, test_grouped_linear, weight)

pytestmark = pytest.mark.gpu


del test_grouped_linear     # a test of its own module; its body is used below
from tests.test_block_ops import test_grouped_linear as check_grouped_linear  # noqa: E402


# ------------------------------------------------------------- quantisation --

@formats
@pytest.mark.parametrize("shape", [(4096, 14336), (9000, 7264), (320001, 96), (3, 2000, 7200)], ids=str)
def test_quantize_and_back(dev, fmt, shape):  # noqa: F811
    """Runs of several scale blocks per CTA, with and without streaming accesses: codes and
    scales bit for bit, and the values that they stand for."""
    x = randn(1, *shape)
    x[..., 7] *= 30
    codes, scales = ops.fp4_quantize(x, fmt, scale=SCALE[fmt])
    out = ops.fp4_dequantize(codes, scales, fmt, scale=SCALE[fmt])
    g = float(torch.tensor(SCALE[fmt], dtype=torch.float32))
    n = shape[-1] // ref.BLOCK[fmt]
    stack = [(x, codes, scales, out)] if len(shape) == 2 else list(zip(x, codes, scales, out))
    for xs, c, s, o in stack:
        held_at = ref.scale_at(s, xs.shape[0], s.shape[-2] * 4)
        assert not held_at[:, n:].any()
        for lo in range(0, xs.shape[0], 32768):
            hi = min(lo + 32768, xs.shape[0])
            want, byte = ref.quantize(xs[lo:hi], fmt, SCALE[fmt])
            assert torch.equal(held_at[lo:hi, :n], byte)
            assert torch.equal(ref.unpack(c[lo:hi]).long(), want)
            grid = torch.tensor(ref.GRID + tuple(-v for v in ref.GRID), dtype=torch.float64, device="cuda")
            v = (grid[want].unflatten(-1, (-1, ref.BLOCK[fmt])) * ref.scale_value(byte, fmt, g)[..., None]).flatten(-2)
            check(o[lo:hi], v, ref.half_ulp(v, BF16) * (1 + 2.0 ** -10) + v.abs() * 2.0 ** -23)


# ----------------------------------------------------------------- products --

def check_linear(M, N, K, fmt, dt=BF16, rows=1 << 18):
    x = randn(M + N + K, M, K, dt=dt)
    w, ws, wg, vals = weight(3, 1, N, K, fmt)
    y = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    ops.qsw_check_device_errors()
    a = held(x, fmt)
    for lo in range(0, M, rows):
        part = a[lo:lo + rows]
        want = part @ vals[0].T
        check(y[lo:lo + rows], want, ref.half_ulp(want, dt) * (1 + 2.0 ** -8)
              + ref.sum_bound(part.abs() @ vals[0].abs().T, K) + 2.0 ** -26)


@formats
@pytest.mark.parametrize("M,N,K", [(1, 20001, 512), (3, 60000, 256), (16, 39000, 512), (2, 20000, 4096)])
def test_several_tiles_for_rows_that_each_cta_quantises(dev, fmt, M, N, K):  # noqa: F811
    check_linear(M, N, K, fmt, F16)


@formats
@pytest.mark.parametrize("M,N,K", [(1, 5_000_065, 32), (1_880_003, 257, 32)], ids=["single", "pairs"])
def test_more_tiles_than_records(dev, fmt, M, N, K):  # noqa: F811
    """More than 256 tiles per CTA, or pair: the grid grows."""
    check_linear(M, N, K, fmt)


@formats
@pytest.mark.parametrize("N,K", [(2100, 160), (1793, 576)])
def test_grouped_linear_on_cta_pairs(dev, fmt, N, K):  # noqa: F811
    """Ragged groups of 213 rows on average, enough for the two-CTA form; empty ones among them."""
    check_grouped_linear(dev, fmt, [100, 0, 257, 64, 31, 192, 0, 193, 128, 900, 1, 700], N, K)


@formats
@pytest.mark.parametrize("sizes,N,K", [([3000, 0, 2100, 41, 3051], 64, 7168), ([2500, 1, 5700], 300, 4128)], ids=str)
def test_grouped_linear_with_long_rows(dev, fmt, sizes, N, K):  # noqa: F811
    """The ragged quantiser's runs of several scale blocks."""
    check_grouped_linear(dev, fmt, sizes, N, K)


# ------------------------------------------------------------------ experts --

def experts(E, H, I, fmt):
    gu, gus, gug, vgu = weight(8, E, 2 * I, H, fmt)
    d, ds, dg, vd = weight(9, E, H, I, fmt)

    def mlp(x, r, residual=None, d_scale=dg):
        return ops.fp4_moe_mlp(x, r, gu, gus, d, ds, fmt, x_scale=SCALE[fmt], h_scale=SCALE[fmt], gu_scale=gug,
                               d_scale=d_scale, residual=residual)
    return mlp, vgu, vd, dg


def test_moe_rows_do_not_overflow(dev):  # noqa: F811
    """Rows of experts beyond f16's largest value whose weighted sum is within it, in a
    batch of any size (here 0.1 to 13 MB of rows): finite, and the bits that a token gets alone."""
    fmt, E, k, H, I = ops.FP4_NV, 8, 8, 2048, 32
    mlp, _, _, dg = experts(E, H, I, fmt)
    x, logits = randn(1, 200, H, dt=F16), randn(2, 200, E, dt=torch.float32)
    big = dg * 1e8

    def run(rows):
        return mlp(x[rows], ops.moe_route(logits[rows], k, scale=1e-5), d_scale=big)
    y = run(slice(None))
    assert float(mlp(x[:4], ops.moe_route(logits[:4], k), d_scale=dg).abs().max()) * 1e8 / 8 > 65504
    assert torch.isfinite(y).all()
    for a, b in ((0, 2), (100, 128), (199, 200)):
        assert torch.equal(y[a:b], run(slice(a, b))), (a, b)


@formats
@dtypes
@pytest.mark.parametrize("T,E,k,H,I", [(300, 8, 8, 2048, 64), (1500, 6, 3, 1056, 96), (700, 3, 2, 2112, 1056)])
def test_moe_long_batch(dev, fmt, dt, T, E, k, H, I):  # noqa: F811
    """Long batches (the last with both products on CTA pairs): sampled tokens against
    float64, and the bits that they get in small batches."""
    mlp, vgu, vd, _ = experts(E, H, I, fmt)
    x, logits, res = randn(T, T, H, dt=dt), randn(T + 1, T, E, dt=torch.float32), randn(T + 2, T, H, dt=dt)
    r = ops.moe_route(logits, k)
    y = mlp(x, r, res)
    ops.qsw_check_device_errors()
    some = torch.tensor([0, 1, T // 3, T // 2, T - 130, T - 1], device="cuda")
    want, bound = moe_reference(x[some], r._replace(ids=r.ids[some], weights=r.weights[some]), k, vgu, vd, fmt, dt, res[some])
    check(y[some], want, bound)
    for a, b in ((0, 1), (T // 2, T // 2 + 20), (T - 1, T)):
        assert torch.equal(y[a:b], mlp(x[a:b], ops.moe_route(logits[a:b], k), res[a:b])), (a, b)


# -------------------------------------------------------------------- norms --

def norm_case(rows, H, dt, gates):
    h, y, w, wn = randn(1, rows, H, dt=dt, std=4.0), randn(2, rows, H, dt=dt), randn(3, H, dt=dt), randn(4, H, dt=dt)
    gate = randn(5, gates, H, dt=dt)
    return h, y, w, wn, gate


@dtypes
@pytest.mark.parametrize("rows,H,gates", [(1000, 4096, 4), (2600, 512, 1), (5000, 100, 5000), (700, 8200, 7), (400, 8191, 2),
                                          (320, 16390, 4), (310, 20001, 1), (330, 10002, 2), (330, 12001, 1), (8192, 4096, 4)])
def test_norms_over_many_rows(dev, dt, rows, H, gates):  # noqa: F811
    """Several rows per CTA, of each width; the last with streaming accesses.  In place the same bits."""
    h, y, w, wn, gate = norm_case(rows, H, dt, gates)
    out, n = ops.post_norm(h, y, w, gate=gate, scale=0.7, next_weight=wn, eps=1e-5)
    alone = ops.rms_norm(h, wn, eps=1e-5)
    hh, yy = h.clone(), y.clone()
    ops.post_norm(hh, yy, w, gate=gate, scale=0.7, next_weight=wn, eps=1e-5, out=hh, next_out=yy)
    assert torch.equal(hh, out) and torch.equal(yy, n)
    rel = (H / 2 + 16) * 2.0 ** -24      # as in test_post_norm
    for lo in range(0, rows, 1024):
        s = slice(lo, min(lo + 1024, rows))
        each = torch.arange(lo, s.stop, device="cuda") // (rows // gates)
        add = 0.7 * gate[each].double() * ref.rms(y[s].double(), w.double(), 1e-5)
        want = h[s].double() + add
        slack = (add.abs() + want.abs()) * rel
        check(out[s], want, ref.half_ulp(want, dt) * 1.01 + slack)
        nw = ref.rms(want, wn.double(), 1e-5)
        f = (nw / want).abs().nan_to_num(0)
        check(n[s], nw, ref.half_ulp(nw, dt) * 1.01 + slack * f + nw.abs() * 2 * rel + 1e-30)
        want = ref.rms(h[s].double(), wn.double(), 1e-5)
        check(alone[s], want, ref.half_ulp(want, dt) * 1.01 + want.abs() * (H / 2 + 8) * 2.0 ** -24)
