"""The block operators at the sizes of long prompts, where the kernels loop, stream and
share tiles differently than for the small cases of test_block_ops.py."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import block_ref as ref
from tests.test_block_ops import BF16, F16, SCALE, check, dev, dtypes, formats, moe_reference, randn, weight  # noqa: F401

pytestmark = pytest.mark.gpu


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
@pytest.mark.parametrize("T,E,k,H,I", [(300, 8, 8, 2048, 64), (1500, 6, 3, 1056, 96)])
def test_moe_long_batch(dev, fmt, dt, T, E, k, H, I):  # noqa: F811
    """More than 8 MB of expert rows: sampled tokens against float64, and the bits that they get in small batches."""
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
