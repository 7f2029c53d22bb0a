"""Arguments of the block operators that are refused, or have to be taken with care."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_block_ops import BF16, SCALE, dev, formats, randn, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 64), (0,), (4, 0), (0, 1)], ids=str)
def test_post_norm_refuses_an_empty_gate(dev, shape):  # noqa: F811
    h, y = randn(1, 4, 64), randn(2, 4, 64)
    with pytest.raises(ValueError, match="gate"):
        ops.post_norm(h, y, gate=torch.empty(shape, dtype=BF16, device="cuda"))
    out, n = ops.post_norm(h[:0], y[:0], gate=torch.empty(0, 64, dtype=BF16, device="cuda"))
    assert out.shape == n.shape == (0, 64)


@formats
@pytest.mark.parametrize("M,K,N", [(1, 512, 512), (4, 2048, 2048), (16, 512, 512), (3, 96, 2400), (40, 512, 512), (300, 256, 256)])
def test_products_over_their_own_input(dev, fmt, M, K, N):  # noqa: F811
    """y over x, exactly or shifted: the bits of a call with an output of its own."""
    w, ws, wg, _ = weight(4, 1, N, K, fmt)
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    for shift in (0, 64):
        size = M * max(K, N) + shift
        for grouped in (False, True):
            def product(a, out):
                if grouped:
                    return ops.fp4_grouped_linear(a, offsets, w, ws, fmt, x_scale=SCALE[fmt], w_scale=wg, out=out)
                return ops.fp4_linear(a, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg, out=out)
            for rep in range(5):
                buf = randn(M + N + rep, size)
                x = buf[:M * K].view(M, K)
                want = product(x.clone(), None)
                got = product(x, buf[shift:shift + M * N].view(M, N))
                assert torch.equal(got, want), (shift, grouped, rep)
