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
