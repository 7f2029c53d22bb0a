"""Values that the C entries of the block operators must refuse, and sizes that no call
accepts, on the CPU."""
from __future__ import annotations

import pytest

from tests.test_abi_cpu import BIG, FAKE, INVALID, MX, NV, OK, lib  # noqa: F401


@pytest.mark.parametrize("scale,code", [(1e-45, INVALID), (1e-40, INVALID), (4.8e-40, INVALID), (5e-40, OK), (1e-30, OK),
                                        (3e38, OK)])
def test_tensor_scales_without_a_reciprocal(lib, scale, code):  # noqa: F811
    """1 / (6 g) beyond f32 made blocks of zeros NaN (0 times infinity)."""
    rows = 0 if code == OK else 4      # nothing is launched
    assert lib.qsw_fp4_quantize(FAKE, 1, rows, 64, NV, scale, 0, FAKE, FAKE, None) == code
    assert lib.qsw_fp4_dequantize(FAKE, FAKE, 1, rows, 64, NV, scale, 0, FAKE, None) == code
    assert lib.qsw_fp4_linear(FAKE, rows, 64, 32, NV, scale, FAKE, FAKE, None, 0, FAKE, FAKE, BIG, None) == code
    for x_scale, h_scale in ((scale, 1.0), (1.0, scale)):
        assert lib.qsw_fp4_moe_mlp(FAKE, rows, 64, 64, 8, 2, NV, x_scale, h_scale, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                   FAKE, None, FAKE, FAKE, None, None, 0, FAKE, FAKE, BIG, None) == code
