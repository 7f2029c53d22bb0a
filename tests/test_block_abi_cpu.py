"""Values that the C entries of the block operators must refuse, and sizes that no call
accepts, on the CPU."""
from __future__ import annotations

import pytest
import torch

from tests.test_abi_cpu import BIG, FAKE, INVALID, MX, NV, OK, lib  # noqa: F401

CUDA = 3


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


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are valid: with a device these would be launched")
def test_without_a_device(lib):  # noqa: F811
    """Valid calls on a machine without a GPU return an error."""
    rest = (FAKE, FAKE, None, 0, FAKE, FAKE, BIG, None)
    for fmt in (MX, NV):
        assert lib.qsw_fp4_quantize(FAKE, 1, 4, 64, fmt, 1.0, 0, FAKE, FAKE, None) == CUDA
        assert lib.qsw_fp4_dequantize(FAKE, FAKE, 1, 4, 64, fmt, 1.0, 0, FAKE, None) == CUDA
        for rows in (1, 1000):
            assert lib.qsw_fp4_linear(FAKE, rows, 64, 32, fmt, 1.0, *rest) == CUDA
            assert lib.qsw_fp4_grouped_linear(FAKE, rows, 64, 32, 3, FAKE, fmt, 1.0, *rest) == CUDA
            assert lib.qsw_fp4_moe_mlp(FAKE, rows, 64, 64, 8, 2, fmt, 1.0, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                       None, FAKE, FAKE, None, None, 0, FAKE, FAKE, BIG, None) == CUDA
    for T in (0, 1, 1000):
        assert lib.qsw_moe_route(FAKE, T, 8, 2, 2, 0, 1, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, None) == CUDA
    assert lib.qsw_rms_norm(FAKE, None, 4, 64, 1e-6, 0, FAKE, None) == CUDA
    assert lib.qsw_post_norm(FAKE, FAKE, 1, None, None, 0, 0, 1.0, None, 4, 64, 1e-6, 0, FAKE, None, None) == CUDA


def test_sizes_that_no_call_accepts(lib):  # noqa: F811
    """0, as documented, not a product that passed 64 bits."""
    top, more = 1 << 30, (1 << 30) + 1
    assert lib.qsw_fp4_scale_bytes(1, top, 32, MX) == top // 128 * 512
    assert lib.qsw_fp4_scale_bytes(1, more, 32, MX) == lib.qsw_fp4_scale_bytes(more, 1, 32, MX) == 0
    assert lib.qsw_fp4_scale_bytes(1 << 62, 1 << 62, 64, NV) == lib.qsw_fp4_scale_bytes(3, 1 << 62, 64, NV) == 0
    assert lib.qsw_fp4_scale_bytes(0, 1 << 62, 64, NV) == lib.qsw_fp4_scale_bytes(1 << 62, 0, 64, NV) == 0
    assert lib.qsw_fp4_workspace_bytes(top, 32, 1024, NV) == top * 16 + (top // 128 + 1024) * 512
    assert lib.qsw_fp4_workspace_bytes(more, 32, 1, NV) == lib.qsw_fp4_workspace_bytes(1 << 62, 64, 3, NV) == 0
    assert lib.qsw_fp4_workspace_bytes(4, 64, 1025, NV) == 0
    assert lib.qsw_fp4_moe_workspace_bytes(4, 2, 64, 64, 8, NV) > 0
    for T, k, E in ((1 << 62, 2, 8), ((1 << 29) + 1, 2, 8), (4, 33, 64), (4, 2, 1025), (4, 9, 8)):
        assert lib.qsw_fp4_moe_workspace_bytes(T, k, 64, 64, E, NV) == 0
