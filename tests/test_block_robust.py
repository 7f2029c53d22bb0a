"""Failure handling and the debug build of the block operators' kernels."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def product(M, N, K, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w, s = ops.fp4_quantize((torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).bfloat16(), scale=0.001)
    return lambda: ops.fp4_linear(x, w, s, x_scale=0.02)


@pytest.mark.parametrize("M,N,K", [(1, 8192, 2048), (100, 1000, 2048), (300, 14000, 2048), (40, 256, 96)],
                         ids=["fused", "single", "pairs", "one_stage"])
def test_waits_that_run_out(M, N, K):
    """A product whose weights never arrive gives up within the wait limit; the
    status says so, nothing traps, and the next call is right."""
    call = product(M, N, K)
    want = call()
    ops.qsw_check_device_errors()
    try:
        ops.qsw_set_wait_timeout_ns(2_000_000)
        ops.qsw_debug_withhold_next_product()
        call()
        with pytest.raises(ops.QswError) as e:
            ops.qsw_check_device_errors()
        assert ops.STATUS[e.value.code] == "QSW_ERR_TIMEOUT"
        ops.qsw_check_device_errors()      # the word is cleared
    finally:
        ops.qsw_set_wait_timeout_ns(4_000_000_000)
    for _ in range(3):
        assert torch.equal(call(), want)
        ops.qsw_check_device_errors()


_SCRIPT = r"""
import sys
sys.path.insert(0, {root!r})
import torch
from quantized_swiglu_mlp_gb300 import build, ops
if {debug}:
    ops.load_library(build.DEBUG_LIB_PATH)
assert ops.qsw_debug_build() == {debug}
torch.cuda.set_device(0)
outs = []

def randn(seed, *shape, std=1.0, dt=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

for fmt, g in ((ops.FP4_MX, 1.0), (ops.FP4_NV, 0.02)):
    for M, N, K in ((1, 200, 288), (9, 2048, 512), (40, 130, 1056), (193, 300, 544), (97, 19585, 288), (200, 10001, 320)):
        w, s = ops.fp4_quantize(randn(1, N, K, std=K ** -0.5), fmt, scale=g / 16)if fmt else ops.fp4_quantize(randn(1, N, K, std=K ** -0.5), fmt)
        outs.append(ops.fp4_linear(randn(M, M, K), w, s, fmt, x_scale=g))
        ops.qsw_check_device_errors()
    for T, E, k, H, I in ((1, 16, 4, 96, 160), (20, 3, 2, 256, 96), (230, 8, 4, 1824, 928)):
        sc = dict(scale=g / 16) if fmt else {{}}
        gu, gus = ops.fp4_quantize(randn(2, E, 2 * I, H, std=H ** -0.5), fmt, **sc)
        d, ds = ops.fp4_quantize(randn(3, E, H, I, std=I ** -0.5), fmt, **sc)
        r = ops.moe_route(randn(4, T, E, dt=torch.float32), k)
        outs.append(ops.fp4_moe_mlp(randn(5, T, H), r, gu, gus, d, ds, fmt, x_scale=g, h_scale=g))
        ops.qsw_check_device_errors()
assert all(torch.isfinite(o.float()).all() for o in outs)
torch.save([o.cpu() for o in outs], {path!r})
print("OK")
"""


def test_debug_build_gives_the_same_bits(tmp_path):
    """NaN-filled shared and tensor memory changes nothing, and no check fails."""
    got = []
    for debug in (False, True):
        path = str(tmp_path / f"{debug}.pt")
        r = subprocess.run([sys.executable, "-c", _SCRIPT.format(root=ROOT, debug=debug, path=path)],
                           capture_output=True, text=True, timeout=600, cwd=ROOT)
        assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout[-2000:] + r.stderr[-3000:]
        got.append(torch.load(path))
    assert all(torch.equal(a, b) for a, b in zip(*got))
