"""Failure handling and the debug build for the forms of the product that test_block_robust.py
does not reach: K split over a cluster, SwiGLU and ragged groups on CTA pairs."""
from __future__ import annotations

import subprocess
import sys

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_block_robust import ROOT, product

pytestmark = pytest.mark.gpu


def gives_up(call, check):
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
        check(call(), want)
        ops.qsw_check_device_errors()


@pytest.mark.parametrize("M,N,K", [(1, 128, 6144), (1, 2048, 8192), (40, 256, 6240), (100, 1000, 8192)],
                         ids=["split_fused", "split_in_4", "split_in_4_uneven", "split_in_2"])
def test_waits_that_run_out_in_a_cluster(M, N, K):
    """All CTAs that share a tile give up within the wait limit, and the next call is right."""
    def same(got, want):
        assert torch.equal(got, want)
    gives_up(product(M, N, K), same)


@pytest.mark.parametrize("T", [1, 30, 700], ids=["fused", "single", "pairs"])
def test_expert_mlp_whose_first_product_gives_up(T):
    """The gate and up product's weights never arrive: the rest of the call runs on what
    there is, reports the timeout, and the next call is right."""
    E, k, H, I = 3, 2, 2112, 1056
    g = torch.Generator("cuda").manual_seed(1)

    def weights(*shape):
        return ops.fp4_quantize((torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16(), scale=0.001)
    gu, d = weights(E, 2 * I, H), weights(E, H, I)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    r = ops.moe_route(torch.randn(T, E, generator=g, device="cuda"), k)

    def same(got, want):
        assert torch.equal(got, want)
    gives_up(lambda: ops.fp4_moe_mlp(x, r, *gu, *d, x_scale=0.02, h_scale=0.02), same)


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
    sc = dict(scale=g / 16) if fmt else {{}}
    for M, N, K in ((1, 128, 6144), (1, 2048, 8192), (33, 513, 7200), (100, 1000, 8224), (3, 60000, 256)):
        w, s = ops.fp4_quantize(randn(1, N, K, std=K ** -0.5), fmt, **sc)
        outs.append(ops.fp4_linear(randn(M, M, K), w, s, fmt, x_scale=g))
        ops.qsw_check_device_errors()
    for sizes, N, K in (([0, 40, 0, 9], 200, 6240), ([100, 0, 257, 900, 1, 700], 1793, 576), ([2500, 1, 5700], 300, 4128)):
        w, s = ops.fp4_quantize(randn(2, len(sizes), N, K, std=K ** -0.5), fmt, **sc)
        at = torch.tensor([0] + sizes).cumsum(0).int().cuda()
        outs.append(ops.fp4_grouped_linear(randn(3, sum(sizes), K), at, w, s, fmt, x_scale=g))
        ops.qsw_check_device_errors()
        back = at.flip(0).contiguous()      # all rows in no group
        ops.fp4_grouped_linear(randn(3, sum(sizes), K), back, w, s, fmt, x_scale=g)
        ops.qsw_check_device_errors()
    for T, E, k, H, I in ((5, 2, 2, 6208, 64), (2, 3, 2, 96, 6240), (700, 3, 2, 2112, 1056)):
        gu, gus = ops.fp4_quantize(randn(2, E, 2 * I, H, std=H ** -0.5), fmt, **sc)
        d, ds = ops.fp4_quantize(randn(3, E, H, I, std=I ** -0.5), fmt, **sc)
        r = ops.moe_route(randn(4, T, E, dt=torch.float32), k)
        outs.append(ops.fp4_moe_mlp(randn(5, T, H), r, gu, gus, d, ds, fmt, x_scale=g, h_scale=g))
        ops.qsw_check_device_errors()
assert all(torch.isfinite(o.float()).all() for o in outs)
torch.save([o.cpu() for o in outs], {path!r})
print("OK")
"""


def test_debug_build_gives_the_same_bits_in_every_form(tmp_path):
    """NaN-filled shared and tensor memory changes nothing, and no check fails."""
    got = []
    for debug in (False, True):
        path = str(tmp_path / f"{debug}.pt")
        r = subprocess.run([sys.executable, "-c", _SCRIPT.format(root=ROOT, debug=debug, path=path)],
                           capture_output=True, text=True, timeout=600, cwd=ROOT)
        assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout[-2000:] + r.stderr[-3000:]
        got.append(torch.load(path))
    assert all(torch.equal(a, b) for a, b in zip(*got))
