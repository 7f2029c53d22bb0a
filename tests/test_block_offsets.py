"""Grouped products with offset tables that are not ascending: taken as the header
says, and nothing outside the call's own memory changes.  (That the tiles of
such tables fit in their records is shown on the CPU, in test_tiles_cpu.py.)"""
from __future__ import annotations

import random

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_block_ops import BF16, SCALE, dev, formats, randn, weight  # noqa: F401
from tests.test_tiles_cpu import raised

pytestmark = pytest.mark.gpu


def tables(groups, rows, seed):
    rng = random.Random(seed)
    yield [(e & 1) * rows for e in range(groups + 1)]
    yield [((e + 1) & 1) * rows for e in range(groups + 1)]
    yield sorted((rng.randint(0, rows) for _ in range(groups + 1)), reverse=True)
    yield [rng.randint(-rows, 2 * rows) for _ in range(groups + 1)]
    yield [rows // 3 * (e % 3) + (e // 3) for e in range(groups + 1)]


@formats
@pytest.mark.parametrize("rows,groups,N,K", [
    (2, 64, 128, 256), (16, 40, 200, 512),             # x quantised in the product
    (8192, 64, 2048, 64), (50, 4, 128, 256), (700, 600, 130, 96), (90, 1024, 128, 64),   # single CTAs
    (8192, 32, 2048, 64), (1000, 5, 10000, 96),        # CTA pairs
    (5, 8, 256, 6240), (100, 3, 384, 6176),            # K split over a cluster
])
def test_tables_that_go_backwards(dev, fmt, rows, groups, N, K):  # noqa: F811
    x = randn(rows + N, rows, K)
    w, ws, wg, _ = weight(11, min(groups, 8), N, K, fmt)
    each = torch.arange(groups, device="cuda") % w.shape[0]
    w, ws, wg = w[each], ws[each], wg[each]
    for table in tables(groups, rows, rows + groups):
        got, want = (torch.full((rows + 64, N), 7.0, dtype=BF16, device="cuda") for _ in range(2))
        for t, out in ((table, got), (raised(table, rows), want)):
            ops.fp4_grouped_linear(x, torch.tensor(t, dtype=torch.int32, device="cuda"), w, ws, fmt, x_scale=SCALE[fmt],
                                   w_scale=wg, out=out[32:32 + rows])
        ops.qsw_check_device_errors()
        assert torch.equal(got, want)
        lo, hi = raised(table, rows)[0], raised(table, rows)[-1]
        assert (got[:32 + lo] == 7).all() and (got[32 + hi:] == 7).all()


@formats
@pytest.mark.parametrize("T,E,k,H,I", [(1, 16, 4, 256, 96), (20, 8, 2, 96, 160), (400, 6, 4, 288, 96), (3, 5, 2, 6176, 64)])
def test_expert_mlp_with_a_foreign_routing(dev, fmt, T, E, k, H, I):  # noqa: F811
    """Offsets, slots and orders that are not the routing's: the values are unspecified,
    the memory around the result keeps its own, and the next call is right."""
    x = randn(T + H, T, H)
    gu, gus, gug, _ = weight(8, E, 2 * I, H, fmt)
    d, ds, dg, _ = weight(9, E, H, I, fmt)

    def mlp(r, out=None):
        return ops.fp4_moe_mlp(x, r, gu, gus, d, ds, fmt, x_scale=SCALE[fmt], h_scale=SCALE[fmt], gu_scale=gug,
                               d_scale=dg, out=out)
    r = ops.moe_route(randn(T + E, T, E, dt=torch.float32), k)
    want = mlp(r)
    buf = torch.full((T + 64, H), 7.0, dtype=BF16, device="cuda")
    junk = torch.randint(-2 ** 31, 2 ** 31 - 1, (T * k,), dtype=torch.int32, device="cuda")
    for table in tables(E, T * k, T):
        bad = r._replace(offsets=torch.tensor(table, dtype=torch.int32, device="cuda"))
        for route in (bad, bad._replace(order=junk), bad._replace(slots=junk.view(T, k)), bad._replace(ids=junk.view(T, k))):
            mlp(route, buf[32:32 + T])
            ops.qsw_check_device_errors()
            assert (buf[:32] == 7).all() and (buf[32 + T:] == 7).all()
    assert torch.equal(mlp(r), want)
