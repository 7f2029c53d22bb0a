"""Routing weights where the scores are far out in f32's range."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import block_ref as ref
from tests.test_block_ops import BF16, F16, check, dev, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("mean", [-60, -88, -95, -103, -110, -300, 60, 120])
@pytest.mark.parametrize("renormalize", [True, False])
def test_sigmoid_of_far_logits(dev, dt, mean, renormalize):  # noqa: F811
    """Scores whose exponentials pass f32's range keep their ratios."""
    T, E, k = 70, 40, 6
    logits = (randn(5, T, E, dt=torch.float32, std=3.0) + mean).to(dt)
    logits[3, 5:] = -torch.inf
    logits[4] = -torch.inf
    logits[5] = torch.finfo(dt).min       # a mask: below any score, counts as 0
    r = ops.moe_route(logits, k, scoring=ops.ROUTE_SIGMOID, renormalize=renormalize)
    ids, w, offsets, slots, order = ref.route(logits, k, True, renormalize)
    assert torch.equal(r.ids.long(), ids) and torch.equal(r.slots.long(), slots)
    # as test_route: expf within 2 ulp of arguments rounded once, f32 sums; values below 2^-126 lose bits
    check(r.weights, w, w * (E + 64) * 2.0 ** -23 + 1e-37)
    assert not r.weights[4].any() and not r.weights[5].any()
    if renormalize:
        rest = torch.arange(T, device="cuda") > 5
        assert (r.weights[rest].sum(1) - 1).abs().max() < 1e-5


def test_routings_one_after_another(dev):  # noqa: F811
    """Many routings in a row over the same memory, choices and sort overlapping: each reads its own ids."""
    T, E, k = 3000, 24, 4
    logits = [randn(s, T, E, dt=torch.float32) for s in range(3)]
    want = [ref.route(v, k) for v in logits]
    x, got = torch.empty_like(logits[0]), []

    def round_trip():
        for v in logits:
            x.copy_(v)
            r = ops.moe_route(x, k)
            got.append([t.clone() for t in (r.ids, r.offsets, r.slots, r.order)])
            del r        # the next routing takes the same memory
    round_trip()
    got.clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(5):
            round_trip()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for i, parts in enumerate(got):
            ids, _, offsets, slots, order = want[i % 3]
            for a, b in zip(parts, (ids, offsets, slots, order)):
                assert torch.equal(a.long(), b)
