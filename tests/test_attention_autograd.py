"""The attention half has no derivatives: nothing that autograd follows is cut off silently, and it
learns of what is written."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_attention_ops import BF16, Step, dev, ints, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def parts():
    s = Step([(1, 40), (3, 70)], 4, 2, 64, 16)
    p = s.plan()
    k, v = randn(5, s.tokens, 2, 64), randn(6, s.tokens, 2, 64)
    return s, p, k, v, ops.rope_table(ops.rope_frequencies(64))


def test_tensors_that_require_grad_are_refused():
    s, p, k, v, table = parts()

    def follow(x):
        return x.detach().clone().requires_grad_()
    calls = {
        "rope x": lambda f: ops.rope(f(s.q), p.positions, table),
        "rope out": lambda f: ops.rope(s.q, p.positions, table, out=f(s.q)),
        "append k": lambda f: ops.kv_append(f(k), v, s.k, s.v, p.slots, p.positions, table),
        "append v": lambda f: ops.kv_append(k, f(v), s.k, s.v, p.slots, p.positions, table),
        "append k_cache": lambda f: ops.kv_append(k, v, f(s.k), s.v, p.slots, p.positions, table),
        "append v_cache": lambda f: ops.kv_append(k, v, s.k, f(s.v), p.slots, p.positions, table),
        "append q": lambda f: ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table, q=f(s.q)),
        "append q_out": lambda f: ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table, q=s.q, q_out=f(s.q)),
        "attend q": lambda f: ops.paged_attention(f(s.q), s.k, s.v, p),
        "attend k_cache": lambda f: ops.paged_attention(s.q, f(s.k), s.v, p),
        "attend v_cache": lambda f: ops.paged_attention(s.q, s.k, f(s.v), p),
        "attend out": lambda f: ops.paged_attention(s.q, s.k, s.v, p, out=f(s.q)),
    }
    for name, call in calls.items():
        with pytest.raises(RuntimeError, match="requires grad"):
            call(follow)
            pytest.fail(name)
        # followed by nobody: as ever
        with torch.no_grad():
            got = call(follow)
        want = call(lambda x: x.detach().clone())
        assert got is None and want is None or torch.equal(got, want), name


def test_autograd_learns_of_what_is_written():
    s, p, k, v, table = parts()
    q_out, out = torch.empty_like(s.q), torch.empty_like(s.q)

    def versions():
        return [t._version for t in (s.k, s.v, q_out, out)]
    before = versions()
    ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table, q=s.q, q_out=q_out)
    after = versions()
    assert [a > b for a, b in zip(after, before)] == [True, True, True, False]
    ops.paged_attention(s.q, s.k, s.v, p, out=out)
    assert [a > b for a, b in zip(versions(), after)] == [False, False, False, True]
    before = versions()
    ops.rope(s.q, p.positions, table, out=out)
    assert [a > b for a, b in zip(versions(), before)] == [False, False, False, True]
    # a value that a recorded product needs is overwritten: said, not used
    w = torch.randn(64, 64, device="cuda", dtype=BF16, requires_grad=True)
    y = s.k @ w
    ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_in_inference_mode_and_on_its_tensors():
    s, p, k, v, table = parts()
    want = s.attend(p)
    with torch.inference_mode():
        kc, vc = s.k.clone(), s.v.clone()
        q = ops.kv_append(k, v, kc, vc, p.slots, p.positions, table, q=s.q, q_out=s.q.clone())
        assert torch.equal(ops.paged_attention(s.q, s.k, s.v, p), want)
    again = ops.kv_append(k, v, kc, vc, p.slots, p.positions, table, q=s.q, q_out=q)
    assert torch.equal(again, ops.rope(s.q, p.positions, table))
