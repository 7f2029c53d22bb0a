"""Attention half: results that share memory with what is read, or with themselves."""
from __future__ import annotations

import ctypes

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_attention_ops import BF16, Step, dev, ints, randn  # noqa: F401

pytestmark = pytest.mark.gpu

INVALID = 1


def attend_at(s, plan, q, out):
    """qsw_paged_attention itself, `out` at an address within q's buffer or elsewhere."""
    lib = ops.load_library()
    T, H, D = q.shape
    pages, kv_heads, page, _ = s.k.shape
    strides = [(ctypes.c_int64 * 3)(*x.stride()[:3]) for x in (s.k, s.v)]
    cache = ops.KvCache(s.k.data_ptr(), s.v.data_ptr(), pages, kv_heads, page, *strides)
    B, most = s.table.shape
    need = lib.qsw_paged_attention_workspace_bytes(B, T, H, kv_heads, D, most * page)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    heads = ops.Heads(q.data_ptr(), q.stride(0), q.stride(1))
    return lib.qsw_paged_attention(ctypes.byref(heads), ctypes.byref(cache), s.table.data_ptr(), s.table.stride(0), most,
                                   plan.work.data_ptr(), B, T, H, D, 0, s.scale, 0, out, ws.data_ptr(), need,
                                   torch.cuda.current_stream().cuda_stream)


def test_attention_refuses_results_over_its_queries():
    heads, D = 4, 64
    s = Step([(3, 40), (6, 90)], heads, 2, D, 16)
    T, row = s.tokens, 2 * D             # bytes of a head
    plan = s.plan()
    want = s.attend(plan)
    with pytest.raises(ops.QswError):
        s.attend(plan, out=s.q)
    for shift in (-T * heads * row + row, -row, 0, row, T * heads * row - row):
        buf = torch.zeros(4 * T * heads * D, dtype=BF16, device="cuda")
        q = buf[T * heads * D:2 * T * heads * D].view(T, heads, D)
        q.copy_(s.q)
        assert attend_at(s, plan, q, q.data_ptr() + shift) == INVALID
        assert torch.equal(q, s.q)
    # side by side
    for shift in (-T * heads * row, T * heads * row):
        buf = torch.zeros(4 * T * heads * D, dtype=BF16, device="cuda")
        q = buf[T * heads * D:2 * T * heads * D].view(T, heads, D)
        q.copy_(s.q)
        assert attend_at(s, plan, q, q.data_ptr() + shift) == 0
        at = T * heads * D + shift // 2
        assert torch.equal(buf[at:at + T * heads * D].view(T, heads, D), want)


@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_attention_into_the_room_between_its_queries(order):
    """q's rows with room for the whole result before, between and behind the tokens, or heads:
    exactly the places that meet none of them are taken."""
    heads, D = 2, 64
    s = Step([(3, 40)], heads, 1, D, 16)
    plan, T = s.plan(), 3
    want = s.attend(plan)
    size = T * heads * D                 # elements of the result
    gap = 2 * size
    n = T if order == "tokens" else heads
    inner = heads if order == "tokens" else T
    buf = torch.zeros(gap + n * (inner * D + gap), dtype=BF16, device="cuda")
    outer = inner * D + gap
    strides = (outer, D, 1) if order == "tokens" else (D, outer, 1)
    q = buf.as_strided((T, heads, D), strides, gap)
    held = torch.zeros_like(buf, dtype=torch.bool)
    held.as_strided((T, heads, D), strides, gap).fill_(True)
    for at in range(0, buf.numel() - size + 1, D // 2):
        buf.zero_()
        q.copy_(s.q)
        free = not bool(held[at:at + size].any())
        assert (attend_at(s, plan, q, buf.data_ptr() + 2 * at) == 0) is free, at
        assert torch.equal(q, s.q)
        if free:
            assert torch.equal(buf[at:at + size].view(T, heads, D), want)


def test_outputs_whose_rows_share_memory_are_refused():
    """Expanded outputs of rope and kv_append, and those that cover other rows of the input;
    the input's own place and its neighbours in one buffer are fine."""
    T, H, D = 5, 3, 64
    x = randn(1, T, H, D)
    table = ops.rope_table(ops.rope_frequencies(D))
    pos = ints(range(T))
    want = ops.rope(x, pos, table)
    kc, vc = (torch.zeros(2, H, 8, D, dtype=BF16, device="cuda") for _ in range(2))

    def into(x, out):
        return (lambda: ops.rope(x, pos, table, out=out),
                lambda: ops.kv_append(x, x, kc, vc, pos, pos, table, q=x, q_out=out))
    buf = torch.zeros(T + 1, 2 * H, D, dtype=BF16, device="cuda")
    view = buf[:T, :H]
    view.copy_(x)
    for source, out in ((x, torch.zeros(T, 1, D, dtype=BF16, device="cuda").expand(T, H, D)),
                        (x, torch.zeros(1, H, D, dtype=BF16, device="cuda").expand(T, H, D)),
                        (view, buf[1:, :H]), (view, buf[:T, 1:H + 1])):
        for call in into(source, out):
            with pytest.raises(ops.QswError):
                call()
    assert torch.equal(view, x)
    for out in (buf[:T, H:], view):
        for call in into(view, out):
            view.copy_(x)
            call()
            assert torch.equal(out, want)
