"""Infinities and NaN among values that some rows of a tile see and others do not: who does not
see them keeps every bit, who does gets them, and the call takes no longer than it has to."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_attention_ops import BF16, F16, Step, dev  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = {          # sequences, heads, kv heads, D, page size, window
    "few": ([(3, 100), (4, 4), (2, 700)], 4, 1, 64, 16, 0),
    "few_window": ([(4, 300), (5, 5), (3, 64)], 6, 2, 80, 8, 30),
    "few_split": ([(4, 20000)], 8, 2, 128, 64, 0),
    "few_dense": ([(16, 16), (9, 40)], 1, 1, 128, 24, 3),
    "tile": ([(70, 300), (1, 20)], 4, 2, 128, 16, 0),
    "two_tiles": ([(150, 700)], 2, 1, 64, 128, 0),
    "one_head_each": ([(300, 300)], 2, 2, 128, 8, 0),
    "window": ([(200, 900)], 4, 2, 64, 48, 100),
    "split": ([(30, 9000)], 4, 1, 128, 32, 0),
    "pairs": ([(20 + i % 9, 150 + 9 * i) for i in range(120)], 8, 2, 64, 16, 0),
}


def seers(s, b, at):
    """bool [T]: tokens of sequence b that see its key `at`."""
    n, total = s.seqs[b]
    pos = torch.arange(total - n, total, device="cuda")
    sees = pos >= at
    if s.window:
        sees &= pos < at + s.window
    rows = torch.zeros(s.tokens, dtype=torch.bool, device="cuda")
    rows[s.offsets[b]:s.offsets[b + 1]] = sees
    return rows


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("name", SHAPES)
def test_who_does_not_see_them_keeps_every_bit(name, dt):
    seqs, heads, kv_heads, D, page, window = SHAPES[name]
    s = Step(seqs, heads, kv_heads, D, page, dt=dt, window=window)
    clean = s.attend()
    group, held = heads // kv_heads, s.v.clone()
    odd = torch.full((s.tokens, heads, D), 0, dtype=torch.float64, device="cuda")
    for b in {0, len(seqs) - 1, len(seqs) // 2}:
        n, total = seqs[b]
        # (the last one at a place is what lies there)
        places = {(at, kv, d): value for at, kv, d, value in [
                (total - 1, 0, 0, math.inf), (total - 1, kv_heads - 1, D - 1, math.nan), (total - n, 0, 3, -math.inf),
                (total - 1 - n // 2, kv_heads - 1, D // 2, -math.inf), (total - 1 - n // 2, 0, 3, math.inf),
                (max(0, total - n - window // 2), 0, 5, math.inf)]}
        for (at, kv, d), value in places.items():
            s.v[int(s.table[b, at // page]), kv, at % page, d] = value
            rows = seers(s, b, at)
            odd[rows, kv * group:(kv + 1) * group, d] += value
    got = s.attend()
    fine = odd == 0
    assert torch.equal(got[fine], clean[fine])
    want = odd[~fine]
    same = (got[~fine].double() == want) | (got[~fine].isnan() & want.isnan())
    assert same.all()
    # whole rows
    s.v.copy_(held)
    b = len(seqs) - 1
    at = seqs[b][1] - 1 - seqs[b][0] // 3
    s.v[int(s.table[b, at // page]), :, at % page] = math.inf
    got, rows = s.attend(), seers(s, b, at)
    assert torch.equal(got[~rows], clean[~rows]) and (got[rows] == math.inf).all()
    ops.qsw_check_device_errors()


def test_a_key_of_no_weight_times_infinity_is_nan():
    """Scores of -infinity: weight 0, and 0 times infinity."""
    for tokens in (4, 40):
        s = Step([(tokens, 100)], 2, 1, 64, 16)
        row = int(s.table[0, 98 // 16]), 0, 98 % 16
        s.q[..., 0] = 1.0
        s.k[row + (0,)] = -math.inf
        s.k[row + (slice(1, None),)] = 0.0
        s.v[row + (7,)] = math.inf
        got = s.attend()
        assert got[-2:, :, 7].isnan().all() and got[:-2].isfinite().all()
        assert got[..., :7].isfinite().all() and got[..., 8:].isfinite().all()


def milliseconds(call):
    for _ in range(2):
        call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("n,total,many", [(8192, 8192, 4), (8192, 8192, 8192), (64, 60000, 4), (3, 60000, 4)])
def test_they_hold_nobody_up(n, total, many):
    """`many` keys at the end with infinite values.  The time of the usual call, and what few tiles an item at
    most add, which does not grow with the history: some ms, where whole rows computed again took over 100."""
    s = Step([(n, total)], 16, 4, 128, 64)
    plan = s.plan()
    clean = milliseconds(lambda: s.attend(plan))
    p = torch.arange(total - many, total, device="cuda")
    s.v[s.table[0].long()[p // 64], :, p % 64] = math.inf
    assert milliseconds(lambda: s.attend(plan)) < clean + 20.0


@pytest.mark.parametrize("seqs,window", [([(5, 3), (1, 30)], 0), ([(40, 25), (2, 9)], 0), ([(40, 25), (6, 2)], 4), ([(300, 180)], 0)])
def test_tokens_before_the_first_key(seqs, window):
    """More new tokens than the length counts: those before its first key see nothing, whatever
    the others' keys hold, among pages that are not in the cache."""
    s = Step(seqs, 4, 2, 64, 8, window=window)
    s.table[0, 1] = -1
    n, total = seqs[0]
    clean = s.attend()
    assert (clean[:n - total] == 0).all()
    for at in (0, total - 1):
        s.v[int(s.table[0, at // 8]), 1, at % 8, 5] = math.inf
    got = s.attend()
    rows = seers(s, 0, 0) | seers(s, 0, total - 1)
    assert (got[rows][:, 2:, 5] == math.inf).all()
    got[:, 2:, 5] = torch.where(rows[:, None], clean[:, 2:, 5], got[:, 2:, 5])
    assert torch.equal(got, clean)
