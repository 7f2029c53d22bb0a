"""Attention and its plan where a tile, a list or a type ends."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_attention_ops import Step, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def poison_unseen(s, page_size, value):
    """Everything in the cache but the sequences' own keys and values := value."""
    k, v = s.k.clone(), s.v.clone()
    s.k.fill_(value), s.v.fill_(value)
    for b, total in enumerate(s.lengths):
        p = torch.arange(total, device="cuda")
        rows = s.table[b].long()[p // page_size], slice(None), p % page_size
        s.k[rows], s.v[rows] = k[rows], v[rows]


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens,group", [(5, 4), (17, 1), (4, 8), (9, 7)])
@pytest.mark.parametrize("behind", [31, 36, 96])
def test_warps_without_rows_take_out_what_lies_behind_the_end(tokens, group, D, value, behind):
    """17 to 63 rows: some warps of a row tile have none, but all take out rows of V behind the
    sequence's end, here among the last tile's first 64 keys.  Once alone, once as pairs of
    kv heads among many sequences."""
    for seqs in ([(tokens, 128 + behind)], [(tokens, 128 * (i % 3 + 1) + behind) for i in range(170)]):
        s = Step(seqs, 2 * group, 2, D, 128, spare=3)
        clean = s.check() if len(seqs) == 1 else s.attend()
        poison_unseen(s, 128, value)
        for _ in range(5):
            assert torch.equal(s.attend(), clean)
    ops.qsw_check_device_errors()


@pytest.mark.parametrize("lengths", [[0, 0, 0], [-3, 0, -2 ** 31]])
@pytest.mark.parametrize("group", [1, 4, 32])
def test_tokens_without_any_key(group, lengths):
    """Lengths of 0, as in a step captured before the first request, with a table wide enough to
    split histories: positions and slots of nobody, and zeros in both lists."""
    s = Step([(1, 900), (70, 900), (3, 900)], 2 * group, 2, 64, 16)
    s.lengths = lengths
    s.k.fill_(math.nan), s.v.fill_(math.nan)
    p = s.plan()
    assert (p.positions == -1).all() and (p.slots == -1).all()
    # word 0 and 1: the items of both lists, one per row tile and kv head, nothing split
    rows = [n * group for n in (1, 70, 3)]
    items = p.work[:12].view(torch.int32).tolist()
    assert items == [2 * sum(-(-r // 16) for r in rows if r <= 16), 2 * sum(-(-r // 256) for r in rows if r > 16), 0]
    assert (s.attend(p) == 0).all()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 3, 9], ids=["few", "twelve", "tile"])
@pytest.mark.parametrize("late", [False, True], ids=["first", "last"])
@pytest.mark.parametrize("score,keys", [(12, 250), (15, 250), (18, 250), (12, 40000), (18, 1 << 18), (20, 1 << 20)])
def test_a_long_tail_behind_one_large_weight(dt, tokens, late, score, keys):
    """One key with nearly all the weight and a value of 0, and many with e^-score of it each and
    a value of 1024: what is left is their sum, though in f16 each would be below 2^-14 or 0."""
    D, group, value = 64, 4, 1024
    s = Step([(tokens, keys)], group, 1, D, 256, dt=dt)
    s.q.zero_(), s.k.zero_()
    s.q[..., 0] = 8.0
    s.v.fill_(value)
    at = keys - tokens if late else 0         # (every token sees it)
    row = int(s.table[0, at // 256]), 0, at % 256
    s.k[row + (0,)] = float(score)            # 8 score / 8
    s.v[row] = 0.0
    got = s.attend().double()
    n = torch.arange(keys - tokens, keys, device="cuda").double()      # keys seen but the large one
    tail = n * math.exp(-score)
    want = (value * tail / (1 + tail))[:, None, None].expand_as(got)
    half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    # scores are exact but for their factors' rounding (scale log2 e, and the product: 2^-23 of it, times
    # ln 2 and a weight); weights: half a step, the exponential's 2^-21, and in f16 half of the smallest step
    # 2^-24 against weights of 2^14 (few rows) or 2^7 (tiles) for the large one; f32 sums of
    # up to 2^20 equal terms, 128 or 64 at a time: 2^-24 (n / 64 + 70) of them; the end's half step
    rel = 2.0 ** -22 * score + half + 2.0 ** -21 + 2.0 ** -24 * (keys / 64 + 70) + half
    least = 0.0 if dt != torch.float16 else 2.0 ** -25 * (2.0 ** -14 if tokens * group <= 16 else 2.0 ** -7)
    err = (got - want).abs()
    bound = want * rel + least * value * n[:, None, None]
    assert (err <= bound).all(), (float(err.max()), float((err / bound).max()))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens", [3, 200], ids=["few", "tile"])
@pytest.mark.parametrize("step", [64.0, 4096.0, 32768.0])
@pytest.mark.parametrize("order", ["up", "down", "twice"])
def test_scores_far_from_zero(dt, tokens, step, order):
    """Scores of up to 2^24, exact in f32, hundreds apart: all the weight on the largest one that a row
    sees, or on two equal ones, wherever the bases of the rows lie."""
    keys, D = 250, 64
    s = Step([(tokens, keys)], 4, 2, D, 16, dt=dt)
    s.scale = 2.0
    s.q.zero_(), s.k.zero_()
    s.q[..., 0] = step
    p = torch.arange(keys, device="cuda")
    at = {"up": p, "down": -p, "twice": p // 2}[order]
    rows = s.table[0].long()[p // 16], slice(None), p % 16
    k = s.k[rows]
    k[..., 0] = at[:, None].to(dt)
    s.k[rows] = k
    v = s.v[rows].double()                                           # [keys, kv_heads, D]
    pos = torch.arange(keys - tokens, keys, device="cuda")
    if order == "up":
        want = v[pos]
    elif order == "down":
        want = v[torch.zeros_like(pos)]
    else:
        want = torch.where((pos % 2 == 0)[:, None, None], v[pos], (v[pos] + v[pos - 1]) / 2)
    got = s.attend().double().unflatten(1, (2, 2))
    # weights of one or two equal powers of two, or their roundings alike: v's rounding at the end, and
    # with two a sum of the same size (f32 between: 2^-20)
    half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    err, size = (got - want[:, :, None]).abs(), v.abs().amax()
    assert (err <= want[:, :, None].abs() * half * 2 + size * (2.0 ** -20 + 2 * half)).all(), float(err.max())
