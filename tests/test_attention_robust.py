"""Attention operators: waits that run out, the debug build, many sequences, offsets beyond 32
bits, the block they make up."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import attention_ref as ref
from tests.test_attention_ops import BF16, Step, check, dev, ints, randn  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FORMS = {
    "rows_16": ([(1, 300), (1, 40)], 8, 2, 128),
    "rows_32": ([(8, 700)], 8, 2, 64),
    "tiles": ([(100, 300)], 4, 2, 128),
    "tiles_64": ([(300, 1000)], 4, 2, 64),
    "both": ([(1, 300), (200, 900), (3, 3)], 4, 2, 128),
    "split": ([(1, 20000)], 8, 2, 128),
}


@pytest.mark.parametrize("form", FORMS)
def test_waits_that_run_out(form):
    """An attention whose first keys never arrive gives up within the wait limit; the
    status says so, nothing traps, and the next call is right."""
    s = Step(FORMS[form][0], *FORMS[form][1:], 16)
    want = s.check()
    ops.qsw_check_device_errors()
    try:
        ops.qsw_set_wait_timeout_ns(2_000_000)
        ops.qsw_debug_withhold_next_attention()
        s.attend()
        with pytest.raises(ops.QswError) as e:
            ops.qsw_check_device_errors()
        assert ops.STATUS[e.value.code] == "QSW_ERR_TIMEOUT"
        ops.qsw_check_device_errors()      # the word is cleared
    finally:
        ops.qsw_set_wait_timeout_ns(4_000_000_000)
    for _ in range(3):
        assert torch.equal(s.attend(), want)
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
from tests.test_attention_ops import Step, randn, ints
from tests.test_attention_robust import FORMS
outs = []
for dt in (torch.bfloat16, torch.float16):
    for seqs, heads, kv_heads, D in [*FORMS.values(), ([(5, 90), (33, 33), (0, 7)], 6, 1, 80), ([(2, 1)], 2, 2, 8)]:
        for page, window in ((8, 0), (48, 100)):
            s = Step(seqs, heads, kv_heads, D, page, dt=dt, window=window)
            p = s.plan()
            k, v = randn(5, s.tokens, kv_heads, D, dt=dt), randn(6, s.tokens, kv_heads, D, dt=dt)
            q = ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, ops.rope_table(ops.rope_frequencies(D)), q=s.q)
            outs += [q.cpu(), s.k.cpu(), s.v.cpu(), s.attend(p).cpu()]
            ops.qsw_check_device_errors()
torch.save(outs, sys.argv[1])
"""


def test_debug_build_gives_the_same_bits(tmp_path):
    """Every byte of staging and tensor memory starts as NaN there, and copies and rows are
    checked."""
    outs = []
    for debug in (False, True):
        path = str(tmp_path / f"{debug}.pt")
        r = subprocess.run([sys.executable, "-c", _SCRIPT.format(root=ROOT, debug=debug), path], capture_output=True,
                           text=True, timeout=900, cwd=ROOT)
        assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
        outs.append(torch.load(path))
    assert len(outs[0]) == len(outs[1])
    for i, (a, b) in enumerate(zip(*outs)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("seqs", [[(1, 1 + 7 * i % 60) for i in range(3000)],
                                  [(i % 4, i % 4 + 11 * i % 300) for i in range(1200)],
                                  [(40 if i % 97 == 0 else i % 2, 50 + i % 90) for i in range(1100)]],
                         ids=["decode", "few_tokens", "chunks_among_them"])
def test_many_sequences(seqs):
    Step(seqs, 2, 1, 64, 8).check()


def test_the_most_sequences():
    """65536 of them, one token each, of 1 to 8 keys."""
    B, D = 65536, 64
    lengths = (torch.arange(B, device="cuda") % 8 + 1).int()
    k, v = (randn(i, B, 1, 8, D) for i in (1, 2))
    q = randn(3, B, 1, D, std=2.5)
    table = torch.randperm(B, device="cuda").int()[:, None]
    plan = ops.paged_plan(torch.arange(B + 1, device="cuda").int(), lengths, table, k, B, 1)
    assert torch.equal(plan.positions, lengths - 1)
    assert torch.equal(plan.slots, table[:, 0] * 8 + lengths - 1)
    out = ops.paged_attention(q, k, v, plan)
    pick = torch.arange(0, B, 997, device="cuda")
    want, bound = ref.attention(q[pick], k, v, list(range(len(pick) + 1)), lengths[pick].tolist(), table[pick], D ** -0.5)
    check(out[pick], want, bound)


@pytest.mark.parametrize("n", [1, 12, 140])
def test_offsets_beyond_32_bits(n):
    """A cache of 5 GB a side, whose last pages lie 2^31 elements and more behind its first."""
    KV, P, D, heads = 8, 64, 128, 16
    pages = (1 << 31) // (KV * P * D) * 5 // 4
    k, v = (torch.empty(pages, KV, P, D, dtype=BF16, device="cuda") for _ in range(2))
    table = ints([[pages - 1, 0, pages - 7, 3, pages // 2]])
    total = 290
    slots = torch.tensor([int(table[0, p // P]) * P + p % P for p in range(total)], device="cuda").int()
    kn, vn = randn(1, total, KV, D), randn(2, total, KV, D)
    rope = ops.rope_table(ops.rope_frequencies(D))
    pos = torch.arange(total, device="cuda").int()
    ops.kv_append(kn, vn, k, v, slots, pos, rope)
    assert torch.equal(v[table[0].long()].transpose(1, 2).flatten(0, 1)[:total], vn)
    assert torch.equal(k[table[0].long()].transpose(1, 2).flatten(0, 1)[:total], ops.rope(kn, pos, rope))
    q = randn(3, n, heads, D, std=2.5)
    plan = ops.paged_plan(ints([0, n]), ints([total]), table, k, n, heads)
    got = ops.paged_attention(q, k, v, plan)
    want, bound = ref.attention(q, k, v, [0, n], [total], table, D ** -0.5)
    check(got, want, bound)


@pytest.mark.parametrize("n", [1, 70])
def test_a_million_keys(n):
    Step([(n, 1 << 20)], 2, 1, 64, 256).check()


def test_many_tokens_of_short_sequences_and_a_long_prompt():
    Step([(4100, 4100), (1, 9), (2, 2000)], 2, 1, 64, 64).check()


@pytest.mark.parametrize("prompts,head_dim,heads,kv_heads", [((70, 9), 64, 8, 2), ((1, 260), 128, 4, 4), ((33,), 80, 6, 1)])
def test_attention_block_example(prompts, head_dim, heads, kv_heads):
    from examples import attention_block
    off = attention_block.run(hidden=512 if head_dim != 80 else 320, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                              prompts=prompts)
    # activations rounded to 4 bits twice: half a step of e2m1 is at most a quarter of a value
    # (between 1 and 1.5, less elsewhere), about 0.09 in the mean square; the norms before and the
    # softmax between do not enlarge it
    assert max(off) < 0.125, off


@pytest.mark.parametrize("heads,kv_heads,D,page,window", [(8, 8, 128, 16, 0), (12, 4, 64, 8, 0), (16, 2, 80, 24, 150), (4, 2, 128, 128, 0),
                                                          (6, 3, 64, 16, 0)])
def test_many_sequences_of_a_few_dozen_rows(heads, kv_heads, D, page, window):
    """More items than run at once, each of half a row tile at most: two kv heads an item where
    they are even in number; with longer and shorter sequences among them."""
    group = heads // kv_heads
    seqs = [(max(1, (33 + i * 7 % 96) // group), 40 + 53 * i % 700) for i in range(100)] + [(300, 500), (1, 900), (40, 6000), (0, 3)]
    seqs = [(n, max(n, total)) for n, total in seqs]
    s = Step(seqs, heads, kv_heads, D, page, window=window)
    clean = s.check()
    # what only a last token sees, of one head of each pair
    for b in (3, 50):
        p = seqs[b][1] - 1
        s.v[int(s.table[b, p // page]), kv_heads - 1, p % page] = float("nan")
    got, (want, bound) = s.attend(), s.want()
    check(got, want, bound)
    rows = torch.ones(s.tokens, dtype=torch.bool, device="cuda")
    for b in (3, 50):
        rows[s.offsets[b]:s.offsets[b + 1]] = False
    assert torch.equal(got[rows], clean[rows])


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (32, 1), (17, 1)])
def test_fewer_tokens_than_sequences_unevenly(heads, kv_heads):
    """The sizes look like one token a sequence; one of them has them all."""
    Step([(0, 7)] * 20 + [(30, 300)] + [(0, 0)] * 20, heads, kv_heads, 128, 16).check()
