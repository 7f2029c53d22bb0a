"""Pairs of kv heads in one item, alone and among sequences with few and with many rows: waits
that run out, the debug build; and the debug build over infinities that only some rows see."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_attention_ops import Step, dev  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PAIRS = {
    "pairs": ([(17 + i % 47, 100 + 3 * i) for i in range(160)], 4, 2, 64),
    "pairs_128": ([(5 + i % 28, 60 + 5 * i) for i in range(90)], 16, 4, 128),
    "pairs_and_others": ([(33, 300 + i) for i in range(90)] + [(1, 400), (300, 900), (3, 3), (200, 200)], 4, 2, 128),
}
# a row tile of which one warp has rows, as of drafted tokens
TILES = {
    "tile_32_rows": ([(8, 700)], 8, 2, 64),
    "tile_20_rows_split": ([(5, 9000)], 8, 2, 128),
}


def paired(s, plan):
    """Sequences whose items are two kv heads each."""
    records = plan.work[32:32 + 32 * len(s.seqs)].view(torch.int32).view(-1, 8)
    return int((records[:, 4] >= 1 << 16).sum())


@pytest.mark.parametrize("form", {**PAIRS, **TILES})
def test_waits_that_run_out(form):
    """The first keys never arrive: given up within the limit, told, and the next call is right."""
    seqs, heads, kv_heads, D = {**PAIRS, **TILES}[form]
    s = Step(seqs, heads, kv_heads, D, 16)
    assert (paired(s, s.plan()) > 0) is (form in PAIRS)
    want = s.check()
    ops.qsw_check_device_errors()
    try:
        ops.qsw_set_wait_timeout_ns(2_000_000)
        ops.qsw_debug_withhold_next_attention()
        s.attend()
        with pytest.raises(ops.QswError) as e:
            ops.qsw_check_device_errors()
        assert ops.STATUS[e.value.code] == "QSW_ERR_TIMEOUT"
        ops.qsw_check_device_errors()
    finally:
        ops.qsw_set_wait_timeout_ns(4_000_000_000)
    for _ in range(3):
        assert torch.equal(s.attend(), want)
        ops.qsw_check_device_errors()


_SCRIPT = r"""
import math, sys
sys.path.insert(0, {root!r})
import torch
from quantized_swiglu_mlp_gb300 import build, ops
if {debug}:
    ops.load_library(build.DEBUG_LIB_PATH)
assert ops.qsw_debug_build() == {debug}
torch.cuda.set_device(0)
from tests.test_attention_forms import PAIRS, TILES
from tests.test_attention_ops import Step
from tests.test_attention_unseen import SHAPES
outs = []
for dt in (torch.bfloat16, torch.float16):
    for seqs, heads, kv_heads, D in [*PAIRS.values(), *TILES.values()]:
        for page, window in ((8, 0), (48, 70)):
            s = Step(seqs, heads, kv_heads, D, page, dt=dt, window=window)
            outs.append(s.attend().cpu())
    for seqs, heads, kv_heads, D, page, window in SHAPES.values():
        s = Step(seqs, heads, kv_heads, D, page, dt=dt, window=window)
        for b, (n, total) in enumerate(seqs):
            for at, value in ((total - 1, math.inf), (total - 1 - n // 2, math.nan), (total - n, -math.inf)):
                s.v[int(s.table[b, at // page]), :, at % page, b % D] = value
        outs.append(s.attend().nan_to_num(7.0).cpu())
        ops.qsw_check_device_errors()
torch.save(outs, sys.argv[1])
"""


def test_debug_build_gives_the_same_bits(tmp_path):
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
