"""Frequencies for longer contexts, "ramp": every pair against its number of turns."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops


def plain_ramp(dim, base, factor, length, fast, slow):
    """Pair by pair in plain floats, as published (Peng et al. 2023, "YaRN"): the ramp's ends are
    the pairs that turn `fast` and `slow` times, rounded outwards, from 0 to dim - 1."""
    def pair_of(turns):
        return dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
    first, last = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), dim - 1)
    out = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        part = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
        out.append(f / factor * part + f * (1 - part))
    return out


@pytest.mark.parametrize("dim,base,length,fast,slow", [
    (128, 1e4, 4096, 32.0, 1.0), (128, 1e4, 65536, 32.0, 1.0), (128, 1e4, 131072, 32.0, 1.0), (128, 1e4, 262144, 32.0, 1.0),
    (128, 1e6, 32768, 32.0, 1.0), (64, 5e5, 1 << 20, 40.0, 2.0), (16, 100.0, 1 << 16, 32.0, 1.0), (8, 1e4, 512, 8.0, 3.0)])
@pytest.mark.parametrize("factor", [1.5, 4.0, 40.0])
def test_ramp_by_turns(dim, base, length, fast, slow, factor):
    got = ops.rope_frequencies(dim, base, "ramp", factor, length, fast, slow)
    plain = ops.rope_frequencies(dim, base)
    ratio, turns = plain / got, plain * length / (2 * math.pi)
    # (the formula in f64, a few roundings)
    assert got.tolist() == pytest.approx(plain_ramp(dim, base, factor, length, fast, slow), rel=1e-12)
    for r, t in zip(ratio.tolist(), turns.tolist()):
        # between the two counts a pair is neither left nor interpolated in full
        if slow * 1.0001 < t < fast * 0.9999:
            assert 1 < r < factor, (r, t)
    # beyond them (the ends are rounded to whole pairs, one pair outwards)
    step = base ** (2.0 / dim)
    assert torch.allclose(ratio[turns > fast * step], torch.ones(1, dtype=torch.float64))
    assert torch.allclose(ratio[turns < slow / step], torch.full((1,), factor, dtype=torch.float64))


@pytest.mark.parametrize("length", [1, 3, 6])
def test_ramp_where_no_pair_turns_often_enough(length):
    """All pairs turn less than once: all are interpolated."""
    got = ops.rope_frequencies(64, 1e4, "ramp", 4.0, length)
    assert torch.allclose(ops.rope_frequencies(64, 1e4) / got, torch.full((1,), 4.0, dtype=torch.float64))


def test_ramp_where_every_pair_turns_often_enough():
    got = ops.rope_frequencies(16, 10.0, "ramp", 4.0, 1 << 20)
    assert torch.equal(got, ops.rope_frequencies(16, 10.0))
