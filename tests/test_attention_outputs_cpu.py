"""Results of rope and kv_append at any strides: refused where rows share memory, by brute
force over small sizes.  (What passes ends in the error that a call without a device gives.)"""
from __future__ import annotations

import itertools
import random

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops  # noqa: F401
from tests.test_abi_cpu import FAKE, INVALID, lib  # noqa: F401
from tests.test_attention_abi_cpu import CUDA, cache, heads

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="what is accepted would be launched")

D = 8
AT = FAKE + 0x8000


def elements(at, T, H, strides):
    return [range(at + t * strides[0] + h * strides[1], at + t * strides[0] + h * strides[1] + D)
            for t, h in itertools.product(range(T), range(H))]


def share(a, b):
    return a.start < b.stop and b.start < a.stop


def allowed(T, H, x_at, x, out_at, out):
    rows, other = elements(out_at, T, H, out), elements(x_at, T, H, x)
    if any(share(a, b) for a, b in itertools.combinations(rows, 2)):
        return False
    alike = (T == 1 or x[0] == out[0]) and (H == 1 or x[1] == out[1])
    return not alike or x_at == out_at or not any(share(a, b) for a in rows for b in other)


def test_rows_that_share_memory_are_refused(lib):  # noqa: F811
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        T, H = rng.randint(1, 4), rng.randint(1, 4)
        strides = [rng.choice([0, 1, D - 1, D, D + 3, 2 * D, H * D, H * D + 5, T * D, -D, -T * D, -7, rng.randint(-80, 80)])
                   for _ in range(2)]
        out = strides if rng.random() < 0.7 else [rng.randint(-80, 80) for _ in range(2)]
        shift = rng.choice([0, 0, D, -D, rng.randint(-100, 100), H * D, T * D])
        want = allowed(T, H, 0, strides, shift, out)
        seen[want] += 1
        x = heads(AT, *strides)
        assert lib.qsw_rope(x, T, H, D, None, FAKE, D, 0, 1.0, 0, AT + 2 * shift, *out, None) == (CUDA if want else INVALID), (
            T, H, strides, out, shift)
        k = heads(AT, D, D)
        assert lib.qsw_kv_append(x, k, k, T, H, D, FAKE, None, FAKE, D, 0, 1.0, 0, cache(D=D), AT + 2 * shift, *out,
                                 None) == (CUDA if want else INVALID)
    assert min(seen.values()) > 500, seen


def test_far_strides_do_not_overflow(lib):  # noqa: F811
    far = 1 << 62
    for strides, code in (((far, far), INVALID), ((-far, far), INVALID), ((0, far), INVALID), ((far, 0), INVALID),
                          ((far, D), CUDA), ((D, far), CUDA), ((-far, -D), CUDA)):
        assert lib.qsw_rope(heads(AT, *strides), 1 << 20, 4096, D, None, FAKE, D, 0, 1.0, 0, AT, *strides, None) == code
