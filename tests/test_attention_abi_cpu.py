"""The attention half's C entries on the CPU: refusals before any launch, sizes; the
rotation's table and frequencies."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests.test_abi_cpu import FAKE, INVALID, OK, UNSUPPORTED, lib  # noqa: F401

CUDA = 3


def heads(data=FAKE, token=512, head=64):
    return ctypes.byref(ops.Heads(data, token, head))


def cache(k=FAKE, v=FAKE, pages=10, kv_heads=2, page_size=16, D=64, k_strides=None, v_strides=None):
    dense = (kv_heads * page_size * D, page_size * D, D)
    return ctypes.byref(ops.KvCache(k, v, pages, kv_heads, page_size, (ctypes.c_int64 * 3)(*(k_strides or dense)),
                                    (ctypes.c_int64 * 3)(*(v_strides or dense))))


def rope(lib, x=None, T=0, H=8, D=64, positions=FAKE, table=FAKE, rot=64, scale=1.0, act=0, out=FAKE):  # noqa: F811
    return lib.qsw_rope(x or heads(), T, H, D, positions, table, rot, 0, scale, act, out, 512, 64, None)


def append(lib, q="heads", k=None, v=None, T=0, H=8, D=64, slots=FAKE, positions=FAKE, table=FAKE, rot=64, scale=1.0, act=0,  # noqa: F811
           c=None, q_out=FAKE):
    q = heads() if q == "heads" else q
    return lib.qsw_kv_append(q, k or heads(), v or heads(), T, H, D, slots, positions, table, rot, 0, scale, act, c or cache(),
                             q_out, 512, 64, None)


def plan(lib, offsets=FAKE, lengths=FAKE, B=3, table=FAKE, stride=20, max_pages=20, T=0, H=8, D=64, window=0, c=None,  # noqa: F811
         positions=FAKE, slots=FAKE, work=FAKE):
    return lib.qsw_paged_plan(offsets, lengths, B, table, stride, max_pages, T, H, D, window, c or cache(), positions, slots,
                              work, None)


def attend(lib, q=None, c=None, table=FAKE, stride=20, max_pages=20, work=FAKE, B=3, T=0, H=8, D=64, window=0, scale=0.125,  # noqa: F811
           act=0, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib.qsw_paged_attention(q or heads(), c or cache(), table, stride, max_pages, work, B, T, H, D, window, scale, act,
                                   out, ws, ws_bytes, None)


def test_no_tokens_is_a_noop(lib):  # noqa: F811
    assert rope(lib) == append(lib) == plan(lib) == attend(lib) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(rot=63), INVALID), (dict(rot=66), INVALID),
    (dict(rot=-2), INVALID), (dict(act=2), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(table=None), INVALID), (dict(table=FAKE + 4), UNSUPPORTED), (dict(D=1026), UNSUPPORTED),
    (dict(H=4097), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(T=1, x=heads(0)), INVALID),
    (dict(T=1, out=0), INVALID), (dict(T=1, x=heads(FAKE + 1)), UNSUPPORTED), (dict(T=1, out=FAKE + 1), UNSUPPORTED),
    (dict(T=1, positions=FAKE + 2), UNSUPPORTED)])
def test_rope_rejects(lib, kw, code):  # noqa: F811
    assert rope(lib, **kw) == code


BAD_CACHES = [
    (dict(pages=-1), INVALID), (dict(pages=0), INVALID), (dict(kv_heads=0), INVALID), (dict(page_size=0), INVALID), (dict(k=0), INVALID),
    (dict(v=0), INVALID), (dict(page_size=12), UNSUPPORTED), (dict(kv_heads=1025), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED), (dict(pages=1 << 62), UNSUPPORTED), (dict(k=FAKE + 8), UNSUPPORTED),
    (dict(v=FAKE + 2), UNSUPPORTED), (dict(k_strides=(2048, 1024, 68)), UNSUPPORTED),
    (dict(v_strides=(2044, 1024, 64)), UNSUPPORTED), (dict(v_strides=(2048, -1024, 64)), INVALID),
    (dict(k_strides=(2048, 0, 64)), INVALID), (dict(k_strides=(1 << 39, 1024, 64)), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(lib, kw, code):  # noqa: F811
    assert append(lib, c=cache(**kw)) == plan(lib, c=cache(**kw)) == attend(lib, c=cache(**kw)) == code


@pytest.mark.parametrize("D,code", [(0, INVALID), (-64, INVALID), (60, UNSUPPORTED), (136, UNSUPPORTED), (128, OK)])
def test_head_sizes(lib, D, code):  # noqa: F811
    assert append(lib, D=D, rot=0) == plan(lib, D=D) == attend(lib, D=D) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(rot=66), INVALID), (dict(act=2), INVALID),
    (dict(T=1, slots=0), INVALID), (dict(T=1, k=heads(0)), INVALID), (dict(T=1, v=heads(0)), INVALID),
    (dict(T=1, q=heads(0)), INVALID), (dict(T=1, q_out=0), INVALID), (dict(T=1, slots=FAKE + 1), UNSUPPORTED),
    (dict(T=1, k=heads(FAKE + 1)), UNSUPPORTED), (dict(q=None, H=0), OK)])
def test_append_rejects(lib, kw, code):  # noqa: F811
    assert append(lib, **kw) == code


BAD_STEPS = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=7), INVALID), (dict(max_pages=-1), INVALID),
    (dict(window=-1), INVALID), (dict(B=65537), UNSUPPORTED), (dict(T=(1 << 22) + 1), UNSUPPORTED),
    (dict(H=1026), UNSUPPORTED), (dict(T=1 << 22, H=512), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED),
    (dict(window=(1 << 30) + 1), UNSUPPORTED), (dict(T=1, table=0), INVALID), (dict(T=1, work=0), INVALID),
    (dict(T=1, work=FAKE + 8), UNSUPPORTED), (dict(T=1, table=FAKE + 2), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_STEPS)
def test_bad_steps(lib, kw, code):  # noqa: F811
    assert plan(lib, **kw) == attend(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=3e38), INVALID),
    (dict(act=3), INVALID), (dict(T=1, q=heads(0)), INVALID), (dict(T=1, out=0), INVALID),
    (dict(T=1, q=heads(FAKE + 8)), UNSUPPORTED), (dict(T=1, out=FAKE + 8), UNSUPPORTED),
    (dict(T=1, q=heads(token=516)), UNSUPPORTED), (dict(T=1, q=heads(head=68)), UNSUPPORTED),
    (dict(T=1, ws=FAKE + 128), UNSUPPORTED)])
def test_attention_rejects(lib, kw, code):  # noqa: F811
    assert attend(lib, **kw) == code


def test_plan_rejects(lib):  # noqa: F811
    for name in ("offsets", "lengths", "positions", "slots"):
        assert plan(lib, T=1, **{name: 0}) == INVALID
        assert plan(lib, T=1, **{name: FAKE + 1}) == UNSUPPORTED


def test_sizes_that_no_call_accepts(lib):  # noqa: F811
    assert lib.qsw_paged_plan_bytes(1, 0) > 0
    assert lib.qsw_paged_plan_bytes(0, 4) == lib.qsw_paged_plan_bytes(65537, 4) == 0
    assert lib.qsw_paged_plan_bytes(4, -1) == lib.qsw_paged_plan_bytes(4, 1 << 62) == 0
    for a in ((0, 1, 8, 2, 64), (1, -1, 8, 2, 64), (1, 1, 8, 3, 64), (1, 1, 8, 0, 64), (1, 1, 1 << 40, 1, 64), (1, 1, 8, 2, 60),
              (1, 1, 8, 2, 1 << 40)):
        assert lib.qsw_paged_attention_workspace_bytes(*a, 1000) == 0
    assert lib.qsw_paged_attention_workspace_bytes(1, 1, 8, 2, 64, -1) == 0
    assert lib.qsw_paged_attention_workspace_bytes(1, 1, 8, 2, 64, 1 << 31) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are valid: with a device these would be launched")
def test_without_a_device(lib):  # noqa: F811
    assert rope(lib, T=4) == append(lib, T=4) == plan(lib, T=4) == attend(lib, T=4) == CUDA


# ------------------------------------------------------- table, frequencies --

def turns_of(f):
    """f / 2 pi modulo 1 as an exact fraction, with 2 pi as f64 gives it."""
    return Fraction(f) / Fraction(2 * math.pi) % 1


@pytest.mark.parametrize("f", [0.0, 1.0, -1.0, 1e-4, 1.2345e-7, 3.0, math.pi, 2 * math.pi, 7.0, -2.5, 1e-30, 100.0])
def test_table_holds_turns(f):
    got = ops.rope_table([f], device="cpu")
    assert got.dtype == torch.int64
    # f / 2 pi is one f64 division: off by half a step of the quotient
    off = (Fraction(int(got[0]), 1 << 64) - turns_of(f)) % 1
    assert min(off, 1 - off) <= Fraction(abs(f) / (2 * math.pi)) * Fraction(1, 1 << 53) + Fraction(1, 1 << 64)


def test_table_refuses():
    for f in (math.nan, math.inf):
        with pytest.raises(ValueError):
            ops.rope_table([f], device="cpu")
    assert ops.rope_table(torch.zeros(0), device="cpu").shape == (0,)


def test_frequencies():
    plain = ops.rope_frequencies(8, 10000.0)
    assert plain.tolist() == pytest.approx([1, 0.1, 0.01, 0.001], rel=1e-12)
    assert ops.rope_frequencies(8, scaling="linear", factor=4).tolist() == pytest.approx((plain / 4).tolist(), rel=1e-12)
    base = ops.rope_frequencies(8, scaling="base", factor=4)
    assert base[0] == 1 and float(base[3]) == pytest.approx(0.001 / 4, rel=1e-12)
    ramp = ops.rope_frequencies(128, scaling="ramp", factor=4, original_length=4096)
    plain = ops.rope_frequencies(128)
    ratio = plain / ramp
    turns = plain * 4096 / (2 * math.pi)
    assert torch.allclose(ratio[turns > 33], torch.ones(1, dtype=torch.float64))
    assert torch.allclose(ratio[turns < 0.8], torch.full((1,), 4.0, dtype=torch.float64))
    assert bool((ratio.diff() >= -1e-12).all())
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, base=0.0), dict(dim=8, factor=-1.0), dict(dim=8, scaling="other"),
                dict(dim=8, scaling="ramp"), dict(dim=2, scaling="base"), dict(dim=8, base=math.inf)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(**bad)
