"""The C ABI on the CPU: the library loads, exports every symbol the header
declares, and rejects bad arguments on the host before any CUDA call.
No compute is launched here (no GPU in this environment)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

from quantized_swiglu_mlp_gb300 import build as qbuild
from quantized_swiglu_mlp_gb300 import ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qswiglu.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return ops.load_library()


def declared_functions():
    text = open(HEADER).read()
    return re.findall(r"QSW_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


def test_header_declares_the_abi():
    names = declared_functions()
    assert set(names) == set(ops.EXPORTED), names


def test_every_declared_symbol_is_exported(lib):
    for name in declared_functions():
        assert hasattr(lib, name), name
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value


FAKE = 0x10000          # aligned, never dereferenced: validation fails or M == 0 first


def fwd(lib, M=4, H=256, I=64, gs_g=64, bits_g=4, gs_u=64, bits_u=4, variant=0,
        x=FAKE, wg=FAKE, sg=FAKE, bg=FAKE, wu=FAKE, su=FAKE, bu=FAKE, out=FAKE):
    return lib.qswiglu_forward(x, M, H, I, wg, sg, bg, gs_g, bits_g, wu, su, bu, gs_u, bits_u,
                               variant, out, None)


def test_m_zero_is_a_noop(lib):
    assert fwd(lib, M=0) == OK
    assert lib.affine_qmm(FAKE, 0, 256, 64, FAKE, FAKE, FAKE, 64, 4, FAKE, None) == OK
    assert lib.qsw_silu_mul(FAKE, FAKE, 0, 0, FAKE, None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID),
    (dict(H=0), INVALID),
    (dict(I=0), INVALID),
    (dict(H=48), UNSUPPORTED),                 # H % 32 != 0
    (dict(gs_g=48), UNSUPPORTED),              # group size not a multiple of 32
    (dict(gs_u=96), UNSUPPORTED),              # does not divide H=256
    (dict(bits_g=3), UNSUPPORTED),
    (dict(bits_u=16), UNSUPPORTED),
    (dict(bits_g=2, H=96, gs_g=32, gs_u=32), UNSUPPORTED),   # 2-bit needs H % 64 == 0
    (dict(variant=7), INVALID),
    (dict(x=0), INVALID),
    (dict(wg=0), INVALID),
    (dict(su=0), INVALID),
    (dict(out=0), INVALID),
    (dict(x=FAKE + 8), UNSUPPORTED),           # 16-byte alignment
    (dict(wu=FAKE + 4), UNSUPPORTED),
    (dict(out=FAKE + 2), UNSUPPORTED),
    (dict(sg=FAKE + 1), UNSUPPORTED),
])
def test_forward_rejects(lib, kw, code):
    assert fwd(lib, **kw) == code


def test_affine_qmm_rejects(lib):
    assert lib.affine_qmm(FAKE, 4, 100, 64, FAKE, FAKE, FAKE, 32, 4, FAKE, None) == UNSUPPORTED
    assert lib.affine_qmm(FAKE, 4, 256, -1, FAKE, FAKE, FAKE, 64, 4, FAKE, None) == INVALID
    assert lib.affine_qmm(0, 4, 256, 64, FAKE, FAKE, FAKE, 64, 4, FAKE, None) == INVALID
    assert lib.affine_qmm(FAKE, 4, 256, 64, FAKE, FAKE, FAKE, 64, 5, FAKE, None) == UNSUPPORTED


def test_silu_mul_rejects(lib):
    assert lib.qsw_silu_mul(FAKE, FAKE, -1, 0, FAKE, None) == INVALID
    assert lib.qsw_silu_mul(FAKE, FAKE, 8, 2, FAKE, None) == INVALID     # debug variants only fuse
    assert lib.qsw_silu_mul(0, FAKE, 8, 0, FAKE, None) == INVALID
    assert lib.qsw_silu_mul(FAKE + 2, FAKE, 8, 0, FAKE, None) == UNSUPPORTED


def test_gemv_limit_is_clamped(lib):
    saved = ops.qsw_get_gemv_max_m()
    try:
        ops.qsw_set_gemv_max_m(1000)
        assert ops.qsw_get_gemv_max_m() == 32
        ops.qsw_set_gemv_max_m(-5)
        assert ops.qsw_get_gemv_max_m() == 0
        ops.qsw_set_gemv_max_m(8)
        assert ops.qsw_get_gemv_max_m() == 8
    finally:
        ops.qsw_set_gemv_max_m(saved)


def test_counters_and_strings(lib):
    ops.qsw_reset_counters()
    assert ops.qsw_get_counters() == [0] * ops.NUM_COUNTERS
    assert fwd(lib, M=0) == OK                       # a no-op launches nothing
    assert ops.qsw_get_counters() == [0] * ops.NUM_COUNTERS
    assert ops.qsw_status_string(0) == "ok"
    assert "unsupported" in ops.qsw_status_string(2)
    assert ops.qsw_status_string(99) == "unknown status"
    assert ops.qsw_version() >= 100


def test_python_binding_rejects_host_tensors(lib):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.qswiglu_forward(x, x, x, x, 64, 4, x, x, x, 64, 4)


def test_early_weight_stream_switch():
    """The early weight stream is off by default and toggles process-wide."""
    from quantized_swiglu_mlp_gb300 import ops
    ops.load_library()
    saved = ops.qsw_get_early_weight_stream()
    try:
        ops.qsw_set_early_weight_stream(True)
        assert ops.qsw_get_early_weight_stream() is True
        ops.qsw_set_early_weight_stream(False)
        assert ops.qsw_get_early_weight_stream() is False
    finally:
        ops.qsw_set_early_weight_stream(saved)



def fwd_ws(lib, ws, ws_bytes, M=4):
    return lib.qswiglu_forward_ws(FAKE, M, 256, 64, FAKE, FAKE, FAKE, 64, 4, FAKE, FAKE, FAKE, 64, 4,
                                  0, FAKE, ws, ws_bytes, None)


def test_workspace_entry_points_validate_on_the_host(lib):
    """The *_ws entry points check the workspace before anything is launched:
    a misaligned one is unsupported, a null one means whole tiles only, and
    argument errors are reported as for the plain entry points."""
    assert fwd_ws(lib, FAKE + 64, 1 << 30) == UNSUPPORTED          # 256-byte alignment
    assert fwd_ws(lib, None, 0, M=0) == OK
    assert fwd_ws(lib, FAKE, 1 << 30, M=0) == OK
    assert fwd_ws(lib, FAKE, 1 << 30, M=-1) == INVALID
    assert lib.affine_qmm_ws(FAKE, 4, 256, 64, FAKE, FAKE, FAKE, 64, 4, FAKE, FAKE + 16, 1 << 30,
                             None) == UNSUPPORTED
    assert lib.affine_qmm_ws(FAKE, 0, 256, 64, FAKE, FAKE, FAKE, 64, 4, FAKE, FAKE, 1 << 30, None) == OK
    # no device is current here: the size query answers 0
    assert lib.qsw_workspace_bytes() == 0


def test_stream_k_mode_switch(lib):
    """Stream-K scheduling defaults to auto; out-of-range modes are ignored."""
    saved = ops.qsw_get_stream_k()
    try:
        assert saved == ops.STREAM_K_AUTO
        for mode in (ops.STREAM_K_OFF, ops.STREAM_K_ALWAYS, ops.STREAM_K_AUTO):
            ops.qsw_set_stream_k(mode)
            assert ops.qsw_get_stream_k() == mode
        ops.qsw_set_stream_k(7)
        assert ops.qsw_get_stream_k() == ops.STREAM_K_AUTO
    finally:
        ops.qsw_set_stream_k(saved)


def test_noalloc_entry_point_validates_on_the_host(lib):
    """The static-scratch entry point checks its arguments before anything
    (including its first-use set-up) touches the device."""
    call = lambda M, variant, x=FAKE: lib.qswiglu_forward_noalloc(x, M, 256, 64, FAKE, FAKE, FAKE, 64, 4, FAKE,
                                                                    FAKE, FAKE, 64, 4, variant, FAKE, None)
    assert call(0, 0) == OK
    assert call(-1, 0) == INVALID
    assert call(4, 7) == INVALID
    assert call(4, 0, x=FAKE + 8) == UNSUPPORTED


def test_mlp_entry_point_validates_on_the_host(lib):
    """The whole-MLP entry point checks both stages' arguments first."""
    def mlp(M=4, variant=0, act=0, h=None, hidden=FAKE, I=64, gs_d=32, bits_d=4):
        return lib.qsw_mlp_forward_ex(FAKE, h, M, 256, I, 96, FAKE, FAKE, FAKE, 64, 4, FAKE, FAKE, FAKE, 64, 4,
                                      FAKE, FAKE, FAKE, gs_d, bits_d, variant, act, hidden, FAKE, None, 0, None)
    assert mlp(M=0) == OK
    assert mlp(variant=2) == INVALID            # debug variants have no whole-block meaning
    assert mlp(act=3) == INVALID
    assert mlp(hidden=None) == INVALID
    assert mlp(h=FAKE + 2) == UNSUPPORTED        # residual alignment
    assert mlp(gs_d=48) == UNSUPPORTED           # down group size
    assert mlp(I=48) == UNSUPPORTED              # I is the down projection's K
    assert mlp(bits_d=3) == UNSUPPORTED


def test_debug_build_is_built_and_exports_the_same_abi(lib):
    """The debug build (QSW_DEBUG_BOUNDS) is built beside the regular one,
    exports every declared symbol and says which build it is."""
    dbg = ctypes.CDLL(qbuild.DEBUG_LIB_PATH)
    for name in declared_functions():
        assert hasattr(dbg, name), name
    dbg.qsw_debug_build.restype = ctypes.c_int
    lib.qsw_debug_build.restype = ctypes.c_int
    assert dbg.qsw_debug_build() == 1 and lib.qsw_debug_build() == 0
    dbg.qsw_status_string.restype = ctypes.c_char_p
    assert b"debug" in dbg.qsw_status_string(5)


# ------------------------------------------------- operators around the block

MX, NV = 0, 1
BIG = 1 << 40


def test_fp4_sizes(lib):
    assert lib.qsw_fp4_scale_bytes(1, 1, 32, NV) == 512
    assert lib.qsw_fp4_scale_bytes(1, 128, 64, NV) == 512
    assert lib.qsw_fp4_scale_bytes(1, 129, 96, NV) == 4 * 512
    assert lib.qsw_fp4_scale_bytes(3, 129, 128, MX) == 6 * 512
    assert lib.qsw_fp4_scale_bytes(1, 4, 48, NV) == 0           # K not a multiple of 32
    assert lib.qsw_fp4_scale_bytes(1, 4, 64, 2) == 0
    assert lib.qsw_fp4_workspace_bytes(8, 64, 3, NV) == 256 + 4 * 512
    assert lib.qsw_fp4_workspace_bytes(8, 64, 0, NV) == 0
    assert lib.qsw_fp4_moe_workspace_bytes(0, 2, 64, 64, 4, MX) >= 2 * 4 * 512


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), OK), (dict(groups=0), OK), (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(K=48), UNSUPPORTED),
    (dict(K=(1 << 22) + 32), UNSUPPORTED),
    (dict(fmt=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(fmt=MX, scale=2.0), INVALID), (dict(act=2), INVALID),
    (dict(x=0), INVALID), (dict(codes=FAKE + 8), UNSUPPORTED), (dict(scales=FAKE + 4), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(groups=1 << 31), UNSUPPORTED),
])
def test_fp4_quantize_refuses(lib, kw, code):
    a = dict(x=FAKE, groups=1, rows=4, K=64, fmt=NV, scale=1.0, act=0, codes=FAKE, scales=FAKE) | kw
    assert lib.qsw_fp4_quantize(a["x"], a["groups"], a["rows"], a["K"], a["fmt"], a["scale"], a["act"], a["codes"],
                                a["scales"], None) == code
    assert lib.qsw_fp4_dequantize(a["codes"], a["scales"], a["groups"], a["rows"], a["K"], a["fmt"], a["scale"],
                                  a["act"], a["x"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), OK), (dict(rows=0, x=0, y=0, ws=0), OK), (dict(rows=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=40), UNSUPPORTED), (dict(act=3), INVALID), (dict(w=0), INVALID), (dict(w=FAKE + 8), UNSUPPORTED),
    (dict(w_scale=FAKE + 2), UNSUPPORTED), (dict(x=0), INVALID), (dict(ws=0), INVALID), (dict(ws=FAKE + 16), UNSUPPORTED),
    (dict(ws_bytes=8), INVALID), (dict(y=FAKE + 1), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED),
])
def test_fp4_products_refuse(lib, kw, code):
    a = dict(x=FAKE, rows=4, K=64, N=32, scale=1.0, w=FAKE, w_scales=FAKE, w_scale=None, act=0, y=FAKE, ws=FAKE,
             ws_bytes=BIG) | kw
    rest = (a["w"], a["w_scales"], a["w_scale"], a["act"], a["y"], a["ws"], a["ws_bytes"], None)
    assert lib.qsw_fp4_linear(a["x"], a["rows"], a["K"], a["N"], NV, a["scale"], *rest) == code
    assert lib.qsw_fp4_grouped_linear(a["x"], a["rows"], a["K"], a["N"], 3, FAKE, NV, a["scale"], *rest) == code


def test_fp4_grouped_linear_refuses_groups(lib):
    call = lambda groups, offsets: lib.qsw_fp4_grouped_linear(FAKE, 0, 64, 32, groups, offsets, NV, 1.0, FAKE, FAKE,  # noqa: E731
                                                              None, 0, FAKE, FAKE, BIG, None)
    assert call(3, FAKE) == OK
    assert call(0, FAKE) == INVALID
    assert call(3, None) == INVALID
    assert call(1025, FAKE) == UNSUPPORTED
    assert call(3, FAKE + 2) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(dtype=3), INVALID),
    (dict(scoring=2), INVALID), (dict(scale=float("inf")), INVALID), (dict(E=2000), UNSUPPORTED),
    (dict(E=64, k=33), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(logits=0), INVALID), (dict(offsets=0), INVALID),
    (dict(ids=FAKE + 2), UNSUPPORTED), (dict(logits=FAKE + 2), UNSUPPORTED),
])
def test_moe_route_refuses(lib, kw, code):
    a = dict(logits=FAKE, T=4, E=8, k=2, dtype=2, scoring=0, scale=1.0, ids=FAKE, offsets=FAKE) | kw
    assert lib.qsw_moe_route(a["logits"], a["T"], a["E"], a["k"], a["dtype"], a["scoring"], 1, a["scale"], a["ids"],
                             FAKE, a["offsets"], FAKE, FAKE, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(k=9), INVALID), (dict(H=40), UNSUPPORTED), (dict(I=40), UNSUPPORTED),
    (dict(h_scale=0.0), INVALID), (dict(fmt=MX, h_scale=0.5), INVALID), (dict(wd=0), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(residual=FAKE + 2), UNSUPPORTED), (dict(y=0), INVALID), (dict(E=1025), UNSUPPORTED),
])
def test_fp4_moe_mlp_refuses(lib, kw, code):
    a = dict(T=4, H=64, I=64, E=8, k=2, fmt=NV, h_scale=1.0, wd=FAKE, residual=None, y=FAKE, ws_bytes=BIG) | kw
    assert lib.qsw_fp4_moe_mlp(FAKE, a["T"], a["H"], a["I"], a["E"], a["k"], a["fmt"], 1.0, a["h_scale"], FAKE, FAKE,
                               FAKE, FAKE, FAKE, FAKE, FAKE, None, a["wd"], FAKE, None, a["residual"], 0, a["y"], FAKE,
                               a["ws_bytes"], None) == code


def test_norms_refuse(lib):
    rms = lambda rows=4, H=64, eps=1e-6, act=0, x=FAKE: lib.qsw_rms_norm(x, None, rows, H, eps, act, FAKE, None)  # noqa: E731
    assert rms(rows=0) == OK
    assert rms(rows=-1) == INVALID and rms(H=0) == INVALID and rms(eps=-1.0) == INVALID and rms(act=2) == INVALID
    assert rms(eps=float("nan")) == INVALID and rms(x=0) == INVALID
    assert rms(H=32769) == UNSUPPORTED and rms(x=FAKE + 1) == UNSUPPORTED

    def post(h=FAKE, norm=1, w=None, gate=None, gr=0, gc=0, scale=1.0, rows=4, out=FAKE):
        return lib.qsw_post_norm(h, FAKE, norm, w, gate, gr, gc, scale, None, rows, 64, 1e-6, 0, out, None, None)
    assert post(rows=0) == OK
    assert post(h=0) == INVALID and post(out=0) == INVALID and post(scale=float("nan")) == INVALID
    assert post(norm=0, w=FAKE) == INVALID
    assert post(gate=FAKE, gr=3, gc=64) == INVALID and post(gate=FAKE, gr=2, gc=32) == INVALID
    assert post(gate=FAKE, gr=0, gc=64) == INVALID
    assert post(gate=FAKE + 1, gr=2, gc=64) == UNSUPPORTED


def test_block_bindings_refuse_host_tensors(lib):
    import torch
    x, u8 = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 32, dtype=torch.uint8)
    r = ops.MoeRoute(*[torch.zeros(2, 1, dtype=torch.int32)] * 5)
    for call in (lambda: ops.fp4_quantize(x), lambda: ops.fp4_dequantize(u8, u8), lambda: ops.fp4_linear(x, u8, u8),
                 lambda: ops.fp4_grouped_linear(x, u8, u8, u8), lambda: ops.moe_route(x, 2),
                 lambda: ops.fp4_moe_mlp(x, r, u8, u8, u8, u8), lambda: ops.rms_norm(x), lambda: ops.post_norm(x, x)):
        with pytest.raises(ValueError):
            call()
