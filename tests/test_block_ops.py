"""Microscaled 4-bit floating point, grouped products, expert MLP, routing and
norms on the GPU, against plain float64 implementations."""
from __future__ import annotations

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
DT = {"bf16": BF16, "f16": F16}
NAMES = {ops.FP4_MX: "mx", ops.FP4_NV: "nv"}
SCALE = {ops.FP4_MX: 1.0, ops.FP4_NV: 0.0213}
formats = pytest.mark.parametrize("fmt", [ops.FP4_MX, ops.FP4_NV], ids=NAMES.get)
dtypes = pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])


@pytest.fixture(scope="module")
def dev():
    torch.cuda.set_device(0)
    ops.load_library()
    return torch.device("cuda:0")


def randn(seed, *shape, dt=BF16, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def weight(seed, groups, N, K, fmt):
    """A stack of matrices in 4 bits, its tensor scales and its float64 values."""
    gs = [0.0007 * (1 + 0.13 * (e % 5)) if fmt == ops.FP4_NV else 1.0 for e in range(groups)]
    codes, scales, vals = [], [], []
    for e in range(groups):
        c, s = ops.fp4_quantize(randn(seed * 1000 + e, N, K, std=K ** -0.5), fmt, scale=gs[e])
        g32 = float(torch.tensor(gs[e], dtype=torch.float32))
        codes.append(c)
        scales.append(s)
        vals.append(ref.values(c, s, fmt, g32))
    return torch.stack(codes), torch.stack(scales), torch.tensor(gs, device="cuda"), vals


def check(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound).max()), bad.nonzero()[:4].tolist())


def held(x, fmt):
    """x as the library quantises it, in float64."""
    c, s = ops.fp4_quantize(x, fmt, scale=SCALE[fmt])
    return ref.values(c, s, fmt, float(torch.tensor(SCALE[fmt], dtype=torch.float32)))


# ------------------------------------------------------------- quantisation --

@formats
@dtypes
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (6, 512), (31, 96), (33, 160), (128, 256), (129, 288), (300, 2080)])
def test_quantize_bit_for_bit(dev, fmt, dt, rows, K):
    """Codes and scale bytes equal the documented steps; the scales past the last are 0."""
    x = randn(rows * K, rows, K, dt=dt)
    x[:, 5] *= 30
    x[rows // 2] = 0
    x[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=dt)   # ties of e2m1
    codes, scales = ops.fp4_quantize(x, fmt, scale=SCALE[fmt])
    want, byte = ref.quantize(x, fmt, SCALE[fmt])
    n = K // ref.BLOCK[fmt]
    assert torch.equal(ref.scale_at(scales, rows, scales.shape[-2] * 4)[:, :n], byte)
    assert not ref.scale_at(scales, rows, scales.shape[-2] * 4)[:, n:].any()
    assert torch.equal(ref.unpack(codes).long(), want)


@formats
def test_quantize_every_bf16_value(dev, fmt):
    """All 65,536 bf16 patterns, each alone in its block, as the largest of it."""
    v = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16)
    x = torch.zeros(65536, 32, dtype=BF16, device="cuda")
    x[:, 3] = v
    x[:, 7] = (v.float() * 0.37).to(BF16)
    for g in ([1.0] if fmt == ops.FP4_MX else [1.0, 0.0213, 1e30, 1e-30]):
        codes, scales = ops.fp4_quantize(x, fmt, scale=g)
        want, byte = ref.quantize(x, fmt, g)
        n = 32 // ref.BLOCK[fmt]
        assert torch.equal(ref.scale_at(scales, 65536, n), byte), g
        finite = (byte != (255 if fmt == ops.FP4_MX else 127)).repeat_interleave(ref.BLOCK[fmt], 1)
        assert torch.equal(ref.unpack(codes).long()[finite], want[finite]), g


@formats
@dtypes
@pytest.mark.parametrize("shape", [(1, 32), (7, 96), (130, 512), (3, 129, 224)])
def test_dequantize(dev, fmt, dt, shape):
    """Codes and scales of a matrix and of a stack come back as the values they stand for, rounded once."""
    x = randn(5, *shape, dt=dt)
    codes, scales = ops.fp4_quantize(x, fmt, scale=SCALE[fmt])
    out = ops.fp4_dequantize(codes, scales, fmt, scale=SCALE[fmt], dtype=dt)
    g = float(torch.tensor(SCALE[fmt], dtype=torch.float32))
    stack = [(codes, scales, out)] if len(shape) == 2 else list(zip(codes, scales, out))
    for c, s, o in stack:
        want = ref.values(c, s, fmt, g)
        # the f32 product scale * g and its product with the code: 2^-23 relative
        check(o, want, ref.half_ulp(want, dt) * (1 + 2.0 ** -10) + want.abs() * 2.0 ** -23)
    # a value is within half a step of its block's scale, or saturated
    err = (out.double() - x.double()).abs().reshape(*shape[:-1], -1, ref.BLOCK[fmt])
    amax = x.double().abs().reshape(err.shape).amax(-1, keepdim=True)
    assert (err <= amax * (0.26 if fmt == ops.FP4_MX else 0.2) + SCALE[fmt] * 2.0 ** -8).all()


@formats
def test_quantize_nonfinite_blocks(dev, fmt):
    """A block with an infinity or a NaN comes back as NaN; its neighbours are untouched."""
    x = randn(9, 4, 128)
    plain = ops.fp4_dequantize(*ops.fp4_quantize(x, fmt, scale=SCALE[fmt]), fmt, scale=SCALE[fmt])
    x[1, 40], x[2, 100], x[3, 0] = float("inf"), float("nan"), float("-inf")
    got = ops.fp4_dequantize(*ops.fp4_quantize(x, fmt, scale=SCALE[fmt]), fmt, scale=SCALE[fmt])
    bad = (~torch.isfinite(x)).reshape(4, -1, ref.BLOCK[fmt]).any(-1).repeat_interleave(ref.BLOCK[fmt], 1)
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], plain[~bad])


# ----------------------------------------------------------------- products --

@formats
@dtypes
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 16, 64), (1, 128, 256), (1, 200, 288), (1, 2048, 512), (2, 65, 96), (16, 256, 320), (17, 130, 1024),
    (64, 128, 512), (65, 384, 544), (128, 200, 256), (129, 136, 768), (191, 256, 256), (192, 129, 512), (193, 256, 288),
    (256, 512, 1056), (385, 144, 640), (600, 1300, 2112)])
def test_linear(dev, fmt, dt, M, N, K):
    x = randn(M + N + K, M, K, dt=dt)
    w, ws, wg, vals = weight(3, 1, N, K, fmt)
    y = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    ops.qsw_check_device_errors()
    a = held(x, fmt)
    want = a @ vals[0].T
    check(y, want, ref.half_ulp(want, dt) * (1 + 2.0 ** -8) + ref.sum_bound(a.abs() @ vals[0].abs().T, K) + 2.0 ** -26)


@formats
@pytest.mark.parametrize("M,N,K", [(256, 20000, 64), (64, 19500, 96), (97, 19585, 288), (193, 13000, 544),
                                   (200, 10001, 320), (385, 7100, 640), (1030, 5000, 1056)])
def test_linear_on_cta_pairs(dev, fmt, M, N, K):
    """Sizes with enough tiles for the two-CTA form: ragged rows of both operands."""
    x = randn(M + N + K, M, K)
    w, ws, wg, vals = weight(3, 1, N, K, fmt)
    y = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    ops.qsw_check_device_errors()
    a = held(x, fmt)
    want = a @ vals[0].T
    check(y, want, ref.half_ulp(want, BF16) * (1 + 2.0 ** -8) + ref.sum_bound(a.abs() @ vals[0].abs().T, K) + 2.0 ** -26)


@formats
@dtypes
@pytest.mark.parametrize("M,N,K", [(1, 130, 5920), (1, 128, 7168), (2, 2048, 8192), (3, 1000, 6176), (16, 256, 9216),
                                   (17, 700, 8224), (33, 513, 7200), (64, 128, 10240), (65, 200, 6400), (100, 2047, 6144),
                                   (192, 1024, 6432), (200, 300, 8000), (1, 9000, 6240)])
def test_linear_split_over_a_cluster(dev, fmt, dt, M, N, K):
    """Few tiles and a long K: 2 or 4 CTAs share a tile, uneven parts among them."""
    test_linear(dev, fmt, dt, M, N, K)


@formats
def test_linear_is_deterministic_and_flattens(dev, fmt):
    x = randn(1, 3, 5, 512)
    w, ws, wg, _ = weight(4, 1, 320, 512, fmt)
    y = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    assert y.shape == (3, 5, 320)
    again = ops.fp4_linear(x.reshape(15, 512), w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg,
                           out=torch.empty(15, 320, dtype=BF16, device="cuda"))
    assert torch.equal(y.reshape(15, 320), again)
    none = ops.fp4_linear(x[:0], w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    assert none.shape == (0, 5, 320)


@formats
def test_linear_propagates_nonfinite_rows_only(dev, fmt):
    """An infinity in one row makes that row NaN and leaves the others' bits."""
    x = randn(2, 40, 512)
    w, ws, wg, _ = weight(4, 1, 200, 512, fmt)
    y = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    x[7, 300] = float("inf")
    z = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    assert torch.isnan(z[7]).all()
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(y[keep], z[keep])


@formats
@pytest.mark.parametrize("sizes", [[3], [0, 1, 0], [7, 2], [0, 40, 0, 9]], ids=str)
def test_grouped_linear_split_over_a_cluster(dev, fmt, sizes):
    test_grouped_linear(dev, fmt, sizes, 200, 6240)


SIZES = [
    [0, 0, 5], [1], [0], [3, 0, 0, 130, 1], [192, 193, 0, 64], [128, 128, 128], [500, 0, 37, 1, 0, 0, 260],
    [1] * 40, [0] * 33 + [7] + [0] * 66, [17, 64, 65, 127, 129, 191, 257, 400],
]


@formats
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("N,K", [(128, 256), (200, 352)])
def test_grouped_linear(dev, fmt, sizes, N, K):
    """Ragged groups, empty ones among them; every row belongs to its own group's matrix."""
    rows = sum(sizes)
    x = randn(rows + N, rows, K, dt=F16)
    offsets = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")
    w, ws, wg, vals = weight(6, len(sizes), N, K, fmt)
    y = ops.fp4_grouped_linear(x, offsets, w, ws, fmt, x_scale=SCALE[fmt], w_scale=wg)
    ops.qsw_check_device_errors()
    assert y.shape == (rows, N)
    if not rows:
        return
    a = held(x, fmt)
    for e, n in enumerate(sizes):
        s = slice(int(offsets[e]), int(offsets[e]) + n)
        want = a[s] @ vals[e].T
        check(y[s], want, ref.half_ulp(want, F16) * (1 + 2.0 ** -8) + ref.sum_bound(a[s].abs() @ vals[e].abs().T, K)
              + 2.0 ** -26, e)


@formats
@pytest.mark.parametrize("N,K", [(2100, 160), (1793, 576)])
def test_grouped_linear_on_cta_pairs(dev, fmt, N, K):
    """The two-CTA form over ragged groups, empty ones among them."""
    test_grouped_linear(dev, fmt, [100, 0, 257, 64, 31, 192, 0, 193, 128, 500, 1, 97], N, K)


def test_grouped_linear_clamps_offsets(dev):
    """Offsets that run past the rows or backwards are clamped: the call writes
    only its own rows, and rows that one group alone claims (not 5 to 9) are right."""
    fmt = ops.FP4_NV
    x = randn(3, 50, 256)
    w, ws, wg, _ = weight(7, 4, 128, 256, fmt)
    good = torch.tensor([0, 10, 10, 30, 50], dtype=torch.int32, device="cuda")
    want = ops.fp4_grouped_linear(x, good, w, ws, fmt, x_scale=SCALE[fmt], w_scale=wg)
    bad = torch.tensor([-4, 10, 5, 30, 900], dtype=torch.int32, device="cuda")
    buf = torch.zeros(60, 128, dtype=BF16, device="cuda")
    got = ops.fp4_grouped_linear(x, bad, w, ws, fmt, x_scale=SCALE[fmt], w_scale=wg, out=buf[:50])
    ops.qsw_check_device_errors()
    assert torch.equal(got[:5], want[:5]) and torch.equal(got[30:], want[30:])
    assert not buf[50:].any()


# ------------------------------------------------------------------ routing --

@pytest.mark.parametrize("dt", [torch.float32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (9, 32, 4), (64, 33, 8), (200, 64, 6), (513, 128, 8),
                                   (77, 257, 32), (40, 600, 3), (31, 1024, 17), (5000, 16, 1), (4100, 64, 8), (17001, 9, 8)])
@pytest.mark.parametrize("sigmoid,renormalize", [(False, True), (False, False), (True, True), (True, False)])
def test_route(dev, dt, T, E, k, sigmoid, renormalize):
    logits = randn(T + E, T, E, dt=dt, std=2.0)     # 16-bit logits tie often
    r = ops.moe_route(logits, k, scoring=ops.ROUTE_SIGMOID if sigmoid else ops.ROUTE_SOFTMAX, renormalize=renormalize,
                      scale=2.5)
    ids, w, offsets, slots, order = ref.route(logits, k, sigmoid, renormalize, 2.5)
    assert torch.equal(r.ids.long(), ids)
    assert torch.equal(r.offsets.long(), offsets)
    assert torch.equal(r.slots.long(), slots)
    assert torch.equal(r.order.long(), order)
    # expf within 2 ulp of arguments rounded once (|x| < 20: 20 * 2^-24), E-term f32 sums
    check(r.weights, w, w * (E + 64) * 2.0 ** -23 + 1e-37)


def test_route_masked_rows(dev):
    """-inf masks, a row with everything masked, +inf, NaN and type-lowest logits."""
    x = randn(1, 8, 40, dt=torch.float32)
    inf = float("inf")
    x[0] = -inf
    x[1, 3:] = -inf
    x[2, 7] = inf
    x[3, 7], x[3, 20] = inf, inf
    x[4, 11] = float("nan")
    x[5] = float("nan")
    x[6] = torch.finfo(torch.float32).min
    x[7, 2:] = torch.finfo(torch.float32).min
    for sigmoid in (False, True):
        for renorm in (True, False):
            r = ops.moe_route(x, 5, scoring=int(sigmoid), renormalize=renorm)
            ids, w, offsets, slots, order = ref.route(x, 5, sigmoid, renorm)
            assert torch.equal(r.ids.long(), ids)
            assert torch.equal(r.slots.long(), slots) and torch.equal(r.offsets.long(), offsets)
            check(r.weights, w, w * 104 * 2.0 ** -23 + 1e-37)
    assert not ops.moe_route(x, 5).weights[0].any()


def test_route_ids_at_any_word(dev):
    """The C entry takes ids at any 4-byte boundary."""
    lib = ops.load_library()
    T, E, k = 301, 20, 3
    logits = randn(5, T, E, dt=torch.float32)
    want = ops.moe_route(logits, k)
    ids = torch.empty(T * k + 1, dtype=torch.int32, device="cuda")[1:]
    w = torch.empty(T * k, device="cuda")
    offsets, slots, order = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    st = lib.qsw_moe_route(logits.data_ptr(), T, E, k, 2, ops.ROUTE_SOFTMAX, 1, 1.0, ids.data_ptr(), w.data_ptr(),
                           offsets.data_ptr(), slots.data_ptr(), order.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(ids.view(T, k), want.ids) and torch.equal(offsets, want.offsets)
    assert torch.equal(slots.view(T, k), want.slots.view(T, k)) and torch.equal(order, want.order)


def test_route_without_tokens(dev):
    r = ops.moe_route(torch.empty(0, 7, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and not r.offsets.any()


# ------------------------------------------------------------------ experts --

def moe_reference(x, r, k, vals_gu, vals_d, fmt, dt, residual):
    """Output and bound of the expert MLP in float64.

    The hidden activations carry an f32 error, which may move one across a
    rounding boundary of the 4-bit format: the bound holds the largest change
    that a relative error `d` of them makes, through the down weights."""
    T, H = x.shape
    a = held(x, fmt)
    g = float(torch.tensor(SCALE[fmt], dtype=torch.float32))
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    if residual is not None:
        y += residual.double()
    for t in range(T):
        for j in range(k):
            e, w = int(r.ids[t, j]), float(r.weights[t, j])
            gu = vals_gu[e] @ a[t]
            gate, up = gu.reshape(-1, 2, 16).unbind(1)
            hidden = (gate * torch.sigmoid(gate) * up).reshape(-1)
            err = ref.sum_bound(vals_gu[e].abs() @ a[t].abs(), H).reshape(-1, 2, 16)
            # |d hidden| <= 1.1 |up| dgate + |silu| dup, and 2^-20 relative for the sigmoid
            dh = (1.1 * up.abs() * err[:, 0] + (gate * torch.sigmoid(gate)).abs() * err[:, 1]).reshape(-1)
            dh = dh + hidden.abs() * 2.0 ** -20
            q = ref.hold(hidden, fmt, g)
            d = float((dh / hidden.abs().clamp(min=1e-30)).clamp(max=0.5).median())
            slack = torch.zeros_like(q)
            for other in (hidden + dh, hidden - dh, hidden * (1 + d), hidden * (1 - d)):
                slack = torch.maximum(slack, (ref.hold(other, fmt, g) - q).abs())
            o = vals_d[e] @ q
            y[t] += w * o
            b = vals_d[e].abs() @ slack + ref.sum_bound(vals_d[e].abs() @ q.abs(), q.numel()) + ref.half_ulp(o, dt) * 1.01
            bound[t] += abs(w) * b
    return y, bound + ref.half_ulp(y, dt) * 1.01 + y.abs() * 2.0 ** -20 + 2.0 ** -26


@formats
@dtypes
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 64, 32), (1, 16, 8, 256, 128), (3, 2, 2, 96, 160), (5, 8, 1, 288, 96),
                                       (16, 8, 3, 256, 64), (40, 3, 2, 128, 224), (1, 2, 1, 6176, 96),
                                       (2, 3, 2, 96, 6240), (5, 2, 2, 6208, 64)])
@pytest.mark.parametrize("with_residual", [False, True], ids=["plain", "residual"])
def test_moe_mlp(dev, fmt, dt, T, E, k, H, I, with_residual):
    x = randn(T + H, T, H, dt=dt)
    logits = randn(T + E + 1, T, E, dt=torch.float32)
    gu, gus, gug, vgu = weight(8, E, 2 * I, H, fmt)
    d, ds, dg, vd = weight(9, E, H, I, fmt)
    res = randn(77, T, H, dt=dt) if with_residual else None
    r = ops.moe_route(logits, k)
    y = ops.fp4_moe_mlp(x, r, gu, gus, d, ds, fmt, x_scale=SCALE[fmt], h_scale=SCALE[fmt], gu_scale=gug, d_scale=dg,
                        residual=res)
    ops.qsw_check_device_errors()
    want, bound = moe_reference(x, r, k, vgu, vd, fmt, dt, res)
    check(y, want, bound)
    again = ops.fp4_moe_mlp(x, r, gu, gus, d, ds, fmt, x_scale=SCALE[fmt], h_scale=SCALE[fmt], gu_scale=gug,
                            d_scale=dg, residual=res)
    assert torch.equal(y, again)


@formats
def test_moe_mlp_many_tokens_equals_few(dev, fmt):
    """A token's result does not depend on which others are in the batch: long
    groups, several token tiles, other tile heights."""
    T, E, k, H, I = 700, 5, 2, 256, 192
    x = randn(1, T, H)
    logits = randn(2, T, E, dt=torch.float32)
    logits[:, 4] -= 20        # an expert that gets no token
    logits[:, 0] += 3         # one that gets most
    gu, gus, gug, _ = weight(8, E, 2 * I, H, fmt)
    d, ds, dg, _ = weight(9, E, H, I, fmt)

    def mlp(rows):
        return ops.fp4_moe_mlp(x[rows], ops.moe_route(logits[rows], k), gu, gus, d, ds, fmt, x_scale=SCALE[fmt],
                               h_scale=SCALE[fmt], gu_scale=gug, d_scale=dg)
    y = mlp(slice(None))
    ops.qsw_check_device_errors()
    for a, b in ((0, 1), (13, 14), (100, 117), (300, 430), (699, 700)):
        assert torch.equal(y[a:b], mlp(slice(a, b))), (a, b)


@formats
def test_moe_mlp_on_cta_pairs(dev, fmt):
    """A long batch (two-CTA tiles) gives each token the bits that it gets alone."""
    T, E, k, H, I = 230, 8, 4, 1824, 928
    x = randn(1, T, H)
    logits = randn(2, T, E, dt=torch.float32)
    gu, gus, gug, _ = weight(8, E, 2 * I, H, fmt)
    d, ds, dg, _ = weight(9, E, H, I, fmt)

    def mlp(rows):
        return ops.fp4_moe_mlp(x[rows], ops.moe_route(logits[rows], k), gu, gus, d, ds, fmt, x_scale=SCALE[fmt],
                               h_scale=SCALE[fmt], gu_scale=gug, d_scale=dg)
    y = mlp(slice(None))
    ops.qsw_check_device_errors()
    assert torch.isfinite(y.float()).all()
    for a, b in ((0, 1), (7, 9), (100, 117), (229, 230)):
        assert torch.equal(y[a:b], mlp(slice(a, b))), (a, b)


def test_interleave_gate_up():
    gate, up = torch.arange(64).reshape(32, 2), 1000 + torch.arange(64).reshape(32, 2)
    w = ops.interleave_gate_up(gate, up)
    assert torch.equal(w[:16], gate[:16]) and torch.equal(w[16:32], up[:16])
    assert torch.equal(w[32:48], gate[16:]) and torch.equal(w[48:], up[16:])
    with pytest.raises(ValueError):
        ops.interleave_gate_up(gate[:8], up[:8])


# -------------------------------------------------------------------- norms --

@dtypes
@pytest.mark.parametrize("rows,H", [(1, 1), (1, 2), (3, 7), (2, 8), (5, 100), (4, 999), (1, 2048), (130, 512), (7, 2050),
                                    (3, 4096), (2, 8191), (2, 8200), (1, 20001), (1, 32768)])
def test_rms_norm(dev, dt, rows, H):
    x, w = randn(H, rows, H, dt=dt), randn(H + 1, H, dt=dt)
    want = ref.rms(x.double(), w.double(), 1e-6)
    # f32: the sum of squares (H 2^-24 relative at worst, half of it after the root) and four roundings
    tol = ref.half_ulp(want, dt) * 1.01 + want.abs() * (H / 2 + 8) * 2.0 ** -24
    check(ops.rms_norm(x, w), want, tol)
    want = ref.rms(x.double(), None, 1e-6)
    check(ops.rms_norm(x), want, ref.half_ulp(want, dt) * 1.01 + want.abs() * (H / 2 + 8) * 2.0 ** -24)


@dtypes
@pytest.mark.parametrize("rows,H", [(1, 2048), (6, 96), (4, 333), (8, 1030), (12, 4096)])
@pytest.mark.parametrize("gates", ["none", "vector", "rows", "groups", "scalars"])
@pytest.mark.parametrize("norm,next_norm", [(True, True), (True, False), (False, True)])
def test_post_norm(dev, dt, rows, H, gates, norm, next_norm):
    h, y = randn(1, rows, H, dt=dt, std=4.0), randn(2, rows, H, dt=dt)
    w = randn(3, H, dt=dt) if norm else None
    wn = randn(4, H, dt=dt) if next_norm else None
    gate = {"none": None, "vector": randn(5, H, dt=dt), "rows": randn(5, rows, H, dt=dt),
            "groups": randn(5, max(1, rows // 2), H, dt=dt), "scalars": randn(5, rows, 1, dt=dt)}[gates]
    got = ops.post_norm(h, y, w, gate=gate, scale=0.7, next_weight=wn, eps=1e-5, norm=norm, next_norm=next_norm)
    g = 1.0 if gate is None else (gate if gate.dim() == 1 else gate.repeat_interleave(rows // gate.shape[0], 0)).double()
    z = ref.rms(y.double(), w.double(), 1e-5) if norm else y.double()
    add = 0.7 * g * z
    want = h.double() + add
    rel = (H / 2 + 16) * 2.0 ** -24
    slack = (add.abs() + want.abs()) * rel
    out, n = got if next_norm else (got, None)
    check(out, want, ref.half_ulp(want, dt) * 1.01 + slack)
    if next_norm:
        nw = ref.rms(want, wn.double(), 1e-5)
        f = (nw / want).abs().nan_to_num(0)
        check(n, nw, ref.half_ulp(nw, dt) * 1.01 + slack * f + nw.abs() * 2 * rel + 1e-30)


def test_post_norm_in_place_and_unaligned(dev):
    """In place, and rows that start at odd 2-byte offsets, give the same bits."""
    h, y, w, wn = randn(1, 6, 512), randn(2, 6, 512), randn(3, 512), randn(4, 512)
    want = ops.post_norm(h, y, w, next_weight=wn)
    hh, yy = h.clone(), y.clone()
    ops.post_norm(hh, yy, w, next_weight=wn, out=hh, next_out=yy)
    assert torch.equal(hh, want[0]) and torch.equal(yy, want[1])
    big = torch.empty(6 * 512 + 1, dtype=BF16, device="cuda")
    shifted = big[1:].view(6, 512)
    shifted.copy_(h)
    got = ops.post_norm(shifted, y, w, next_weight=wn)
    for a, b in zip(got, want):
        # another order of the f32 sums: at most one rounding apart
        assert ((a.double() - b.double()).abs() <= 2.1 * ref.half_ulp(b.double(), BF16)).all()


def test_norm_of_zero_and_of_nonfinite_rows(dev):
    x = randn(1, 3, 256)
    x[0] = 0
    x[1, 5] = float("inf")
    n = ops.rms_norm(x)
    assert not n[0].any()
    assert torch.isnan(n[1, 5]) and not n[1, :5].any()
    assert torch.isfinite(n[2]).all()
    assert ops.rms_norm(x[:0]).shape == (0, 256)


# ------------------------------------------------------------------ example --

@pytest.mark.parametrize("tokens,hidden,inner,experts,k", [(1, 512, 256, 8, 2), (70, 256, 512, 6, 3)])
def test_example_block(dev, tokens, hidden, inner, experts, k, capsys):
    """The example's block is near the same block with unrounded activations: an
    e2m1 value is within 1/6 of its block's scaled magnitude, errors of many
    elements average out, so a quarter of the MLP's share (about half of the
    residual stream's) bounds both outputs."""
    from examples.expert_block import main
    off = main(["--tokens", str(tokens), "--hidden", str(hidden), "--inner", str(inner), "--experts", str(experts),
                "--top-k", str(k)])
    assert off < 0.125
    assert "tokens through the block" in capsys.readouterr().out


# ----------------------------------------------- streams, graphs, refusals ---

def test_on_another_stream(dev):
    """A call on a stream that is not the current one uses that stream alone."""
    fmt = ops.FP4_NV
    x = randn(1, 64, 512)
    w, ws, wg, _ = weight(4, 1, 256, 512, fmt)
    want = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg, stream=s) for _ in range(20)]
    raw = ops.fp4_linear(x, w[0], ws[0], fmt, x_scale=SCALE[fmt], w_scale=wg, stream=s.cuda_stream)
    s.synchronize()
    for g in (*got, raw):
        assert torch.equal(g, want)


def test_in_a_cuda_graph(dev):
    """The whole expert block captured: replays follow new inputs."""
    fmt, T, E, k, H, I = ops.FP4_NV, 9, 8, 2, 256, 128
    x, logits = randn(1, T, H), randn(2, T, E, dt=torch.float32)
    gu, gus, gug, _ = weight(8, E, 2 * I, H, fmt)
    d, ds, dg, _ = weight(9, E, H, I, fmt)
    wn = randn(5, H)

    def block():
        n = ops.rms_norm(x, wn)
        y = ops.fp4_moe_mlp(n, ops.moe_route(logits, k), gu, gus, d, ds, fmt, x_scale=SCALE[fmt], h_scale=SCALE[fmt],
                            gu_scale=gug, d_scale=dg)
        return ops.post_norm(x, y, wn, next_weight=wn)
    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for seed in (3, 4):
        x.copy_(randn(seed, T, H))
        logits.copy_(randn(seed + 10, T, E, dt=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, block()):
            assert torch.equal(a, b)


def test_binding_refuses(dev):
    x = randn(1, 4, 64)
    codes, scales = ops.fp4_quantize(x, ops.FP4_NV)
    with pytest.raises(ops.QswError):
        ops.fp4_quantize(randn(1, 4, 48))                                  # K not a multiple of 32
    with pytest.raises(ops.QswError):
        ops.fp4_quantize(x, ops.FP4_MX, scale=2.0)                         # no tensor scale in this format
    with pytest.raises(ops.QswError):
        ops.fp4_quantize(x, ops.FP4_NV, scale=0.0)
    with pytest.raises(ValueError):
        ops.fp4_quantize(x, 5)
    with pytest.raises(TypeError):
        ops.fp4_quantize(x.float())
    with pytest.raises(ValueError):
        ops.fp4_quantize(x.t())
    with pytest.raises(ValueError):
        ops.fp4_dequantize(*ops.fp4_quantize(randn(1, 4, 256), ops.FP4_NV), ops.FP4_MX)   # the other format's scales
    with pytest.raises(ValueError):
        ops.fp4_linear(randn(1, 4, 96), codes, scales)
    with pytest.raises(TypeError):
        ops.fp4_linear(x, codes.view(torch.int8), scales)
    with pytest.raises(ValueError):
        ops.fp4_linear(x, codes, scales, w_scale=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        ops.fp4_grouped_linear(x, torch.tensor([0, 4], device="cuda"), codes[None], scales[None])
    with pytest.raises(ValueError):
        ops.moe_route(randn(1, 4, 8), 9)
    with pytest.raises(ops.QswError):
        ops.moe_route(randn(1, 2, 2000), 2)
    with pytest.raises(ValueError):
        ops.rms_norm(x, torch.ones(32, dtype=BF16, device="cuda"))
    with pytest.raises(ops.QswError):
        ops.rms_norm(randn(1, 1, 40000))
    with pytest.raises(ops.QswError):
        ops.post_norm(x, x, gate=randn(1, 3, 64))                          # 3 gate rows for 4 rows
    with pytest.raises(ops.QswError):
        ops.post_norm(x, x, weight=randn(1, 64), norm=False)
