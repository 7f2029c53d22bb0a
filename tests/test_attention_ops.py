"""Rotary positions, the paged cache and attention over it on the GPU, against plain
float64 implementations."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
dtypes = pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])


@pytest.fixture(scope="module", autouse=True)
def dev():
    torch.cuda.set_device(0)
    ops.load_native()
    yield torch.device("cuda:0")
    ops.qsw_check_device_errors()


def randn(seed, *shape, dt=BF16, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def check(got, want, bound, what=""):
    same = (got.double() == want) | (got.isnan() & want.isnan())
    err = (got.double() - want).abs()
    bad = ~(same | (err <= bound))
    assert not bad.any(), (what, int(bad.sum()), float((err / bound)[bad].max()), bad.nonzero()[:4].tolist())


# ----------------------------------------------------------------- rotation --

@dtypes
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("T,heads,D,rot", [(1, 1, 64, 64), (3, 5, 128, 128), (1000, 8, 128, 64), (37, 3, 80, 80),
                                           (5, 2, 96, 46), (2, 3, 7, 6), (4, 1, 256, 16), (9, 2, 64, 0),
                                           (2500, 2, 72, 24), (9000, 1, 1024, 1024), (700, 1, 1022, 1020)])
def test_rope(dt, interleaved, T, heads, D, rot):
    x = randn(T + D, T, heads, D, dt=dt)
    f = ops.rope_frequencies(rot) if rot else torch.zeros(0)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(-2 ** 31, 2 ** 31, (T,), generator=g).int().cuda()
    pos[::2] = pos[::2] % 5000
    table = ops.rope_table(f, device="cuda")
    want, bound = ref.rope(x, pos, f, interleaved, 1.25)
    # what f64 loses itself: 2^-53 of the angle, twice
    size = x.double().abs().amax() * 3
    check(ops.rope(x, pos, table, interleaved, 1.25), want, bound + size * pos.double().abs()[:, None, None] * 2.0 ** -51)
    same = x.clone()
    assert ops.rope(same, pos, table, interleaved, 1.25, out=same).data_ptr() == same.data_ptr()
    assert torch.equal(same, ops.rope(x, pos, table, interleaved, 1.25))


@dtypes
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("shift", [0, 1, 4, 8])
def test_rope_of_strided_heads(dt, interleaved, shift):
    """Heads of one projection, aligned to 16, 8 and 2 bytes, into strided heads."""
    buf = randn(1, 40, shift + 9 * 64 + 3 * shift, dt=dt)
    x = buf[:, shift:shift + 6 * 64].unflatten(1, (6, 64))
    out = torch.zeros(6, 40, 64, dtype=dt, device="cuda").transpose(0, 1)
    pos, f = ints(range(40)), ops.rope_frequencies(48, 500000.0)
    keep = buf.clone()
    ops.rope(x, pos, ops.rope_table(f), interleaved, out=out)
    check(out, *ref.rope(x, pos, f, interleaved))
    assert torch.equal(buf, keep)
    want = out.clone()
    ops.rope(x, pos, ops.rope_table(f), interleaved, out=x)
    assert torch.equal(x, want)
    keep[:, shift:shift + 6 * 64] = want.flatten(1)
    assert torch.equal(buf, keep)


def test_rotation_there_and_back():
    x = randn(5, 300, 4, 128, dt=F16)
    pos = ints(range(0, 300 * 4001, 4001))
    table = ops.rope_table(ops.rope_frequencies(128))
    back = ops.rope(ops.rope(x, pos, table), -pos, table)
    # two roundings of values up to sqrt(2) times the pair's, and the f32 work of both
    size = x.double().unflatten(-1, (2, 64)).norm(dim=-2).repeat(1, 1, 2)
    check(back, x.double(), 3 * size * ref.HALF[F16] + size * 2.0 ** -19 + 4 * ref.TINY[F16])


# ---------------------------------------------------------- cache and plan --

class Step:
    """Sequences in a paged cache, pages scattered over it; `spare` pages belong to nobody."""

    def __init__(self, seqs, heads, kv_heads, D, page_size, dt=BF16, window=0, spare=2, seed=1, behind=0, strided=False):
        self.seqs, self.heads, self.window = seqs, heads, window
        self.lengths = [total for _, total in seqs]
        self.offsets = [0]
        for n, _ in seqs:
            self.offsets.append(self.offsets[-1] + n)
        self.tokens = self.offsets[-1] + behind
        counts = [max(0, -(-total // page_size)) for total in self.lengths]
        pages = sum(counts) + spare
        g = torch.Generator("cuda").manual_seed(seed)
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.table = torch.full((len(seqs), max(counts + [1])), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        if strided:      # rows of all heads together, keys and values in one buffer
            both = randn(seed + 1, pages, page_size, 2, kv_heads, D, dt=dt)
            self.k, self.v = (both[:, :, i].transpose(1, 2) for i in range(2))
        else:
            self.k, self.v = (randn(seed + i, pages, kv_heads, page_size, D, dt=dt) for i in (1, 2))
        self.q = randn(seed + 3, self.tokens, heads, D, dt=dt, std=2.5)
        self.scale = D ** -0.5

    def plan(self):
        return ops.paged_plan(ints(self.offsets), ints(self.lengths), self.table, self.k, self.tokens, self.heads,
                              window=self.window)

    def attend(self, plan=None, out=None):
        return ops.paged_attention(self.q, self.k, self.v, plan or self.plan(), self.scale, out=out)

    def want(self):
        return ref.attention(self.q, self.k, self.v, self.offsets, self.lengths, self.table, self.scale, self.window)

    def check(self):
        out = torch.full_like(self.q, 7.0)
        self.attend(out=out)
        n = self.offsets[-1]
        assert (out[n:] == 7.0).all()
        want, bound = self.want()
        check(out[:n], want[:n], bound[:n])
        return out


SEQS = {
    "one": [(1, 1)],
    "one_token_of_300": [(1, 300)],
    "prompt_100": [(100, 100)],
    "decode": [(1, 17), (1, 1), (1, 16), (1, 400), (1, 65)],
    "with_empty": [(0, 5), (3, 3), (0, 0), (2, 50), (0, 9)],
    "no_keys": [(2, 0), (5, 3), (1, 1)],
    "mixed": [(1, 700), (90, 90), (7, 263), (33, 500)],
}


@pytest.mark.parametrize("page_size", [8, 24, 64])
@pytest.mark.parametrize("name", SEQS)
def test_plan(name, page_size):
    s = Step(SEQS[name], 4, 2, 64, page_size, behind=3)
    s.table[0, 0] = 10 ** 6          # a page outside the cache
    p = s.plan()
    pos, slots = ref.plan(s.offsets, s.lengths, s.table.tolist(), page_size, s.k.shape[0], s.tokens)
    assert p.positions.tolist() == pos
    assert p.slots.tolist() == slots


@dtypes
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("strided", [False, True], ids=["dense", "strided"])
@pytest.mark.parametrize("name,page_size,D,rot", [("decode", 16, 128, 128), ("mixed", 24, 64, 30), ("no_keys", 8, 80, 80),
                                                  ("with_empty", 64, 96, 32), ("prompt_100", 8, 128, 0)])
def test_append(dt, interleaved, strided, name, page_size, D, rot):
    s = Step(SEQS[name], 6, 2, D, page_size, dt=dt, behind=2, strided=strided)
    p = s.plan()
    qkv = randn(9, s.tokens, 10 * D, dt=dt).unflatten(1, (10, D))
    q, k, v = qkv.split((6, 2, 2), 1)
    f = ops.rope_frequencies(rot) if rot else torch.zeros(0)
    table = ops.rope_table(f, device="cuda") if rot else None
    kc, vc = s.k.clone(), s.v.clone()
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    got = ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table, q=q, interleaved=interleaved, q_out=out)
    assert got.data_ptr() == out.data_ptr()
    live = p.positions >= 0
    want, bound = ref.rope(q, p.positions, f, interleaved)
    check(out[live], want[live], bound[live])
    assert (out[~live] == 7.0).all()
    want, bound = ref.rope(k, p.positions, f, interleaved)
    for t in range(s.tokens):
        slot = int(p.slots[t])
        if slot >= 0:
            row = slot // page_size, slice(None), slot % page_size
            check(s.k[row], want[t], bound[t], t)
            assert torch.equal(s.v[row], v[t])
            kc[row], vc[row] = s.k[row], s.v[row]
    assert torch.equal(s.k, kc) and torch.equal(s.v, vc)       # and nothing else
    # q in its own place; without q
    assert ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table, interleaved=interleaved) is None
    ops.kv_append(k, v, s.k, s.v, p.slots, p.positions, table, q=q, interleaved=interleaved, q_out=q)
    assert torch.equal(q[live], out[live])
    assert torch.equal(s.k, kc) and torch.equal(s.v, vc)


def test_append_leaves_out_bad_slots():
    k, v = randn(1, 6, 2, 64), randn(2, 6, 2, 64)
    kc, vc = torch.zeros(3, 2, 8, 64, dtype=BF16, device="cuda"), torch.zeros(3, 2, 8, 64, dtype=BF16, device="cuda")
    ops.kv_append(k, v, kc, vc, ints([-1, 24, 2 ** 31 - 1, -2 ** 31, 23, 0]))
    assert torch.equal(kc[2, :, 7], k[4]) and torch.equal(vc[0, :, 0], v[5])
    assert int((kc != 0).any(-1).sum()) == int((vc != 0).any(-1).sum()) == 4


# ---------------------------------------------------------------- attention --

@dtypes
@pytest.mark.parametrize("heads,kv_heads,D", [(4, 4, 64), (8, 2, 128), (5, 1, 80), (32, 1, 128), (6, 2, 8), (3, 1, 104)])
@pytest.mark.parametrize("name", SEQS)
def test_attention(dt, heads, kv_heads, D, name):
    Step(SEQS[name], heads, kv_heads, D, 16, dt=dt, behind=2).check()


@pytest.mark.parametrize("window", [1, 15, 64, 200, 10 ** 9])
@pytest.mark.parametrize("page_size", [8, 24, 256])
@pytest.mark.parametrize("name", SEQS)
def test_attention_windows_and_pages(name, page_size, window):
    Step(SEQS[name], 8, 2, 64, page_size, window=window).check()


@pytest.mark.parametrize("name", ["decode", "mixed"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_of_strided_tensors(name, D):
    s = Step(SEQS[name], 8, 2, D, 16, strided=True)
    s.q = randn(3, s.tokens, 12 * D, std=2.5).unflatten(1, (12, D))[:, 2:10]
    s.check()
    wide = torch.full((s.table.shape[0], s.table.shape[1] + 5), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, :s.table.shape[1]] = s.table
    s.table = wide[:, :s.table.shape[1]]
    s.check()


@dtypes
@pytest.mark.parametrize("heads,kv_heads,seqs", [(8, 1, [(1, 30011)]), (32, 8, [(1, 5000), (1, 3), (1, 12345)]),
                                                 (4, 2, [(3, 20000), (0, 0), (1, 100)]), (8, 2, [(200, 9000)]),
                                                 (4, 1, [(300, 300), (700, 2500)])])
def test_attention_over_long_histories(dt, heads, kv_heads, seqs):
    """Split over CTAs and joined: the same bits again."""
    s = Step(seqs, heads, kv_heads, 128, 32, dt=dt)
    assert torch.equal(s.check(), s.check())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("seqs", [[(1, 37), (5, 100)], [(1, 20000)], [(70, 300)], [(300, 300)], [(40, 9000)]], ids=str)
def test_nothing_unseen_has_an_effect(seqs, window, value):
    """Infinities and NaN past the end of a sequence, in pages of nobody, in keys that only
    later tokens see and in those before the window."""
    s = Step(seqs, 8, 2, 64, 24, window=window)
    clean = s.check()
    kc, vc = s.k.clone(), s.v.clone()
    s.k.fill_(value), s.v.fill_(value)
    for b, (n, total) in enumerate(seqs):
        first = max(0, total - n - window + 1) if window else 0
        p = torch.arange(first, total, device="cuda")
        rows = s.table[b].long()[p // 24], slice(None), p % 24
        s.k[rows], s.v[rows] = kc[rows], vc[rows]
    assert torch.equal(s.attend(), clean)
    # the last token's own key and value: only it sees them
    b = len(seqs) - 1
    total = seqs[b][1]
    row = int(s.table[b, (total - 1) // 24]), slice(None), (total - 1) % 24
    s.v[row] = value
    # (the rows of its tile are summed again with f32 weights: the same within the bound, not to
    # the bit)
    got = s.attend()
    want, bound = s.want()
    check(got[:-1], want[:-1], bound[:-1])
    assert torch.equal(got[-1].isnan(), want[-1].isnan()) and torch.equal(got[-1].isinf(), want[-1].isinf())
    s.v[row] = vc[row]
    s.k[row] = value
    got = s.attend()
    check(got[:-1], want[:-1], bound[:-1])


def test_pages_outside_the_cache_count_as_zeros():
    s = Step([(1, 200), (60, 90), (1, 9000)], 8, 2, 128, 16)
    s.table[0, 3] = -1
    s.table[0, 5] = s.k.shape[0]
    s.table[1, 2] = 2 ** 31 - 1
    s.table[1, 5] = -2 ** 31
    s.table[2, 100:300] = -7
    s.check()


def test_lengths_and_offsets_of_any_values():
    """Lengths beyond the table and below 0 are taken as its end and 0; backward and far
    offsets read and write nothing out of range."""
    s = Step([(2, 64), (3, 40), (1, 10)], 4, 2, 64, 16)
    s.lengths = [2 ** 31 - 1, -5, 10 ** 6]
    s.check()
    guard = torch.full((s.tokens + 200, 4, 64), 7.0, dtype=BF16, device="cuda")
    out = guard[100:100 + s.tokens]
    for offsets in ([5, 3, 1, 0], [-2 ** 31, 2 ** 31 - 1, -1, 2 ** 31 - 1], [6, 6, 6, 6], [0, 2 ** 30, 0, 6]):
        plan = ops.paged_plan(ints(offsets), ints([64, 40, 10]), s.table, s.k, s.tokens, 4)
        assert int(plan.positions.min()) >= -1 and int(plan.slots.max()) < s.k.shape[0] * 16
        s.attend(plan, out=out)
        assert (guard[:100] == 7.0).all() and (guard[100 + s.tokens:] == 7.0).all()


def test_no_tokens():
    s = Step([(0, 40), (0, 0)], 4, 2, 64, 16)
    p = s.plan()
    assert s.attend(p).shape == (0, 4, 64) and p.slots.numel() == 0
    ops.kv_append(s.q[:, :2], s.q[:, :2], s.k, s.v, p.slots, p.positions)
    assert ops.rope(s.q, p.positions, ops.rope_table([1.0])).shape == (0, 4, 64)
    # tokens that belong to no sequence
    s = Step([(0, 40)], 4, 2, 64, 16, behind=5)
    s.check()


# ------------------------------------------------------------ run together --

def test_a_decoder_step_by_step():
    """A prompt in chunks, then token by token, through rotation, append and attention: the
    rows of one pass over the whole sequence."""
    heads, kv_heads, D, page, total = 8, 2, 128, 16, 150
    qkv = randn(4, total, (heads + 2 * kv_heads) * D).unflatten(1, (-1, D))
    f = ops.rope_frequencies(D, scaling="linear", factor=2.0)
    table = ops.rope_table(f)

    def passes(sizes):
        kc, vc = (torch.full((12, kv_heads, page, D), math.nan, dtype=BF16, device="cuda") for _ in range(2))
        pages = ints([[7, 2, 9, 4, 1, 11, 0, 3, 10, 5, 8, 6]])
        out, at = [], 0
        for n in sizes:
            q, k, v = qkv[at:at + n].split((heads, kv_heads, kv_heads), 1)
            at += n
            plan = ops.paged_plan(ints([0, n]), ints([at]), pages, kc, n, heads)
            q = ops.kv_append(k, v, kc, vc, plan.slots, plan.positions, table, q=q)
            out.append(ops.paged_attention(q, kc, vc, plan))
        return torch.cat(out), kc, vc, pages

    whole, kc, vc, pages = passes([total])
    steps, kc2, vc2, _ = passes([100, 33] + [1] * 17)
    assert torch.equal(kc[pages[0, :9].long()], kc2[pages[0, :9].long()])
    pos = ints(range(total))
    q = ref.rope(qkv[:, :heads], pos, f)[0].to(BF16)
    want, bound = ref.attention(q, kc, vc, [0, total], [total], pages, D ** -0.5)
    # (q as rounded by the library may be the next number where the f64 value is a tie)
    extra = 2.0 ** -8 * want.abs().amax()
    check(whole, want, bound + extra)
    check(steps, want, bound + extra)


def test_captured_and_replayed_with_other_lengths():
    s = Step([(1, 90), (1, 31), (4, 200)], 8, 2, 128, 16)
    lengths, offsets = ints(s.lengths), ints(s.offsets)
    out = torch.empty_like(s.q)

    def step():
        plan = ops.paged_plan(offsets, lengths, s.table, s.k, s.tokens, 8)
        ops.paged_attention(s.q, s.k, s.v, plan, s.scale, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([90, 31, 200], [1, 17, 150], [96, 5, 4]):
        s.lengths = new
        lengths.copy_(ints(new))
        graph.replay()
        check(out, *s.want())


def test_one_plan_on_two_streams():
    s = Step([(1, 9000), (1, 7000)], 8, 2, 128, 16)
    plan = s.plan()
    want = s.attend(plan)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[ops.paged_attention(s.q, s.k, s.v, plan, s.scale, stream=st) for _ in range(20)] for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for part in got for x in part)


def test_refusals():
    s = Step([(1, 90)], 8, 2, 64, 16)
    plan = s.plan()
    table = ops.rope_table(ops.rope_frequencies(64))
    bad = [
        (ValueError, lambda: ops.paged_attention(s.q[:, :4], s.k, s.v, plan)),
        (ValueError, lambda: ops.paged_attention(s.q, s.k[:-1], s.v[:-1], plan)),
        (ValueError, lambda: ops.paged_attention(s.q, s.k, s.v[:, :1], plan)),
        (ValueError, lambda: ops.paged_attention(s.q, s.k.transpose(2, 3), s.v.transpose(2, 3), plan)),
        (ValueError, lambda: ops.paged_attention(s.q.cpu(), s.k, s.v, plan)),
        (TypeError, lambda: ops.paged_attention(s.q.half(), s.k, s.v, plan)),
        (TypeError, lambda: ops.paged_attention(s.q.float(), s.k.float(), s.v.float(), plan)),
        (TypeError, lambda: ops.paged_attention(s.q, s.k, s.v, None)),
        (ValueError, lambda: ops.paged_attention(s.q, s.k, s.v, plan, out=s.q[:, :, :32])),
        (ops.QswError, lambda: ops.paged_attention(s.q, s.k, s.v, plan, scale=0.0)),
        (ops.QswError, lambda: ops.paged_attention(s.q, s.k, s.v, plan, scale=math.inf)),
        (ops.QswError, lambda: ops.paged_attention(torch.zeros(9 * 64 + 8, dtype=BF16, device="cuda")[1:513].view(1, 8, 64),
                                                   s.k, s.v, plan)),
        (ops.QswError, lambda: ops.paged_plan(ints([0, 1]), ints([90]), s.table, s.k, 1, 7)),
        (ops.QswError, lambda: ops.paged_plan(ints([0, 1]), ints([90]), s.table, s.k, 1, 8, window=-1)),
        (ops.QswError, lambda: ops.paged_plan(ints([0, 1]), ints([90]), s.table, s.k, 1 << 23, 8)),
        (ValueError, lambda: ops.paged_plan(ints([0, 1]), ints([90]), s.table, s.k, -1, 8)),
        (ValueError, lambda: ops.paged_plan(ints([0, 1, 1]), ints([90]), s.table, s.k, 1, 8)),
        (ValueError, lambda: ops.paged_plan(ints([0, 1]), ints([90, 1]), s.table, s.k, 1, 8)),
        (TypeError, lambda: ops.paged_plan(ints([0, 1]), ints([90], torch.int64), s.table, s.k, 1, 8)),
        (TypeError, lambda: ops.paged_plan(ints([0, 1]), ints([90]), s.table.long(), s.k, 1, 8)),
        (ops.QswError, lambda: ops.paged_plan(ints([0, 1]), ints([90]), s.table, s.k[:, :, :12], 1, 8)),
        (ValueError, lambda: ops.rope(s.q, None, table)),
        (ValueError, lambda: ops.rope(s.q, ints([0, 1]), table)),
        (TypeError, lambda: ops.rope(s.q, ints([0], torch.int64), table)),
        (TypeError, lambda: ops.rope(s.q, ints([0]), table.int())),
        (ValueError, lambda: ops.rope(s.q[..., :32], ints([0]), table)),
        (ValueError, lambda: ops.rope(s.q.transpose(1, 2), ints([0]), table[:1])),
        (ops.QswError, lambda: ops.rope(s.q, ints([0]), table, scale=math.nan)),
        (ValueError, lambda: ops.kv_append(s.q[:, :2], s.q[:, :3], s.k, s.v, ints([0]))),
        (ValueError, lambda: ops.kv_append(s.q[:, :3], s.q[:, :3], s.k, s.v, ints([0]))),
        (ValueError, lambda: ops.kv_append(s.q[:, :2], s.q[:, :2], s.k, s.v, ints([0, 1]))),
        (ValueError, lambda: ops.kv_append(s.q[:, :2], s.q[:, :2], s.k, s.v, ints([0]), q_out=s.q)),
        (ValueError, lambda: ops.kv_append(s.q[:, :2], s.q[:, :2], s.k, s.v, ints([0]), table=table)),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was accepted")
