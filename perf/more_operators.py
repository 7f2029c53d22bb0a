"""Measured cases of the operators of a decoder's attention half.

Three operators, each in two forms: with ``own`` false ``run`` computes the
operator from elementary torch operations, with ``own`` true it makes the calls
of ``quantized_swiglu_mlp_gb300.ops`` that a program makes.

  rope    rotary positions of queries or keys: half or interleaved pairs, the
          whole head or its first part, magnitude scaled for long contexts
  append  q rotated, k rotated and written with v to a paged cache
  attend  attention of new tokens over the paged cache, causal, with or without
          a sliding window, grouped heads

A cache is [pages, kv_heads, page_size, D]; a sequence's token p lies in row
p % page_size of page page_table[sequence, p // page_size].  The new tokens of a
sequence are its last ones.  The plan of a step (positions, cache rows, how long
histories are split) is made once per step and shared by all layers.
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of each of 64 sequences, far positions; a long prompt behind a cached half, half of each head
        # rotated, in adjacent pairs, frequencies divided by 4
        dict(name="rope_64_tokens", op="rope", T=64, heads=32, D=128, rot=128, interleaved=False, start=120000,
             spread=1017, factor=1.0, magnitude=1.0, dtype="bf16"),
        dict(name="rope_8192_part", op="rope", T=8192, heads=32, D=128, rot=64, interleaved=True, start=8192, spread=1,
             factor=4.0, magnitude=1.1386, dtype="f16"),
        # decoding: one sequence, then a batch; a prefill of four ragged prompts
        dict(name="append_1_token", op="append", B=1, new=1, new_to=1, old=500, old_to=500, heads=32, kv_heads=8,
             D=128, rot=128, page=16, interleaved=False, dtype="bf16"),
        dict(name="append_48_tokens_f16", op="append", B=48, new=1, new_to=1, old=10, old_to=900, heads=20, kv_heads=4,
             D=128, rot=128, page=24, interleaved=True, dtype="f16"),
        dict(name="append_prefill", op="append", B=4, new=1500, new_to=2500, old=0, old_to=200, heads=32, kv_heads=8,
             D=128, rot=128, page=64, interleaved=False, dtype="bf16"),
        # decoding: a few short sequences; one long one; a ragged batch
        dict(name="attend_decode_short", op="attend", B=4, new=1, new_to=1, old=20, old_to=180, heads=16, kv_heads=8,
             D=128, page=16, window=0, dtype="bf16"),
        dict(name="attend_decode_one_long", op="attend", B=1, new=1, new_to=1, old=40000, old_to=40000, heads=32,
             kv_heads=8, D=128, page=16, window=0, dtype="bf16"),
        dict(name="attend_decode_64", op="attend", B=64, new=1, new_to=1, old=128, old_to=16000, heads=32, kv_heads=8,
             D=128, page=64, window=0, dtype="bf16"),
        # checking 5 drafted tokens per sequence, 5 query heads per kv head
        dict(name="attend_draft_f16", op="attend", B=16, new=5, new_to=5, old=300, old_to=9000, heads=20, kv_heads=4,
             D=128, page=32, window=0, dtype="f16"),
        # a chunk of a long prompt; a whole prompt; decoding sequences among chunks, window, smaller heads
        dict(name="attend_chunk", op="attend", B=1, new=512, new_to=512, old=32000, old_to=32000, heads=32, kv_heads=8,
             D=128, page=128, window=0, dtype="bf16"),
        dict(name="attend_prefill", op="attend", B=1, new=8192, new_to=8192, old=0, old_to=0, heads=32, kv_heads=8,
             D=128, page=64, window=0, dtype="bf16"),
        dict(name="attend_mixed_window_f16", op="attend", B=24, new=1, new_to=400, old=0, old_to=6000, heads=16,
             kv_heads=16, D=64, page=48, window=1024, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1)))


def _sequences(c):
    """(new tokens, whole length) of each sequence: sizes of the case, the same for every seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    out = []
    for _ in range(c["B"]):
        n = _log_int(rng, c["new"], c["new_to"])
        out.append((n, n + _log_int(rng, c["old"], c["old_to"])))
    return out


def _cost(c):
    w = work(c)
    return w["bytes"] / 5e12 + w["flops"] / 1e15


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = dict(op=rng.choice(["rope", "append", "attend", "attend", "attend"]), dtype=rng.choice(["bf16", "f16"]))
        D = rng.choice([64, 80, 96, 128, 128])
        if c["op"] == "rope":
            c.update(T=_log_int(rng, 1, 8192), heads=rng.choice([1, 4, 8, 20, 32, 40]), D=D,
                     rot=rng.choice([D, D, D // 2, D // 4 * 2 - 2]), interleaved=rng.random() < 0.5,
                     start=_log_int(rng, 0, 200000), spread=_log_int(rng, 1, 100),
                     factor=rng.choice([1.0, 2.0, 8.0]), magnitude=rng.choice([1.0, 1.2]))
            return c
        kv_heads = rng.choice([1, 2, 4, 8])
        c.update(heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv_heads, D=D,
                 page=rng.choice([8, 16, 16, 24, 64, 128, 256]))
        if c["op"] == "append":
            new = _log_int(rng, 1, 2048)
            c.update(B=_log_int(rng, 1, 64), new=max(1, new // 3), new_to=new, old=0, old_to=_log_int(rng, 0, 1000),
                     rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.5)
        else:
            new = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 4096)])
            old = _log_int(rng, 1, 40000)
            c.update(B=_log_int(rng, 1, 64), new=rng.choice([1, new]), new_to=new, old=rng.choice([0, old // 20, old]),
                     old_to=old, window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]))
        tokens, rows = sum(n for n, _ in _sequences(c)), sum(t for _, t in _sequences(c))
        if tokens <= 16384 and rows * kv_heads * D <= 3e8 and _cost(c) <= top:
            return c


def _seen(c, n, total):
    """(keys of a sequence that some new token sees, pairs of new token and key)."""
    w = c["window"]
    pairs = sum(min(p + 1, w) if w else p + 1 for p in range(total - n, total))
    return min(total, n + w - 1) if w else total, pairs


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["heads"] * c["D"]
        return {"bytes": 4 * n + 4 * c["T"], "flops": 3.0 * n}
    tokens = sum(n for n, _ in _sequences(c))
    if c["op"] == "append":
        n = tokens * (c["heads"] + 2 * c["kv_heads"]) * c["D"]
        return {"bytes": 4 * n + 8 * tokens, "flops": 3.0 * n}
    keys, pairs = map(sum, zip(*(_seen(c, n, t) for n, t in _sequences(c))))
    return {"bytes": 4 * tokens * c["heads"] * c["D"] + 4 * keys * c["kv_heads"] * c["D"],
            "flops": 4.0 * pairs * c["heads"] * c["D"]}


def _frequencies(rot, factor):
    """Angle per position of each pair, f64."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return 10000.0 ** (-2.0 * i / rot) / factor


# ------------------------------------------------------------- plain forms --

def _rotated(x, positions, frequencies, interleaved, magnitude):
    """f32 [T, heads, D] -> rotated; angles in 64 bits."""
    half = frequencies.numel()
    angle = positions.double()[:, None] * frequencies
    cos, sin = (torch.cos(angle) * magnitude).float()[:, None], (torch.sin(angle) * magnitude).float()[:, None]
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _attend_rows(q, k, v, first, window, scale):
    """f32 q [kv_heads, tokens, group, D], the tokens at positions first, first + 1, ...; k, v [kv_heads, keys, D]."""
    j = torch.arange(k.shape[1], device=q.device)
    at = first + torch.arange(q.shape[1], device=q.device)[:, None]
    seen = j <= at
    if window:
        seen &= j > at - window
    s = (q.flatten(1, 2) @ k.transpose(1, 2)).unflatten(1, (-1, q.shape[2])) * scale
    s = torch.where(seen[None, :, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(1, 2) @ v).unflatten(1, (-1, q.shape[2]))
    return o / torch.where(total == 0, 1.0, total)


def _plain(s):
    c = s["case"]
    t = DTYPE[c["dtype"]]
    if c["op"] == "rope":
        return _rotated(s["x"].float(), s["positions"], s["frequencies"], c["interleaved"], c["magnitude"]).to(t)
    if c["op"] == "append":
        q, k = (_rotated(s[n].float(), s["positions"], s["frequencies"], c["interleaved"], 1.0).to(t) for n in "qk")
        page, row = s["slots"] // c["page"], s["slots"] % c["page"]
        s["k_cache"][page, :, row] = k
        s["v_cache"][page, :, row] = s["v"]
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out = torch.empty_like(s["q"])
    at = 0
    for b, (n, total) in enumerate(_sequences(c)):
        pages = s["page_table"][b, :-(-total // c["page"])].long()
        k, v = (s[x][pages].transpose(0, 1).flatten(1, 2)[:, :total].float() for x in ("k_cache", "v_cache"))
        q = s["q"][at:at + n].float().unflatten(1, (c["kv_heads"], -1)).transpose(0, 1)
        step = max(1, int(2.5e8) // (c["heads"] * total))
        for i in range(0, n, step):
            o = _attend_rows(q[:, i:i + step], k, v, total - n + i, c["window"], s["scale"])
            out[at + i:at + i + o.shape[1]] = o.transpose(0, 1).flatten(1, 2).to(t)
        at += n
    return out


# ------------------------------------------------------------------- cases --

def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    t = DTYPE[c["dtype"]]

    def normal(*shape, of=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=t) * of

    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = normal(c["T"], c["heads"], c["D"])
        s["positions"] = c["start"] + c["spread"] * torch.arange(c["T"], dtype=torch.int32, device="cuda")
        s["frequencies"] = _frequencies(c["rot"], c["factor"]).cuda()
        if own:
            from quantized_swiglu_mlp_gb300 import ops
            s["table"] = ops.rope_table(s["frequencies"])
        return s
    # every sequence's pages lie scattered over the cache; what no sequence holds is old data
    D, H, KV, P = c["D"], c["heads"], c["kv_heads"], c["page"]
    seqs = _sequences(c)
    counts = [-(-total // P) for _, total in seqs]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")[:sum(counts)].int()
    s["page_table"] = torch.full((len(seqs), max(counts)), -1, dtype=torch.int32, device="cuda")
    for b, own_pages in enumerate(order.split(counts)):
        s["page_table"][b, :counts[b]] = own_pages
    s["offsets"] = torch.tensor([0] + [n for n, _ in seqs], device="cuda").cumsum(0).int()
    s["lengths"] = torch.tensor([total for _, total in seqs], dtype=torch.int32, device="cuda")
    T = sum(n for n, _ in seqs)
    s["k_cache"], s["v_cache"] = normal(pages, KV, P, D), normal(pages, KV, P, D)
    if c["op"] == "append":
        # the projections come as one matrix
        qkv = normal(T, (H + 2 * KV) * D).unflatten(1, (-1, D))
        s["q"], s["k"], s["v"] = qkv.split((H, KV, KV), 1)
        s["frequencies"] = _frequencies(c["rot"], 1.0).cuda()
        where = [(b, p) for b, (n, total) in enumerate(seqs) for p in range(total - n, total)]
        b, p = torch.tensor(where, device="cuda").unbind(1)
        s["positions"] = p.int()
        s["slots"] = s["page_table"][b, p // P].long() * P + p % P
    else:
        # scores of standard deviation 2.5
        s["q"] = normal(T, H, D, of=2.5)
        s["scale"] = D ** -0.5
    if own:
        from quantized_swiglu_mlp_gb300 import ops
        s["plan"] = ops.paged_plan(s["offsets"], s["lengths"], s["page_table"], s["k_cache"], T, H,
                                   window=c.get("window", 0))
        if c["op"] == "append":
            s["table"] = ops.rope_table(s["frequencies"])
    return s


def run(s):
    if not own:
        return _plain(s)
    from quantized_swiglu_mlp_gb300 import ops
    c = s["case"]
    if c["op"] == "rope":
        return ops.rope(s["x"], s["positions"], s["table"], interleaved=c["interleaved"], scale=c["magnitude"])
    plan = s["plan"]
    if c["op"] == "append":
        q = ops.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], plan.slots, plan.positions, s["table"],
                          q=s["q"], interleaved=c["interleaved"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return ops.paged_attention(s["q"], s["k_cache"], s["v_cache"], plan, scale=s["scale"])


# ------------------------------------------------------------ 64-bit values --

def _turned(x, positions, rot, factor, interleaved, magnitude):
    """x (float64) with the pairs of its first `rot` elements as complex numbers times magnitude e^(i angle)."""
    pair = torch.arange(rot // 2, device=x.device)
    first, second = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + rot // 2)
    angle = torch.outer(positions.double(), torch.exp(-math.log(10000.0) * pair.double() * 2 / rot) / factor)
    z = torch.complex(x[:, :, first], x[:, :, second])
    z = z * torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
    y = x.clone()
    y[:, :, first], y[:, :, second] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _turned(s["x"].double(), s["positions"], c["rot"], c["factor"], c["interleaved"], c["magnitude"])
    if c["op"] == "append":
        k = _turned(s["k"].double(), s["positions"], c["rot"], 1.0, c["interleaved"], 1.0)
        held = {n: s[n].double() for n in ("k_cache", "v_cache")}
        flat = {n: v.transpose(1, 2).flatten(0, 1) for n, v in held.items()}
        flat["k_cache"][s["slots"]] = k
        flat["v_cache"][s["slots"]] = s["v"].double()
        pages = {n: v.unflatten(0, (-1, c["page"])).transpose(1, 2).contiguous() for n, v in flat.items()}
        return {"q": _turned(s["q"].double(), s["positions"], c["rot"], 1.0, c["interleaved"], 1.0), **pages}
    if work(c)["flops"] > 2e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, total) in enumerate(_sequences(c)):
        p = torch.arange(total, device="cuda")
        where = (s["page_table"][b, p // c["page"]].long(), p % c["page"])
        for h in range(c["heads"]):
            kv = h * c["kv_heads"] // c["heads"]
            k, v = (s[x][where[0], kv, where[1]].double() for x in ("k_cache", "v_cache"))
            for i in range(0, n, 4096):
                m = min(4096, n - i)
                score = s["q"][row + i:row + i + m, h].double() @ k.T / math.sqrt(c["D"])
                behind = (total - n + i + torch.arange(m, device="cuda"))[:, None] - p[None]
                gone = behind < 0
                if c["window"]:
                    gone |= behind >= c["window"]
                weights = torch.softmax(score.masked_fill(gone, -math.inf), 1)
                out[row + i:row + i + m, h] = weights @ v
        row += n
    return out
