"""The attention half of a decoder block over a paged cache, from its norm to the MLP's.

    python examples/attention_block.py [--prompt 300] [--steps 8] [--hidden 1024] [--heads 8] [--kv-heads 2]

Weights are drawn at random and held in 4 bits (16 codes per E4M3 scale).  Per step a
plan is made once for all layers; then, per layer:

    n = rms_norm(h)                                    the block's input
    q, k, v = fp4_linear(n, ...)                       one matrix
    q = kv_append(k, v, caches, plan, q=q)             rotation, k and v into the cache
    a = paged_attention(q, caches, plan)
    y = fp4_linear(a, ...)
    h, n = post_norm(h, y, norm=False, ...)            residual and the MLP's input

Two sequences of different lengths are prefilled in one step, then decoded token by token
with the step captured as a CUDA graph.  The result is compared with the same block in
f32 torch operations on the dequantised weights over the whole sequences at once (its
activations are not held in 4 bits, so the two differ by that rounding).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_swiglu_mlp_gb300 import ops  # noqa: E402


class AttentionBlock:
    """Weights of one block, held in 4 bits, and its cache."""

    def __init__(self, hidden, heads, kv_heads, head_dim, pages, page_size, dtype=torch.bfloat16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.norm, self.next = (1 + 0.1 * torch.randn(2, hidden, generator=g, device="cuda")).to(dtype)
        self.qkv = self.hold(torch.randn((heads + 2 * kv_heads) * head_dim, hidden, generator=g, device="cuda"), dtype)
        self.o = self.hold(torch.randn(hidden, heads * head_dim, generator=g, device="cuda"), dtype)
        self.frequencies = ops.rope_frequencies(head_dim)
        self.table = ops.rope_table(self.frequencies)
        shape = (pages, kv_heads, page_size, head_dim)
        self.k_cache, self.v_cache = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
        self.x_scale = 16 / (6 * 448)        # of activations, for a largest magnitude of 16

    @staticmethod
    def hold(w, dtype):
        """A matrix in 4 bits: codes, scales, its f32 scale on the device and on the host."""
        w = (w * w.shape[1] ** -0.5).to(dtype)
        g = float(w.abs().max()) / (6 * 448)
        return *ops.fp4_quantize(w, ops.FP4_NV, scale=g), torch.full((1,), g, device="cuda"), g

    def linear(self, x, w):
        return ops.fp4_linear(x, w[0], w[1], x_scale=self.x_scale, w_scale=w[2])

    def __call__(self, h, plan):
        n = ops.rms_norm(h, self.norm)
        qkv = self.linear(n, self.qkv).unflatten(1, (-1, self.head_dim))
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        q = ops.kv_append(k, v, self.k_cache, self.v_cache, plan.slots, plan.positions, self.table, q=q)
        a = ops.paged_attention(q, self.k_cache, self.v_cache, plan)
        return ops.post_norm(h, self.linear(a.flatten(1), self.o), norm=False, next_weight=self.next)

    def plain(self, h):
        """The block over one whole sequence h [tokens, hidden], in f32."""
        def norm(x, w):
            return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()

        def value(w):
            return ops.fp4_dequantize(w[0], w[1], scale=w[3]).float()
        h = h.float()
        qkv = (norm(h, self.norm) @ value(self.qkv).T).unflatten(1, (-1, self.head_dim))
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        angle = torch.arange(h.shape[0], device="cuda", dtype=torch.float64)[:, None] * self.frequencies.cuda()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turn(x):
            a, b = x.chunk(2, -1)
            return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        q, k = turn(q), turn(k)
        group = self.heads // self.kv_heads
        k, v = (x.repeat_interleave(group, 1) for x in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * self.head_dim ** -0.5
        s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), float("-inf"))
        a = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).flatten(1)
        h = h + a @ value(self.o).T
        return h, norm(h, self.next)


def run(hidden=512, heads=8, kv_heads=2, head_dim=64, prompts=(70, 9), steps=4, page_size=16):
    """(relative difference of h, of n) of a prefill and decoded steps against the plain block."""
    total = [p + steps for p in prompts]
    most = -(-max(total) // page_size)
    block = AttentionBlock(hidden, heads, kv_heads, head_dim, most * len(prompts), page_size)
    table = torch.randperm(most * len(prompts), device="cuda").int().view(len(prompts), most)
    hs = [torch.randn(t, hidden, device="cuda").bfloat16() for t in total]
    got = [([], []) for _ in prompts]

    def keep(out, counts):
        for result, parts in enumerate(zip(*(o.split(counts) for o in out))):
            for x, part in enumerate(parts):
                got[result][x].append(part.clone())

    # both prompts in one step
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, *prompts], device="cuda").cumsum(0).int()
    plan = ops.paged_plan(offsets, lengths, table, block.k_cache, sum(prompts), heads)
    keep(block(torch.cat([h[:p] for h, p in zip(hs, prompts)]), plan), prompts)

    # one token each: the captured step follows its inputs and lengths
    ones = torch.arange(len(prompts) + 1, device="cuda").int()
    h = torch.empty(len(prompts), hidden, dtype=torch.bfloat16, device="cuda")

    def step():
        return block(h, ops.paged_plan(ones, lengths, table, block.k_cache, len(prompts), heads))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h.copy_(torch.stack([x[p - 1] for x, p in zip(hs, prompts)]))
        step()                                    # (rewrites the prompts' last tokens with themselves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(steps):
        h.copy_(torch.stack([x[p + i] for x, p in zip(hs, prompts)]))
        lengths += 1
        graph.replay()
        keep(out, [1] * len(prompts))
    ops.qsw_check_device_errors()
    off = [0.0, 0.0]
    for h, parts in zip(hs, got):
        for x, want in enumerate(block.plain(h)):
            have = torch.cat(parts[x]).float()
            off[x] = max(off[x], float((have - want).norm() / want.norm()))
    return tuple(off)


def main():
    p = argparse.ArgumentParser()
    for name, default in (("prompt", 300), ("steps", 8), ("hidden", 1024), ("heads", 8), ("kv-heads", 2), ("head-dim", 128)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    off = run(a.hidden, a.heads, a.kv_heads, a.head_dim, (a.prompt, max(1, a.prompt // 7)), a.steps)
    print(f"prompts of {a.prompt} and {max(1, a.prompt // 7)} tokens and {a.steps} decoded: "
          f"h differs by {off[0]:.4f}, the MLP's input by {off[1]:.4f} of the f32 block's")


if __name__ == "__main__":
    main()
