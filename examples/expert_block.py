"""One mixture-of-experts MLP block of a decoder, from its norm to the next block's.

    python examples/expert_block.py [--tokens 4] [--hidden 1024] [--inner 512] [--experts 16] [--top-k 4]

Weights are drawn at random, held in 4 bits (16 codes per E4M3 scale) and put in
the layout of the expert kernels once; then, per call:

    n = rms_norm(h)                                  the block's input
    r = moe_route(n . Wr^T)                          experts of each token
    y = fp4_moe_mlp(n, r, ...)                       their SwiGLU MLPs, weighted
    h, n = post_norm(h, y, gate, scale, ...)         residual and the next block's input

The result is compared with the same block in f32 torch operations on the
dequantised weights (its activations are not held in 4 bits, so the two differ
by the format's rounding of the activations), and timed as a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_swiglu_mlp_gb300 import ops  # noqa: E402


class ExpertBlock:
    """Weights of one block, held in 4 bits."""

    def __init__(self, hidden, inner, experts, top_k, dtype=torch.bfloat16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(dtype)

        self.top_k = top_k
        self.norm, self.post, self.next = (1 + 0.1 * torch.randn(3, hidden, generator=g, device="cuda")).to(dtype)
        self.gate = torch.rand(hidden, generator=g, device="cuda").to(dtype)
        self.router = normal(experts, hidden)
        self.gu, self.gu_scales, self.gu_scale = self.hold(ops.interleave_gate_up(normal(experts, inner, hidden),
                                                                                  normal(experts, inner, hidden)))
        self.d, self.d_scales, self.d_scale = self.hold(normal(experts, hidden, inner))
        # scales of the activations, for largest magnitudes of 16 and 32
        self.x_scale, self.h_scale = 16 / (6 * 448), 32 / (6 * 448)

    @staticmethod
    def hold(w):
        """A stack of matrices in 4 bits, one f32 scale for all of them."""
        g = float(w.abs().max()) / (6 * 448)
        codes, scales = ops.fp4_quantize(w.contiguous(), ops.FP4_NV, scale=g)
        return codes, scales, torch.full((w.shape[0],), g, device=w.device)

    def __call__(self, h):
        n = ops.rms_norm(h, self.norm)
        r = ops.moe_route((n @ self.router.T).float(), self.top_k)
        y = ops.fp4_moe_mlp(n, r, self.gu, self.gu_scales, self.d, self.d_scales, x_scale=self.x_scale,
                            h_scale=self.h_scale, gu_scale=self.gu_scale, d_scale=self.d_scale)
        return ops.post_norm(h, y, self.post, gate=self.gate, scale=0.5, next_weight=self.next)

    def plain(self, h):
        """The same block in f32, activations not held in 4 bits."""
        def rms(v, w):
            return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.float()

        gu = ops.fp4_dequantize(self.gu, self.gu_scales, scale=float(self.gu_scale[0])).float()
        d = ops.fp4_dequantize(self.d, self.d_scales, scale=float(self.d_scale[0])).float()
        hf = h.float()
        n = rms(hf, self.norm)
        # the logits of the call above: a rounding of n may decide between two experts
        logits = (ops.rms_norm(h, self.norm) @ self.router.T).float()
        ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :self.top_k]
        p = torch.softmax(logits, -1).gather(1, ids)
        p = p / p.sum(-1, keepdim=True)
        y = torch.zeros_like(hf)
        for j in range(self.top_k):
            pair = torch.einsum("th,tfh->tf", n, gu[ids[:, j]]).unflatten(-1, (-1, 2, 16))
            hidden = (torch.nn.functional.silu(pair[:, :, 0]) * pair[:, :, 1]).flatten(1)
            y += p[:, j, None] * torch.einsum("tf,thf->th", hidden, d[ids[:, j]])
        out = hf + 0.5 * self.gate.float() * rms(y, self.post)
        return out, rms(out, self.next)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4), ("hidden", 1024), ("inner", 512), ("experts", 16), ("top-k", 4)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args(argv)
    block = ExpertBlock(a.hidden, a.inner, a.experts, a.top_k)
    h = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    got, want = block(h), block.plain(h)
    ops.qsw_check_device_errors()
    off = [float((g.float() - w).norm() / w.norm()) for g, w in zip(got, want)]
    print(f"residual stream off by {off[0]:.4f}, next input by {off[1]:.4f} (4-bit activations)")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(h)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    end.synchronize()
    print(f"{a.tokens} tokens through the block: {start.elapsed_time(end) / 20 * 1e3:.1f} us")
    return max(off)


if __name__ == "__main__":
    main()
