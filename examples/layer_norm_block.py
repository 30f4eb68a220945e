#!/usr/bin/env python3
"""A mixture-of-experts block of a layer-normed network: a serving step with
8-bit experts, and a training step of the block's ends with dropout.

  python examples/layer_norm_block.py [--tokens T] [--hidden H] [--experts E] [--topk k] [--width I] [--steps N]

The serving step sends the normed rows to their experts, makes 8-bit integers of
them with a scale for each, multiplies them with 8-bit weights (gate and up with
SwiGLU, then down, its rows quantised in between), combines the outputs, and ends
in the residual sum and the layer norm before the next block.  The training step
runs a chain of such ends, forwards and backwards, and is captured into a CUDA
graph that counts the dropout's step up by itself.  The router's and the blocks'
own small matrix products are torch's; the rest runs in this library's kernels,
on one stream, without a synchronise.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_ep_get_04_gb300 as ep  # noqa: E402


def quantize_rows(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """8-bit codes i8 and scales f32 [E, rows] of w [E, rows, K]."""
    scales = w.float().abs().amax(2) / 127
    return (w.float() / scales.clamp_min(1e-30)[..., None]).round().clamp(-127, 127).to(torch.int8), scales


class I8Block:
    """Weights, plan and buffers of one block for batches of T tokens."""

    def __init__(self, T: int, H: int, E: int, k: int, I: int, capacity: int | None = None, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        self.w_router = rand(H, E, scale=H ** -0.5).bfloat16()
        self.router = ep.Router(T, E, k, dtype=torch.bfloat16)
        self.plan = ep.Plan(T, H, E, k, capacity=capacity)
        self.gate_up = ep.I8Weights(*quantize_rows(rand(E, 2 * I, H, scale=H ** -0.5)), paired=True)
        self.down = ep.I8Weights(*quantize_rows(rand(E, H, I, scale=I ** -0.5)))
        R, dev = self.plan.R, dict(device="cuda")
        self.rows = torch.zeros(R, H, dtype=torch.int8, **dev), torch.zeros(R, **dev)
        self.hidden, self.y = torch.zeros(R, I, dtype=torch.bfloat16, **dev), torch.zeros(R, H, dtype=torch.bfloat16, **dev)
        self.hidden_rows = torch.zeros(R, I, dtype=torch.int8, **dev), torch.zeros(R, **dev)
        self.norm = ep.LayerNorm(T, H)
        self.w, self.b = 1 + rand(H, scale=0.1), rand(H, scale=0.1)

    def forward(self, h: torch.Tensor, n: torch.Tensor, token_mask: torch.Tensor | None = None):
        """(h, n) bf16 [T, H] -> (h, n) of the next block."""
        r = self.router.route(n @ self.w_router, token_mask=token_mask)
        self.plan.layout_dispatch(r.topk_idx, n, clear_flags=False)
        x = self.plan.quant_i8(out=self.rows[0], scales=self.rows[1])
        hidden = self.plan.expert_i8(self.gate_up, *x, out=self.hidden)
        x = self.plan.quant_i8(hidden, out=self.hidden_rows[0], scales=self.hidden_rows[1])
        y = self.plan.expert_i8(self.down, *x, out=self.y)
        return self.norm.forward(h, self.plan.combine(y, r.topk_w), self.w, self.b)


class Chain:
    """A network of `layers` dense blocks y = n W between layer norms, with
    dropout of each y and of the first rows; its gradients by the kernels."""

    def __init__(self, T: int, H: int, layers: int, p: float, dtype: torch.dtype = torch.float32, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")     # noqa: E731
        self.p, self.layers = p, layers
        self.rng = torch.tensor([seed + 1, 0], device="cuda")
        self.first = ep.LayerNorm(T, H, dtype, block=False, train=True)
        self.ends = [ep.LayerNorm(T, H, dtype, p=p, site=i + 1, train=True) for i in range(layers)]
        self.w = [1 + 0.1 * rand(H) for _ in range(layers + 1)]
        self.b = [0.1 * rand(H) for _ in range(layers + 1)]
        self.mats = [(rand(H, H) / H ** 0.5).bfloat16() for _ in range(layers)]

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """The last normed rows of x (stream type [T, H])."""
        self.h0 = ep.dropout(x, self.p, self.rng, site=0)
        h, n = self.first.forward(self.h0, w=self.w[0], b=self.b[0])
        self.n, self.h = [n], [h]
        for m, end, w, b in zip(self.mats, self.ends, self.w[1:], self.b[1:]):
            h, n = end.forward(h, n @ m, w, b, self.rng)
            self.n.append(n)
            self.h.append(h)
        return n

    def backward(self, d_n: torch.Tensor):
        """Gradients of the input, the matrices and the norms' weights, from
        that of forward()'s result."""
        d_h, d_mats, d_w, d_b = None, [None] * self.layers, [None] * (self.layers + 1), [None] * (self.layers + 1)
        for i in reversed(range(self.layers)):
            d = self.ends[i].backward(self.h[i + 1], self.w[i + 1], d_n, d_h, self.rng)
            d_w[i + 1], d_b[i + 1], d_h = d.d_w, d.d_b, d.d_h
            d_mats[i] = self.n[i].t() @ d.d_y
            d_n = d.d_y @ self.mats[i].t()
        d = self.first.backward(self.h0, self.w[0], d_n, d_h)
        d_w[0], d_b[0] = d.d_w, d.d_b
        return ep.dropout(d.d_h, self.p, self.rng, site=0), d_mats, d_w, d_b


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    block = I8Block(a.tokens, a.hidden, a.experts, a.topk, a.width)
    h = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    _, n = ep.LayerNorm(a.tokens, a.hidden, block=False).forward(h, w=block.w, b=block.b)
    for _ in range(3):
        block.forward(h, n)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        block.forward(h, n)
    torch.cuda.synchronize()
    print("block of %d tokens, %d experts top-%d, %d -> %d, 8-bit: %.1f us a step" % (
        a.tokens, a.experts, a.topk, a.hidden, a.width, (time.perf_counter() - t) / a.steps * 1e6))

    chain, x = Chain(2048, 1024, 4, 0.1), torch.randn(2048, 1024, device="cuda")
    d_n = torch.randn(2048, 1024, device="cuda").bfloat16()

    def step():
        chain.forward(x)
        chain.backward(d_n)
        chain.rng[1] += chain.layers + 1            # the next step's dropouts are others

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    print("training step of %d ends of 2048 x 1024, replayed: %.1f us" % (chain.layers + 1, (time.perf_counter() - t) / a.steps * 1e6))


if __name__ == "__main__":
    main()
