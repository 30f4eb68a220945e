#!/usr/bin/env python3
"""A mixture-of-experts block from norm to norm, for serving, and a router's
training step.

  python examples/moe_block.py [--tokens T] [--hidden H] [--experts E] [--topk k] [--width I] [--steps N]

The block takes the residual stream h and its normed rows n, chooses each
token's experts from router logits, sends the rows to them as fp8, runs the
experts on 4-bit weights (gate and up with SwiGLU, then down), combines their
outputs, and ends in the norm after the block, the gated residual sum and the
norm before the next block.  Everything but the router's own small matrix
product runs in this library's kernels, on one stream, without a synchronise.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_ep_get_04_gb300 as ep  # noqa: E402


def quantize_w4(w: torch.Tensor, group: int) -> tuple[torch.Tensor, torch.Tensor]:
    """Symmetric 4-bit codes u8 [E, rows, K/2] and bf16 scales [E, rows, K/group]
    of w [E, rows, K]."""
    E, rows, K = w.shape
    g = w.float().view(E, rows, K // group, group)
    scales = (g.abs().amax(3) / 7).clamp_min(1e-8).bfloat16()
    q = (g / scales.float()[..., None]).round().clamp(-8, 7).add(8).to(torch.uint8).view(E, rows, K)
    return (q[..., 0::2] | q[..., 1::2] << 4).contiguous(), scales.contiguous()


class MoEBlock:
    """Weights, plan and buffers of one block for batches of T tokens."""

    def __init__(self, T: int, H: int, E: int, k: int, I: int, group: int = 128, capacity: int | None = None, seed: int = 0,
                 groups: int = 1, topk_groups: int = 1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        self.T, self.k = T, k
        self.w_router = rand(H, E, scale=H ** -0.5).bfloat16()
        self.router = ep.Router(T, E, k, groups=groups, topk_groups=topk_groups, dtype=torch.bfloat16)
        self.plan = ep.Plan(T, H, E, k, capacity=capacity, fp8=True)
        self.gate_up = ep.W4Weights(*quantize_w4(rand(E, 2 * I, H, scale=H ** -0.5), group), group=group, paired=True)
        self.down = ep.W4Weights(*quantize_w4(rand(E, H, I, scale=I ** -0.5), group), group=group)
        R = self.plan.R
        self.hidden = torch.empty(R, I, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
        self.norm = ep.BlockNorm(T, H, gate="channel", scaled=True)
        self.w_post, self.w_pre = 1 + rand(H, scale=0.1), 1 + rand(H, scale=0.1)
        self.layer_gate = torch.full((H,), 0.5, device="cuda")
        self.res_scale = torch.ones(1, device="cuda")

    def forward(self, h: torch.Tensor, n: torch.Tensor, token_mask: torch.Tensor | None = None):
        """(h, n) bf16 [T, H] -> (h, n) of the next block."""
        r = self.router.route(n @ self.w_router, token_mask=token_mask)
        _, recv, scales, _ = self.plan.layout_dispatch(r.topk_idx, n, clear_flags=False)
        hidden = self.plan.expert_w4(self.gate_up, recv, scales, out=self.hidden)
        y = self.plan.expert_w4(self.down, hidden, out=self.y)
        out = self.plan.combine(y, r.topk_w)
        return self.norm.forward(h, out, self.w_post, self.w_pre, self.layer_gate, self.res_scale)


def balance_router(n: torch.Tensor, w: torch.Tensor, k: int, steps: int, rate: float):
    """Trains router weights w f32 [H, E] on rows n by the balance and z losses
    alone; returns the largest expert's load over the mean, before and after."""
    T, E = n.shape[0], w.shape[1]
    router = ep.Router(T, E, k, balance_coef=1.0, z_coef=1e-3, train=True)
    d_losses = torch.ones(2, device=n.device)
    load = []
    for step in range(steps + 1):
        logits = n.float() @ w
        r = router.route(logits)
        if step in (0, steps):
            load.append(r.counts[0].max().item() * E / (T * k))
        if step < steps:
            w -= rate * (n.float().t() @ router.backward(logits, None, d_losses))
    return load[0], load[1]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    block = MoEBlock(a.tokens, a.hidden, a.experts, a.topk, a.width)
    h = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    first = ep.BlockNorm(a.tokens, a.hidden, post=False, block=False)
    _, n = first.forward(h, w_pre=block.w_pre)
    for _ in range(3):
        block.forward(h, n)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        block.forward(h, n)
    torch.cuda.synchronize()
    print("block of %d tokens, %d experts top-%d, %d -> %d: %.1f us a step" % (
        a.tokens, a.experts, a.topk, a.hidden, a.width, (time.perf_counter() - t) / a.steps * 1e6))
    n = torch.randn(4096, 256, device="cuda") + torch.randn(256, device="cuda")
    before, after = balance_router(n, torch.randn(256, a.experts, device="cuda") / 16, a.topk, 100, 1e-2)
    print("router trained on its balance loss: largest load over the mean %.2f -> %.2f" % (before, after))


if __name__ == "__main__":
    main()
