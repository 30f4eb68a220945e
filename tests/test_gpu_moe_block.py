"""The block operators together, as examples/moe_block.py runs them: a serving
step against the same block in 64 bits, and a router trained on its losses.

The kernels round to bf16 four times on the way (experts' hidden rows, their
outputs, the combined row, the stream) and to e4m3 once; the 64-bit block takes
the dispatched fp8 rows as they are, so what remains is at most 2^-8 of a value
for each of the four, at random signs: under 1 % of the result's norm.
"""
import os
import sys

import numpy as np
import pytest
import torch

import combine_ep_get_04_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def reference(b, h, n, codes, recv, scales, layout, topk_idx, topk_w):
    """The block in float64 from the dispatched rows on."""
    def weights(w):
        c, s, group = codes[w]
        q = torch.stack([c & 15, c >> 4], dim=-1).reshape(*c.shape[:2], -1).double() - 8
        return q * s.double().repeat_interleave(group, 2)

    x = recv.float().double() * scales.double().repeat_interleave(128, 1)
    gu, down = weights("gate_up"), weights("down")
    out = torch.zeros(h.shape, dtype=torch.float64, device="cuda")
    slot = layout.slot_of.cpu()
    for t in range(h.shape[0]):
        for j in range(topk_idx.shape[1]):
            e, r = int(topk_idx[t, j]), int(slot[t, j])
            if e < 0:
                assert r == -1
                continue
            v = gu[e] @ x[r]
            g, u = v[: v.numel() // 2], v[v.numel() // 2:]
            out[t] += topk_w[t, j].double() * (down[e] @ (g * torch.sigmoid(g) * u))
    eps = 1e-6
    u = out / (out.pow(2).mean(1, keepdim=True) + eps).sqrt() * b.w_post.double()
    u[out.abs().sum(1) == 0] = 0
    hh = b.res_scale.double() * h.double() + b.layer_gate.double() * u
    return hh, hh / (hh.pow(2).mean(1, keepdim=True) + eps).sqrt() * b.w_pre.double()


@pytest.mark.parametrize("capacity,groups,topk_groups,masked", [(None, 1, 1, False), (24, 4, 2, True)])
def test_serving_step(monkeypatch, capacity, groups, topk_groups, masked):
    T, H, E, k, I = 24, 512, 16, 4, 256
    codes = {}
    real = moe_block.quantize_w4

    def keep(w, group):
        c, s = real(w, group)
        codes["gate_up" if len(codes) == 0 else "down"] = (c, s, group)
        return c, s

    monkeypatch.setattr(moe_block, "quantize_w4", keep)
    b = moe_block.MoEBlock(T, H, E, k, I, capacity=capacity, groups=groups, topk_groups=topk_groups)
    g = torch.Generator(device="cuda").manual_seed(1)
    h, n = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    mask = (torch.arange(T, device="cuda") % 5 != 0) if masked else None
    h2, n2 = b.forward(h, n, mask)
    torch.cuda.synchronize()
    assert int(b.plan.layout_out.err_flags) == 0
    r = b.router.out
    if masked:
        assert (r.topk_idx[~mask] == -1).all()
    hh, nn = reference(b, h, n, codes, b.plan.recv, b.plan.recv_scales, b.plan.layout_out, r.topk_idx.cpu(), r.topk_w)
    for got, want in ((h2, hh), (n2, nn)):
        off = torch.linalg.norm(got.double() - want) / torch.linalg.norm(want)
        assert off < 0.01, off


def test_two_steps_give_the_same(capsys):
    b = moe_block.MoEBlock(16, 256, 8, 2, 128)
    h, n = torch.randn(16, 256, device="cuda").bfloat16(), torch.randn(16, 256, device="cuda").bfloat16()
    first = [t.clone() for t in b.forward(h, n)]
    assert all(torch.equal(x, y) for x, y in zip(first, b.forward(h, n)))


def test_a_step_replays_from_a_graph():
    """Nothing on the way synchronises or depends on the host: a captured step
    gives what it gives call by call, also on new inputs."""
    b = moe_block.MoEBlock(16, 256, 8, 2, 128)
    h, n = torch.randn(16, 256, device="cuda").bfloat16(), torch.randn(16, 256, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.forward(h, n)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            h2, n2 = b.forward(h, n)
    h.copy_(torch.randn(16, 256, device="cuda").bfloat16())
    n.copy_(torch.randn(16, 256, device="cuda").bfloat16())
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = [h2.clone(), n2.clone()]
    assert all(torch.equal(x, y) for x, y in zip(got, b.forward(h, n)))


def test_the_balance_loss_balances():
    g = torch.Generator(device="cuda").manual_seed(3)
    n = torch.randn(2048, 64, generator=g, device="cuda") + torch.randn(64, generator=g, device="cuda")
    before, after = moe_block.balance_router(n, torch.randn(64, 32, generator=g, device="cuda") / 8, 4, 100, 1e-2)
    assert before > 2.0 and after < 1.5, (before, after)


def test_plan_refusals():
    b = moe_block.MoEBlock(16, 256, 8, 2, 128)
    other = moe_block.MoEBlock(16, 256, 4, 2, 128)
    with pytest.raises(ValueError):
        b.plan.expert_w4(other.gate_up)
    with pytest.raises(ValueError):
        b.plan.expert_w4(b.down, torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda"))
