"""Layer norm, dropout, quantisation and 8-bit products together, as
examples/layer_norm_block.py runs them: a serving step against the same block in
64 bits, and a chain's gradients against autograd's in 64 bits.

Between 64-bit steps the reference rounds where the block stores bf16 or codes,
so that what remains of a step is its own rounding to bf16, at most 2^-8 of a
value, at random signs.
"""
import os
import sys

import numpy as np
import pytest
import torch

import combine_ep_get_04_gb300 as ep
import layer_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import layer_norm_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def close(got, want, rel):
    off = torch.linalg.norm(got.double() - want.double()) / torch.linalg.norm(want.double())
    assert off < rel, float(off)


@pytest.mark.parametrize("T,capacity,masked", [(24, None, False), (24, 24, True), (700, None, False)])
def test_serving_step(monkeypatch, T, capacity, masked):
    H, E, k, I = 512, 16, 4, 264 - 8
    kept = []
    real = layer_norm_block.quantize_rows
    monkeypatch.setattr(layer_norm_block, "quantize_rows", lambda w: kept.append(real(w)) or kept[-1])
    b = layer_norm_block.I8Block(T, H, E, k, I, capacity=capacity)
    (gu, gu_s), (down, down_s) = ((c.double(), s.double()) for c, s in kept)
    g = torch.Generator(device="cuda").manual_seed(1)
    h, n = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8) if masked else None
    h2, n2 = b.forward(h, n, mask)
    torch.cuda.synchronize()
    L = b.plan.layout_out
    assert int(L.err_flags) == 0
    w = b.router.out.topk_w.double()
    owner = torch.full((b.plan.R,), -1, dtype=torch.int64)
    for e in range(E):
        a = e * capacity if capacity else int(L.offsets[e])
        owner[a:a + int(L.counts[e])] = e
    rows = (owner >= 0).nonzero()[:, 0].cuda()
    of = owner[owner >= 0].cuda()
    # the codes of the dispatched rows are exactly the 64-bit ones; the hidden rows' are taken as they are
    q, s = ref.quant_i8(b.plan.recv[rows].double().cpu().numpy())
    assert np.array_equal(b.rows[0][rows].cpu().numpy(), q)
    x = torch.from_numpy(q).cuda().double() * torch.from_numpy(s).cuda()[:, None]
    hidden = torch.empty(len(rows), I, dtype=torch.float64, device="cuda")
    y = torch.empty(len(rows), H, dtype=torch.float64, device="cuda")
    hq = b.hidden_rows[0][rows].double() * b.hidden_rows[1][rows].double()[:, None]
    for e in range(E):
        m = of == e
        v = x[m] @ (gu[e] * gu_s[e][:, None]).t()
        hidden[m] = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
        y[m] = hq[m] @ (down[e] * down_s[e][:, None]).t()
    close(b.hidden[rows], hidden, 2.0 ** -8)
    close(b.y[rows], y, 2.0 ** -8)
    there = b.router.out.topk_idx >= 0
    out = (b.y.double()[L.slot_of.clamp_min(0).long()] * torch.where(there, w, 0.0)[..., None]).sum(1)
    hh = h.double() + out.bfloat16().double()
    close(h2, hh, 2.0 ** -7)               # the combined row and the sum: two roundings
    want = ref.layer_norm(h2.double().cpu().numpy(), b.w.double().cpu().numpy(), b.b.double().cpu().numpy(), 1e-5)[0]
    close(n2, torch.from_numpy(want).cuda(), 2.0 ** -8)
    if masked:
        assert torch.equal(h2[~mask], h[~mask])
    # captured, then replayed on another batch
    graph, want = torch.cuda.CUDAGraph(), [t.clone() for t in (h2, n2)]
    with torch.cuda.graph(graph):
        b.forward(h, n, mask)
    first = h.clone(), n.clone()
    h.copy_(torch.randn(T, H, generator=g, device="cuda"))
    n.copy_(torch.randn(T, H, generator=g, device="cuda"))
    graph.replay()
    again = [t.clone() for t in b.forward(h, n, mask)]
    graph.replay()
    assert all(torch.equal(a, c) for a, c in zip(again, (b.norm.h_out, b.norm.n)))
    h.copy_(first[0])
    n.copy_(first[1])
    graph.replay()
    assert all(torch.equal(a, c) for a, c in zip(want, (b.norm.h_out, b.norm.n)))


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_gradients_of_a_chain(p):
    """bf16 rows enter every block and its gradient, so each of the chain's three blocks adds roundings of 2^-8 at random
    signs: of the order of 1 % of a gradient's norm in all, and 3 % bounds it."""
    T, H, layers = 96, 256, 3
    chain = layer_norm_block.Chain(T, H, layers, p)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d_n = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda").bfloat16()
    n = chain.forward(x)
    got = chain.backward(d_n)
    leaves = [t.double().requires_grad_() for t in [x, *chain.mats, *chain.w, *chain.b]]
    lx, mats, w, b = leaves[0], leaves[1:1 + layers], leaves[1 + layers:2 + 2 * layers], leaves[2 + 2 * layers:]
    rng = chain.rng.tolist()
    f = [torch.from_numpy(np.broadcast_to(ref.factors(T, H, p, rng, i), (T, H)).copy()).cuda() for i in range(layers + 1)]

    def norm(h, w, b):
        c = h - h.mean(1, keepdim=True)
        return c / (c.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * w + b

    h = lx * f[0]
    want = norm(h, w[0], b[0])
    for i in range(layers):
        h = h + (want @ mats[i]) * f[i + 1]
        want = norm(h, w[i + 1], b[i + 1])
    (want * d_n.double()).sum().backward()
    close(n, want.detach(), 0.03)
    for a, leaf in zip([got[0], *got[1], *got[2], *got[3]], leaves):
        close(a, leaf.grad, 0.03)
