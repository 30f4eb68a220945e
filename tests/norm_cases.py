"""Inputs and bounds for checks of ep_block_norm_backward over many rows a CTA.

The bounds follow the kernels' own chains of additions, so that a lost or
doubled share of a sum lies outside them: a row's sums go over 4 pairs of
channels, a pair, 32 lanes, 16 warps and 4 CTAs (some 20 roundings); sums over rows
go over the rows of a CTA, then over every sixteenth CTA and 16 warps, and
d_res_scale over 4 values a row of each half of a pair, 32 lanes, the warps and
every 32nd CTA.
"""
import numpy as np
import torch

import block_reference as ref

EPS = 1e-6


def clusters(T, H, sms):
    """Groups of CTAs that share the rows, one row a group at a time."""
    cluster = 1 if H <= 4096 else 2 if H <= 8192 else 4
    warps = -(-(-(-H // 8 // cluster)) // 32)
    per_sm = max(1, min(6, 16 // warps, 20 // (warps + 2)))
    return min(T, sms * per_sm // cluster), cluster


def make(T, H, dtype, gate, post, pre, scaled, d_h_out=True, seed=0):
    """CPU tensors.  The gradient of the stream goes with the stream itself, as
    a decaying one would: d_res_scale is a large part of its terms' sum."""
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, dt=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt)

    h = rand(T, H, dt=dtype, scale=2.0)
    inputs = dict(h=h, y=rand(T, H, dt=torch.bfloat16, scale=0.5), w_post=1 + rand(H, scale=0.1) if post else None,
                  w_pre=1 + rand(H, scale=0.1) if pre else None,
                  gate=None if gate is None else 0.5 + rand(H if gate == "channel" else T, scale=0.2),
                  res_scale=torch.full((1,), 0.9) if scaled else None)
    return inputs, dict(d_h_out=(rand(T, H) + 0.5 * h.float()).to(dtype) if d_h_out else None,
                        d_n=(rand(T, H) + (0.0 if d_h_out else 0.5) * h.float()).bfloat16() if pre else None)


def reference(inputs, grads):
    f64 = lambda t: None if t is None else t.double().cpu().numpy()    # noqa: E731
    r = {k: f64(v) for k, v in inputs.items()}
    if r["gate"] is not None and len(r["gate"]) == len(r["h"]):
        r["gate"] = r["gate"][:, None]
    r["res_scale"] = 1.0 if r["res_scale"] is None else r["res_scale"][0]
    return ref.block_norm(**r, eps=EPS, **{k: f64(x) for k, x in grads.items()})


def bound(name, value, size, T, H, gate, sms, bf16):
    groups, cluster = clusters(T, H, sms)
    rows = -(-T // groups)
    terms = 64                                           # of a row's own values (and 64 more in ref.bound)
    if name in ("d_w_post", "d_w_pre") or (name == "d_gate" and gate == "channel"):
        terms += rows + groups // 16 + 17
    elif name == "d_res_scale":
        terms += 4 * rows + 1 + 5 + 16 + groups * cluster // 32 + 6
    return ref.bound(value, size, terms, bf16)
