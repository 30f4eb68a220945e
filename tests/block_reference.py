"""Plain 64-bit implementations of the operators at the ends of a
mixture-of-experts block, and bounds on how far a 32-bit computation of the
same formulas may be from them.

Each reference also returns a "size": the same expression with every term
taken by its magnitude.  A computation in 32 bits whose sums have n terms is
within about (n + a few) * 2^-24 * size of the value, however much the terms
cancel; a result kept in bf16 adds half a unit in its last place: bf16 keeps 8 significant bits, so at most
2^-8 of the value.
"""
import numpy as np

EPS32 = 2.0 ** -24
HALF_ULP_BF16 = 2.0 ** -8


def bound(value, size, terms, bf16):
    """Largest accepted |got - value|."""
    b = (terms + 64) * EPS32 * size
    return b + (HALF_ULP_BF16 * (np.abs(value) + b) if bf16 else 0.0)


def block_norm(h, y, w_post, w_pre, gate, res_scale, eps, d_h_out=None, d_n=None):
    """Values and sizes of ep_block_norm and its gradients, by name.  gate is
    None, [H] or [T, 1]; res_scale a number."""
    H = h.shape[1]
    one = np.ones((1, 1))
    g = one if gate is None else gate
    v, z = {}, {}
    if y is None:
        u = np.zeros_like(h)
        yn = r1 = None
    else:
        r1 = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if w_post is not None else one
        yn = y * r1
        u = yn * (w_post if w_post is not None else 1.0)
    hh = res_scale * h + g * u
    hh_size = np.abs(res_scale * h) + np.abs(g * u)
    v["h_out"], z["h_out"] = hh, hh_size
    if w_pre is not None:
        r2 = 1 / np.sqrt((hh * hh).mean(1, keepdims=True) + eps)
        hn, hn_size = hh * r2, hh_size * r2
        v["n"], z["n"] = hn * w_pre, hn_size * np.abs(w_pre)
    if d_h_out is None and d_n is None:
        return v, z
    d = np.zeros_like(h) if d_h_out is None else d_h_out
    d_size = np.abs(d)
    if w_pre is not None:
        t = d_n * w_pre
        d = d + r2 * (t - hn * (t * hn).mean(1, keepdims=True))
        d_size = d_size + r2 * (np.abs(t) + hn_size * (np.abs(t) * hn_size).mean(1, keepdims=True))
        v["d_w_pre"], z["d_w_pre"] = (d_n * hn).sum(0), (np.abs(d_n) * hn_size).sum(0)
    v["d_h"], z["d_h"] = res_scale * d, np.abs(res_scale) * d_size
    v["d_res_scale"], z["d_res_scale"] = (d * h).sum().reshape(1), (d_size * np.abs(h)).sum().reshape(1)
    if y is None:
        return v, z
    du, du_size = g * d, np.abs(g) * d_size
    if w_post is not None:
        t, t_size = du * w_post, du_size * np.abs(w_post)
        v["d_y"] = r1 * (t - yn * (t * yn).mean(1, keepdims=True))
        z["d_y"] = r1 * (t_size + np.abs(yn) * (t_size * np.abs(yn)).mean(1, keepdims=True))
        v["d_w_post"], z["d_w_post"] = (du * yn).sum(0), (du_size * np.abs(yn)).sum(0)
    else:
        v["d_y"], z["d_y"] = du, du_size
    if gate is not None:
        axis = 0 if gate.ndim == 1 else 1
        v["d_gate"], z["d_gate"] = (d * u).sum(axis), (d_size * np.abs(u)).sum(axis)
    return v, z
