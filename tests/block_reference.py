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


def choose(logits32, select_bias32, mask, k, groups, topk_groups):
    """topk_idx of ep_route by sorting; the rank of an expert is one fp32 sum."""
    T, E = logits32.shape
    pick = logits32 if select_bias32 is None else logits32 + select_bias32
    live = (logits32 > -np.inf).any(1)
    if mask is not None:
        live &= mask != 0
    pick = np.where(live[:, None] & ~np.isnan(pick), pick, -np.inf).astype(np.float64)
    if groups > 1:
        best = pick.reshape(T, groups, -1).max(2)
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1, kind="stable")
        pick[np.repeat(rank >= topk_groups, E // groups, axis=1)] = -np.inf
    idx = np.argsort(-pick, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(pick, idx, 1) > -np.inf, idx, -1), live


def route(logits, idx, live, bounds, full, balance_coef, z_coef, d_topk_w=None, d_losses=(0.0, 0.0)):
    """Values and sizes of ep_route and its gradient for the choice `idx`.
    bounds: the sequences' ends, S + 1 of them."""
    T, E = logits.shape
    k, S = idx.shape[1], len(bounds) - 1
    v, z = {}, {}
    lv = live[:, None]
    top = np.where(live, np.max(np.where(lv, logits, 0.0), axis=1, initial=-np.inf), 0.0)
    ex = np.where(lv, np.exp(np.where(lv, logits, 0.0) - top[:, None]), 0.0)
    total = np.where(live, ex.sum(1), 1.0)
    p = ex / total[:, None]
    lse = np.where(live, top + np.log(total), 0.0)
    got = idx >= 0
    at = np.where(got, idx, 0)
    w = np.where(got, np.take_along_axis(p, at, 1), 0.0)
    if not full:
        s = w.sum(1, keepdims=True)
        # from the chosen logits themselves: probabilities may underflow
        c = np.where(got, np.take_along_axis(logits, at, 1), -np.inf)
        c = np.exp(c - np.max(np.where(got, c, -np.inf), axis=1, keepdims=True, initial=-1e300))
        c = np.where(got, c, 0.0)
        s = c.sum(1, keepdims=True)
        w = c / np.where(s > 0, s, 1.0)
    v["topk_w"], z["topk_w"] = w, w
    v["lse"], z["lse"] = np.where(live, lse, -np.inf), np.abs(top) + np.abs(lse) + 1
    counts, sums, tokens = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    for i in range(S):
        a, b = bounds[i], bounds[i + 1]
        counts[i] = np.bincount(idx[a:b][got[a:b]], minlength=E)
        sums[i] = p[a:b].sum(0)
        tokens[i] = live[a:b].sum()
    n, filled = tokens.sum(), (tokens > 0).sum()
    v["counts"], v["seq_tokens"] = counts, np.concatenate([tokens, [n, filled]])
    v["prob_sums"], z["prob_sums"] = sums, sums
    share = np.where(tokens > 0, E / (k * np.maximum(tokens, 1.0) ** 2), 0.0) / max(filled, 1)
    balance = balance_coef * (share * (counts * sums).sum(1)).sum()
    zl = z_coef * (lse ** 2).sum() / max(n, 1)
    v["losses"] = np.array([balance, zl])
    z["losses"] = np.array([balance, z_coef * ((np.abs(top) + np.abs(lse) + 1) ** 2 * live).sum() / max(n, 1)])
    dw = np.zeros((T, k)) if d_topk_w is None else np.where(got, d_topk_w, 0.0)
    seq = np.clip(np.searchsorted(bounds[1:], np.arange(T), side="right"), 0, S - 1)
    g = d_losses[0] * balance_coef * share[seq][:, None] * counts[seq]
    extra = np.zeros((T, E))
    rows = np.broadcast_to(np.arange(T)[:, None], idx.shape)
    np.add.at(extra, (rows[got], at[got]), (dw if full else w * (dw - (w * dw).sum(1, keepdims=True)))[got])
    size = np.zeros((T, E))
    np.add.at(size, (rows[got], at[got]), (np.abs(dw) if full else w * (np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True)))[got])
    if full:
        g, extra = g + extra, 0.0
        g_size, size = np.abs(g) + size, 0.0
    else:
        g_size = np.abs(g)
    zg = 2 * d_losses[1] * z_coef / max(n, 1)
    v["d_logits"] = p * (g - (p * g).sum(1, keepdims=True)) + (zg * lse)[:, None] * p + extra
    z["d_logits"] = p * (g_size + (p * g_size).sum(1, keepdims=True)) + (abs(zg) * (np.abs(top) + np.abs(lse) + 1))[:, None] * p + size
    return v, z


def expert_w4(x, codes, scales, group, paired, spans):
    """Values and bounds' sizes of ep_expert_w4, in rows; spans: (expert, first
    row, rows).  x in float64, scales applied already; codes u8 [E, rows, K/2].
    Returns (rows written, value, size of an error of one 2^-24 per term)."""
    R, K = x.shape
    rows = codes.shape[1]
    N = rows // 2 if paired else rows
    q = np.empty((codes.shape[0], rows, K))
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    w = (q - 8) * np.repeat(scales, group, axis=2)[..., :K]
    y, size, live = np.zeros((R, N)), np.zeros((R, N)), np.zeros(R, bool)
    for e, a, n in spans:
        v, z = x[a:a + n] @ w[e].T, np.abs(x[a:a + n]) @ np.abs(w[e]).T
        if paired:
            g, u = v[:, :N], v[:, N:]
            s = 1 / (1 + np.exp(-g))
            # |d silu / d g| <= 1.1
            y[a:a + n], size[a:a + n] = g * s * u, 1.1 * z[:, :N] * np.abs(u) + np.abs(g * s) * z[:, N:] + z[:, :N] * z[:, N:] * K * EPS32
        else:
            y[a:a + n], size[a:a + n] = v, z
        live[a:a + n] = True
    return live, y, size
