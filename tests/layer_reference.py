"""Plain 64-bit implementations of dropout from counters, layer norm and the
8-bit products, and bounds on how far 32-bit computations of the same formulas
may be from them.

u = 2^-24 is half a step of fp32 next to 1.  A sum whose terms pass through a
tree of depth d is within d u of the sum of the terms' magnitudes.  A row's sums
here add up to 32 terms one after the other in a thread and 12 levels across
threads: 64 u covers them with the roundings of the terms.  What is stored in
bf16 adds half a step: 2^-8 of the value.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP_BF16 = 2.0 ** -8
LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key, rounds=10):
    """Philox4x32: counter [..., 4] and key (two numbers) below 2^32 -> [..., 4]."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [p1 >> np.uint64(32) ^ c[1] ^ np.uint64(k[0]), p1 & LOW, p0 >> np.uint64(32) ^ c[3] ^ np.uint64(k[1]), p0 & LOW]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, axis=-1)


def factors(T, H, p, rng, site, rows=None):
    """What elements [rows, H] of a [T, H] are multiplied by, in 64 bits."""
    if rng is None:
        return np.ones((1, 1))
    seed, step = (int(v) % 2 ** 64 for v in rng)
    step = (step + site) % 2 ** 64
    rows = np.arange(T) if rows is None else np.asarray(rows)
    blocks = -(-H // 8)
    at = (rows[:, None].astype(np.uint64) * np.uint64(blocks) + np.arange(blocks, dtype=np.uint64)).reshape(-1)
    counter = np.stack([at & LOW, at >> np.uint64(32), np.full_like(at, step % 2 ** 32), np.full_like(at, step >> 32)], axis=-1)
    words = philox(counter, (seed % 2 ** 32, seed >> 32))
    bits = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], axis=-1).reshape(len(rows), blocks * 8)[:, :H]
    limit = round(p * 65536)
    return np.where(bits >= limit, 65536 / (65536 - limit) if limit < 65536 else 0.0, 0.0)


def stored(value, error, bf16):
    """The bound with the rounding to what is stored: bf16, or fp32, which the error counts already.  Steps of
    subnormal numbers are absolute."""
    return error + (HALF_STEP_BF16 * (np.abs(value) + error) + 2.0 ** -134 if bf16 else 2.0 ** -149)


def dropped_sum(x, factor, residual=0.0):
    """residual + x * factor and its error: the factor, the product and the sum are rounded."""
    y = np.where(factor > 0, x * np.where(factor > 0, factor, 1.0), 0.0) if np.ndim(factor) else x * factor
    v = residual + y
    return v, 2 * U * np.abs(y) + U * (np.abs(residual) + np.abs(y))


def layer_norm(x, w, b, eps):
    """n of rows x, its error, and what the gradients need."""
    w = np.ones(x.shape[1]) if w is None else w
    b = np.zeros(x.shape[1]) if b is None else b
    mean = x.mean(1, keepdims=True)
    dev = x - mean
    var = (dev * dev).mean(1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    e_dev = 64 * U * np.abs(x).mean(1, keepdims=True) + 2 * U * (np.abs(x) + np.abs(mean))
    e_var = (2 * np.abs(dev) * e_dev + e_dev * e_dev).mean(1, keepdims=True) + 64 * U * var
    e_r = 0.5 * e_var / (var + eps) + 8 * U              # relative; the reciprocal root itself is good to 4 u
    xn = dev * r
    e_xn = e_dev * r + np.abs(xn) * (e_r + 4 * U)
    n = xn * w + b
    e_n = np.abs(w) * e_xn + 4 * U * (np.abs(xn * w) + np.abs(b))
    return n, e_n, dict(mean=mean, r=r, e_r=e_r, xn=xn, e_xn=e_xn, w=w)


def layer_norm_gradients(s, d_n, d_h_out, factor):
    """{name: (value, error)} from layer_norm's third result."""
    r, xn, e_xn, e_r = s["r"], s["xn"], s["e_xn"], s["e_r"]
    T = xn.shape[0]
    t = d_n * s["w"]
    m1, m2 = t.mean(1, keepdims=True), (t * xn).mean(1, keepdims=True)
    e_m1 = 64 * U * np.abs(t).mean(1, keepdims=True)
    e_m2 = 64 * U * np.abs(t * xn).mean(1, keepdims=True) + (np.abs(t) * e_xn).mean(1, keepdims=True)
    inner = t - m1 - xn * m2
    size = np.abs(t) + np.abs(m1) + np.abs(xn * m2)
    dh = 0.0 if d_h_out is None else d_h_out
    d = dh + r * inner
    e = r * (e_m1 + np.abs(xn) * e_m2 + np.abs(m2) * e_xn) + (e_r + 8 * U) * r * size + 8 * U * np.abs(dh)
    out = {"d_h": (d, e), "d_y": (d * factor, e * factor + 2 * U * np.abs(d * factor))}
    out["d_w"] = ((d_n * xn).sum(0), (np.abs(d_n) * e_xn).sum(0) + (T + 64) * U * np.abs(d_n * xn).sum(0))
    out["d_b"] = (d_n.sum(0), (T + 64) * U * np.abs(d_n).sum(0))
    return out


def expert_i8(x, x_scales, codes, scales, paired, spans):
    """(rows written, value, size of an error of u a term), as block_reference.expert_w4's.  x i64 [R, K], codes
    [E, rows, K]; products and sums of codes are whole numbers below 2^53."""
    R, K = x.shape
    rows = codes.shape[1]
    N = rows // 2 if paired else rows
    y, size, live = np.zeros((R, N)), np.zeros((R, N)), np.zeros(R, bool)
    for e, a, n in spans:
        q, w = x[a:a + n].astype(np.float64), codes[e].astype(np.float64)
        f = x_scales[a:a + n, None] * scales[e]
        v, z = (q @ w.T) * f, (np.abs(q) @ np.abs(w).T) * f
        if paired:
            g, up = v[:, :N], v[:, N:]
            s = 1 / (1 + np.exp(-g))
            y[a:a + n], size[a:a + n] = g * s * up, 1.1 * z[:, :N] * np.abs(up) + np.abs(g * s) * z[:, N:] + z[:, :N] * z[:, N:] * K * U
        else:
            y[a:a + n], size[a:a + n] = v, z
        live[a:a + n] = True
    return live, y, size


def quant_i8(x):
    """(codes, scales) of rows x from bf16: 127 x and the comparisons with halves are exact in 64 bits."""
    amax = np.abs(x).max(1, initial=0.0)
    fine = np.isfinite(amax)
    top = np.where(fine & (amax > 0), amax, 1.0)[:, None]
    q = np.where(fine[:, None] & (amax > 0)[:, None], np.rint(127 * np.where(np.isfinite(x), x, 0.0) / top), 0.0)
    return q.astype(np.int64), np.where(fine, amax / 127, np.nan)
