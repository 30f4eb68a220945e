"""Cases for the ends of a layer-normed block in training, and for expert products in 8-bit integers.

  ln     residual sum of a block's output after dropout and the layer norm before the next block, with gradients
  drop   dropout from counters, alone or with the residual sum, and its gradient
  i8     the experts' products over the receive buffer with 8-bit weights and rows, scaled by channel and by token, alone
         or as the gate/up pair of a SwiGLU
  quant  rows of the receive buffer to 8-bit integers with a scale for each

Sizes are those of this library's workloads (hidden 1024, 4096 and 7168; 16, 128 and 256 experts; batches of 128,
4096 and 16384 tokens) with an expert width of 2048, and generic odd ones.

The random numbers of dropout are the generator Philox4x32 with ten rounds (J. K. Salmon, M. A. Moraes, R. O. Dror and
D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC11): 16 bits for each element, one counter for eight
neighbours of a row.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
SITE = 5  # which dropout of the network it is


# ------------------------------------------------------------------ cases

def listed():
    return [
        # serving: block end of one decode batch, nothing dropped
        dict(name="ln_serve_128x7168", op="ln", T=128, H=7168, dtype="bf16", p=0.0, bias=True, train=False),
        # training step over the prefill batch
        dict(name="ln_train_4096x7168", op="ln", T=4096, H=7168, dtype="bf16", p=0.1, bias=True, train=True),
        # training step over the largest batch, residual stream in 32 bits
        dict(name="ln_train_16384x4096", op="ln", T=16384, H=4096, dtype="f32", p=0.1, bias=True, train=True),
        # odd sizes, a norm without a bias, nothing dropped
        dict(name="ln_train_odd_333x1000", op="ln", T=333, H=1000, dtype="bf16", p=0.0, bias=False, train=True),
        # dropout of the largest batch's hidden rows and of their gradient
        dict(name="drop_train_16384x4096", op="drop", T=16384, H=4096, dtype="bf16", p=0.1, residual=False),
        # odd sizes, with the residual sum
        dict(name="drop_train_odd_777x1001", op="drop", T=777, H=1001, dtype="f32", p=0.25, residual=True),
        # one token through one matrix: the smallest product
        dict(name="i8_one_row_7168x4096", op="i8", T=1, E=1, k=1, K=7168, N=4096, paired=False, cap=0),
        # gate and up products of the decode batch in the capacity buffer
        dict(name="i8_decode_gate_up", op="i8", T=128, E=256, k=8, K=7168, N=2048, paired=True, cap=128),
        # down product of the same batch, packed rows
        dict(name="i8_decode_down", op="i8", T=128, E=256, k=8, K=2048, N=7168, paired=False, cap=0),
        # gate and up products of the prefill batch, about 128 rows an expert
        dict(name="i8_prefill_gate_up", op="i8", T=4096, E=256, k=8, K=7168, N=2048, paired=True, cap=0),
        # the decode batch's rows in its capacity buffer
        dict(name="quant_decode_7168", op="quant", T=128, E=256, k=8, K=7168, cap=128),
        # the prefill batch's rows between the products
        dict(name="quant_prefill_2048", op="quant", T=4096, E=256, k=8, K=2048, cap=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "drop", "i8", "quant"])
    if op in ("ln", "drop"):
        H = _log(rng, 64, 8192)
        if op == "ln":
            H = max(8, H - H % 8)
        T = min(_log(rng, 1, 16384), 16384 * 4096 // H)
        dtype = rng.choice(["bf16", "f32"])
        if op == "drop":
            return dict(op="drop", T=T, H=H, dtype=dtype, p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=rng.random() < 0.5)
        return dict(op="ln", T=T, H=H, dtype=dtype, p=rng.choice([0.0, 0.05, 0.1, 0.25]), bias=rng.random() < 0.7,
                    train=rng.random() < 0.7)
    E = rng.choice([1, _log(rng, 2, 256)])
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 4096)
    K = _log(rng, 128, 7168)
    K = max(16, K - K % 16)
    cap = rng.choice([0, min(T, 256)])
    if op == "quant":
        return dict(op="quant", T=T, E=E, k=k, K=K, cap=cap)
    paired = rng.random() < 0.5
    N = min(_log(rng, 64, 7168), 256 * 2048 * 7168 // (E * K))
    N = max(8, N - N % 8)
    return dict(op="i8", T=T, E=E, k=k, K=K, N=N, paired=paired, cap=cap)


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"ln": _prepare_ln, "drop": _prepare_drop, "i8": _prepare_i8, "quant": _prepare_quant}[case["op"]](case, g)


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _rng(g):
    # seed and step, as a training loop keeps them on the device
    return torch.randint(-2**62, 2**62, (2,), generator=g, device="cuda")


def _stream(g, T, H, dtype):
    # a residual stream: rows off zero, some channels larger than the rest
    h = torch.randn(T, H, generator=g, device="cuda") * 1.5 + _randn(g, T, 1, scale=0.3)
    return h.mul_(1 + 3 * (torch.rand(H, generator=g, device="cuda") < 0.01)).to(dtype)


def _prepare_ln(c, g):
    T, H = c["T"], c["H"]
    dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = dict(c, h=_stream(g, T, H, dtype), y=_randn(g, T, H, scale=0.5, dtype=torch.bfloat16), w=1 + _randn(g, H, scale=0.1),
             b=_randn(g, H, scale=0.1) if c["bias"] else None, rng=_rng(g) if c["p"] else None)
    if c["train"]:
        s["d_h_out"] = _randn(g, T, H, dtype=dtype)
        s["d_n"] = _randn(g, T, H, dtype=torch.bfloat16)
    if own:
        import combine_ep_get_04_gb300 as ep
        s["norm"] = ep.LayerNorm(T, H, dtype=dtype, p=c["p"], site=SITE, bias=c["bias"], eps=EPS, train=c["train"])
    return s


def _prepare_drop(c, g):
    T, H = c["T"], c["H"]
    dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = dict(c, x=_randn(g, T, H, dtype=dtype), dy=_randn(g, T, H, dtype=dtype), res=_randn(g, T, H, dtype=dtype) if c["residual"] else None,
             rng=_rng(g))
    s["out"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    return s


def _layout(c, g):
    """Counts and offsets of the experts' rows, as the layout gives them; rows past a capacity are dropped."""
    T, E, k, cap = c["T"], c["E"], c["k"], c["cap"]
    # some experts are liked more than others
    liking = _randn(g, 1, E, scale=0.3) + torch.rand(T, E, generator=g, device="cuda").clamp_min(1e-9).log().neg().log().neg()
    counts = torch.bincount(liking.topk(k, 1).indices.reshape(-1), minlength=E).to(torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)
    held = counts.clamp_max(cap) if cap else counts
    return dict(counts=counts, offsets=offsets, R=E * cap if cap else T * k, most=int(held.max()))


def _prepare_i8(c, g):
    E, K, N = c["E"], c["K"], c["N"]
    rows = 2 * N if c["paired"] else N
    s = dict(c, **_layout(c, g))
    codes = torch.randint(-127, 128, (E, rows, K), generator=g, device="cuda", dtype=torch.int8)
    scales = (torch.rand(E, rows, generator=g, device="cuda") + 0.5) * (0.014 / math.sqrt(K))
    # rows as quantisation leaves them: bell-shaped, the largest at 127
    s["x"] = (torch.randn(s["R"], K, generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8)
    s["x_scales"] = (torch.rand(s["R"], generator=g, device="cuda") + 0.5) * 0.03
    s["out"] = torch.zeros(s["R"], N, dtype=torch.bfloat16, device="cuda")
    if own:
        import combine_ep_get_04_gb300 as ep
        s["weights"] = ep.I8Weights(codes, scales, paired=c["paired"])
    else:
        s["codes"], s["scales"] = codes, scales
    return s


def _prepare_quant(c, g):
    s = dict(c, **_layout(c, g))
    R, K = s["R"], c["K"]
    s["x"] = (torch.randn(R, K, generator=g, device="cuda") * torch.exp(_randn(g, R, 1))).to(torch.bfloat16)
    s["q"], s["scales"] = torch.zeros(R, K, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")
    return s


# ------------------------------------------------------------------- runs

def run(s):
    return {"ln": _run_ln, "drop": _run_drop, "i8": _run_i8, "quant": _run_quant}[s["op"]](s)


def _kept(rng, T, H, p):
    """Which elements of [T, H] stay, and what they are multiplied by."""
    mask32, blocks = 0xFFFFFFFF, -(-H // 8)
    at = torch.arange(T * blocks, device=rng.device)
    step, key0, key1 = rng[1] + SITE, rng[0] & mask32, rng[0] >> 32 & mask32
    c0, c1 = at & mask32, at >> 32
    c2, c3 = (step & mask32).expand_as(at), (step >> 32 & mask32).expand_as(at)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & mask32) ^ c1 ^ key0, b & mask32, (a >> 32 & mask32) ^ c3 ^ key1, a & mask32
        key0, key1 = key0 + 0x9E3779B9 & mask32, key1 + 0xBB67AE85 & mask32
    words = torch.stack([c0, c1, c2, c3], dim=1)
    u = torch.stack([words & 0xFFFF, words >> 16], dim=2).view(T, blocks * 8)[:, :H]
    limit = round(p * 65536)
    return u >= limit, 65536 / (65536 - limit)


def _run_ln(s):
    if own:
        m = s["norm"]
        h_out, n = m.forward(s["h"], s["y"], s["w"], s["b"], s["rng"])
        out = {"h_out": h_out, "n": n}
        if s["train"]:
            d = m.backward(h_out, s["w"], s["d_n"], s["d_h_out"], s["rng"])
            out.update(d_h=d.d_h, d_y=d.d_y, d_w=d.d_w)
            if s["b"] is not None:
                out["d_b"] = d.d_b
        return out
    h, y = s["h"].float(), s["y"].float()
    keep = scale = None
    if s["p"]:
        keep, scale = _kept(s["rng"], s["T"], s["H"], s["p"])
        y = torch.where(keep, y * scale, 0.0)
    h_out = (h + y).to(s["h"].dtype)  # the norm is of the stream as it is stored
    x = h_out.float()
    x = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    xn = x * rstd
    n = xn * s["w"]
    if s["b"] is not None:
        n = n + s["b"]
    out = {"h_out": h_out, "n": n.to(torch.bfloat16)}
    if not s["train"]:
        return out
    dn = s["d_n"].float()
    t = dn * s["w"]
    d = s["d_h_out"].float() + rstd * (t - t.mean(1, keepdim=True) - xn * (t * xn).mean(1, keepdim=True))
    out["d_h"] = d.to(s["h"].dtype)
    out["d_y"] = (d if keep is None else torch.where(keep, d * scale, 0.0)).to(torch.bfloat16)
    out["d_w"] = (dn * xn).sum(0)
    if s["b"] is not None:
        out["d_b"] = dn.sum(0)
    return out


def _run_drop(s):
    if own:
        import combine_ep_get_04_gb300 as ep
        return {"y": ep.dropout(s["x"], s["p"], s["rng"], site=SITE, residual=s["res"], out=s["out"]),
                "dx": ep.dropout(s["dy"], s["p"], s["rng"], site=SITE, out=s["dx"])}
    keep, scale = _kept(s["rng"], s["T"], s["H"], s["p"])
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(s["x"].dtype), "dx": torch.where(keep, s["dy"].float() * scale, 0.0).to(s["x"].dtype)}


def _rows(s):
    """Rows of the receive buffer that hold a copy, [E, most]; R stands for none."""
    at = torch.arange(s["most"], device="cuda")
    start = (torch.arange(s["E"], device="cuda") * s["cap"] if s["cap"] else s["offsets"][:-1].long())[:, None] + at
    return torch.where(at < s["counts"][:, None], start, s["R"])


def _run_i8(s):
    if own:
        import combine_ep_get_04_gb300 as ep
        return ep.expert_i8(s["x"], s["x_scales"], s["weights"], s["counts"], s["offsets"], capacity=s["cap"] or None,
                            max_rows=s["T"] * s["k"], out=s["out"])
    N, R = s["N"], s["R"]
    rows = _rows(s)
    at = rows.clamp_max(R - 1)
    y = torch.bmm(s["x"][at].float(), s["codes"].float().transpose(1, 2))
    y = y * s["scales"][:, None, :] * s["x_scales"][at][..., None]
    if s["paired"]:
        gate, up = y[..., :N], y[..., N:]
        y = gate / (1 + torch.exp(-gate)) * up
    out = torch.zeros(R + 1, N, dtype=torch.bfloat16, device="cuda")
    return out.index_copy_(0, rows.reshape(-1), y.reshape(-1, N).to(torch.bfloat16))[:R]


def _run_quant(s):
    if own:
        import combine_ep_get_04_gb300 as ep
        q, scales = ep.quant_i8(s["x"], s["counts"], s["offsets"], capacity=s["cap"] or None, out=s["q"], scales=s["scales"])
        return {"q": q * scales[:, None], "scales": scales}
    R = s["R"]
    held = torch.zeros(R + 1, dtype=torch.bool, device="cuda").index_fill_(0, _rows(s).reshape(-1), True)[:R]
    x = s["x"].float()
    top = x.abs().amax(1)
    q = torch.round(x * 127 / torch.where(top > 0, top, 1.0)[:, None])
    scales = torch.where(held, top / 127, 0.0)
    return {"q": q * scales[:, None], "scales": scales}


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] in ("ln", "drop"):
        n, size = c["T"] * c["H"], 4 if c["dtype"] == "f32" else 2
        if c["op"] == "drop":
            return {"bytes": n * size * (5 if c["residual"] else 4), "flops": n * 20}
        b, f = n * (2 * size + 4), n * 12
        if c["train"]:  # the stream again, its gradients in and out, d_n and d_y
            b += n * (3 * size + 2 + (2 if c["p"] or c["dtype"] == "f32" else 0))
            f += n * 24
        return {"bytes": b + 16 * c["T"], "flops": f}
    T, E, k, K = c["T"], c["E"], c["k"], c["K"]
    copies = min(T * k, E * c["cap"]) if c["cap"] else T * k
    if c["op"] == "quant":
        return {"bytes": copies * (3 * K + 4), "flops": copies * K * 3}
    rows = 2 * c["N"] if c["paired"] else c["N"]
    used = E * (1 - (1 - k / E) ** T)  # experts that some token chooses
    return {"bytes": used * rows * (K + 4) + copies * (K + 4 + 2 * c["N"]), "flops": 2.0 * copies * rows * K}


# -------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "drop": _exact_drop, "i8": _exact_i8, "quant": _exact_quant}[case["op"]](s)


def _factors(s):
    """What each element is multiplied by, from the generator in 64-bit unsigned words."""
    T, H = s["T"], s["H"]
    if not s["p"]:
        return torch.ones((), dtype=torch.float64, device="cuda")
    seed, step = (int(v) % 2**64 for v in s["rng"].tolist())
    step = (step + SITE) % 2**64
    low, half = np.uint64(2**32 - 1), np.uint64(32)
    at = np.arange(T * ((H + 7) // 8), dtype=np.uint64)
    ctr = [at & low, at >> half, np.full_like(at, step % 2**32), np.full_like(at, step >> 32)]
    for i in range(10):
        k0, k1 = np.uint64((seed + i * 0x9E3779B9) % 2**32), np.uint64(((seed >> 32) + i * 0xBB67AE85) % 2**32)
        left, right = np.uint64(0xD2511F53) * ctr[0], np.uint64(0xCD9E8D57) * ctr[2]
        ctr = [(right >> half) ^ ctr[1] ^ k0, right & low, (left >> half) ^ ctr[3] ^ k1, left & low]
    bits = np.empty((at.size, 8), dtype=np.uint16)
    for j in range(8):
        bits[:, j] = ctr[j // 2] >> np.uint64(16 * (j % 2)) & np.uint64(0xFFFF)
    limit = round(s["p"] * 65536)
    kept = (bits.reshape(T, -1)[:, :H] >= limit).astype(np.float64)
    return torch.from_numpy(kept * (65536 / (65536 - limit))).cuda()


def _exact_drop(s):
    f = _factors(s)
    y = s["x"].double() * f
    return {"y": y if s["res"] is None else y + s["res"].double(), "dx": s["dy"].double() * f}


def _exact_ln(s):
    H = s["H"]
    f = _factors(s)
    z = s["h"].double() + s["y"].double() * f
    v = z.to(s["h"].dtype).double()
    mu = v.sum(1, keepdim=True) / H
    sd = ((v - mu).pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
    xn = (v - mu) / sd
    w = s["w"].double()
    out = {"h_out": z, "n": xn * w + (0.0 if s["b"] is None else s["b"].double())}
    if s["train"]:
        dn = s["d_n"].double()
        g = dn * w
        d = s["d_h_out"].double() + (H * g - g.sum(1, keepdim=True) - xn * (g * xn).sum(1, keepdim=True)) / (H * sd)
        out.update(d_h=d, d_y=d * f, d_w=(dn * xn).sum(0))
        if s["b"] is not None:
            out["d_b"] = dn.sum(0)
    return out


def _exact_i8(s):
    N = s["N"]
    out = torch.zeros(s["R"], N, dtype=torch.float64, device="cuda")
    counts, offsets = s["counts"].tolist(), s["offsets"].tolist()
    weights = (s["codes"], s["scales"])
    for e in range(s["E"]):
        a = e * s["cap"] if s["cap"] else offsets[e]
        n = min(counts[e], s["cap"]) if s["cap"] else counts[e]
        if n == 0:
            continue
        y = (s["x"][a:a + n].double() * s["x_scales"][a:a + n, None].double()) @ (weights[0][e].double() * weights[1][e, :, None].double()).t()
        out[a:a + n] = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:] if s["paired"] else y
    return out


def _exact_quant(s):
    x = s["x"].double()
    live = torch.zeros(s["R"], 1, dtype=torch.float64, device="cuda")
    counts, offsets = s["counts"].tolist(), s["offsets"].tolist()
    for e, n in enumerate(counts):
        a = e * s["cap"] if s["cap"] else offsets[e]
        live[a:a + (min(n, s["cap"]) if s["cap"] else n)] = 1
    top = x.abs().amax(1, keepdim=True)
    step = top / 127
    # 127 x is exact here, so halves are halves
    q = torch.where(top > 0, torch.round(127 * x / torch.where(top > 0, top, 1.0)), 0.0)
    return {"q": q * step * live, "scales": (step * live)[:, 0]}
