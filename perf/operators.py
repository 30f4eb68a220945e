"""Cases for the operators around dispatch and combine in a mixture-of-experts block.

  route  the choice of experts from router logits, with the balance loss, the z loss, per-expert counts
         and their gradients
  w4     the experts' products over the receive buffer with 4-bit weights and group scales, alone or as
         the gate/up pair of a SwiGLU
  norm   the norm after a block, its gate and residual scale, and the norm before the next block, with
         gradients

Sizes are those of this library's workloads (hidden 1024, 4096 and 7168; 16, 128 and 256 experts; batches
of 128, 4096 and 16384 tokens) with an expert width of 2048, and generic odd ones.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BALANCE, ZCOEF = 1e-2, 1e-3


# ------------------------------------------------------------------ cases

def listed():
    return [
        # router of one decode batch while serving: latency of the top-k choice alone
        dict(name="route_serve_128x256", op="route", T=128, E=256, k=8, groups=1, topk_groups=1, dtype="f32", train=False,
             seqs=1, full=False, bias=True, holes=False),
        # router of a prefill-sized training batch, one sequence
        dict(name="route_train_4096x256", op="route", T=4096, E=256, k=8, groups=1, topk_groups=1, dtype="f32", train=True,
             seqs=1, full=False, bias=False, holes=False),
        # group-limited routing of the largest batch, ragged sequences with padding, loss per sequence
        dict(name="route_train_grouped_16384x128", op="route", T=16384, E=128, k=8, groups=8, topk_groups=4, dtype="bf16",
             train=True, seqs=9, full=False, bias=True, holes=True),
        # odd sizes, masked experts and rows with nothing to choose, weights from the full softmax
        dict(name="route_train_odd_777x60", op="route", T=777, E=60, k=4, groups=1, topk_groups=1, dtype="f32", train=True,
             seqs=3, full=True, bias=False, holes=True),
        # one token through one matrix: the smallest product
        dict(name="w4_one_row_7168x4096", op="w4", T=1, E=1, k=1, K=4096, N=7168, group=128, paired=False, x="bf16", cap=0),
        # gate and up products of the decode batch, fp8 rows as the dispatch left them in the capacity buffer
        dict(name="w4_decode_gate_up", op="w4", T=128, E=256, k=8, K=7168, N=2048, group=128, paired=True, x="fp8", cap=128),
        # down product of the same batch, packed rows, finer groups
        dict(name="w4_decode_down", op="w4", T=128, E=256, k=8, K=2048, N=7168, group=64, paired=False, x="bf16", cap=0),
        # the tiny workload: 32 rows an expert, an odd width
        dict(name="w4_tiny_32_rows", op="w4", T=128, E=16, k=4, K=1024, N=1000, group=32, paired=True, x="bf16", cap=0),
        # serving: block end of one decode batch
        dict(name="norm_serve_128x7168", op="norm", T=128, H=7168, dtype="bf16", gate="channel", scale=True, post=True, train=False),
        # training step over the prefill batch
        dict(name="norm_train_4096x7168", op="norm", T=4096, H=7168, dtype="bf16", gate="channel", scale=True, post=True, train=True),
        # training step over the largest batch with a residual stream in 32 bits and a gate for each token
        dict(name="norm_train_16384x4096", op="norm", T=16384, H=4096, dtype="f32", gate="token", scale=True, post=True, train=True),
        # odd sizes, no gate
        dict(name="norm_train_odd_333x1000", op="norm", T=333, H=1000, dtype="bf16", gate="none", scale=False, post=True, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "w4", "norm"])
    if op == "route":
        per = _log(rng, 4, 64)
        groups = rng.choice([1, 1, 2, 4, 8])
        E = min(per * groups, 512)
        E -= E % groups
        T = min(_log(rng, 1, 32768), (16384 * 256) // E)
        topk_groups = max(1, groups // 2)
        k = rng.randint(1, min(8, E // groups * topk_groups))
        return dict(op="route", T=T, E=E, k=k, groups=groups, topk_groups=topk_groups, dtype=rng.choice(["f32", "bf16"]),
                    train=rng.random() < 0.7, seqs=rng.randint(1, 16), full=rng.random() < 0.4, bias=rng.random() < 0.5,
                    holes=rng.random() < 0.5)
    if op == "w4":
        E = rng.choice([1, _log(rng, 2, 256)])
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 192)
        x = rng.choice(["bf16", "fp8", "ue8m0"])
        K = _log(rng, 512, 7168)
        K = max(128, K - K % (8 if x == "bf16" else 128))
        paired = rng.random() < 0.5
        N = _log(rng, 256, 7168)
        N = min(N, 256 * 2048 * 7168 // (E * K))
        N = max(8, N - N % 8)
        return dict(op="w4", T=T, E=E, k=k, K=K, N=N, group=rng.choice([32, 64, 128]), paired=paired, x=x,
                    cap=rng.choice([0, T]))
    H = _log(rng, 256, 8192)
    H = max(8, H - H % 8)
    T = min(_log(rng, 1, 16384), 16384 * 4096 // H)
    return dict(op="norm", T=T, H=H, dtype=rng.choice(["bf16", "f32"]), gate=rng.choice(["none", "channel", "token"]),
                scale=rng.random() < 0.5, post=rng.random() < 0.8, train=rng.random() < 0.7)


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"route": _prepare_route, "w4": _prepare_w4, "norm": _prepare_norm}[case["op"]](case, g)


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _prepare_route(c, g):
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    # some experts are liked more than others, as early in training
    logits = _randn(g, T, E) + _randn(g, 1, E, scale=0.7)
    if c["holes"]:
        # experts that are switched off for a token, and tokens for which all or almost all are
        logits.masked_fill_(torch.rand(T, E, generator=g, device="cuda") < 0.05, -math.inf)
        few = torch.rand(T, 1, generator=g, device="cuda")
        logits = torch.where((few < 0.01) & (torch.arange(E, device="cuda") > 1), torch.full_like(logits, -math.inf), logits)
        logits = torch.where(few > 0.995, torch.full_like(logits, -math.inf), logits)
    logits = logits.to(dtype)
    s = dict(c, logits=logits, select_bias=_randn(g, E, scale=0.1) if c["bias"] else None, mask=None, seq_offsets=None)
    if c["holes"]:
        s["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)  # padding
    if S > 1:
        cut = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, T], device="cuda")
        s["seq_offsets"] = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)
    if c["train"]:
        s["d_topk_w"] = _randn(g, T, k, scale=1e-3)
        s["d_losses"] = torch.tensor([1.0, 0.5], device="cuda")
    if own:
        import combine_ep_get_04_gb300 as ep
        s["router"] = ep.Router(T, E, k, groups=c["groups"], topk_groups=c["topk_groups"], full_softmax=c["full"], dtype=dtype,
                                num_seqs=S, balance_coef=BALANCE, z_coef=ZCOEF, train=c["train"])
    return s


def _prepare_w4(c, g):
    T, E, k, K, N, G = c["T"], c["E"], c["k"], c["K"], c["N"], c["group"]
    rows = 2 * N if c["paired"] else N
    topk = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k]
    counts = torch.bincount(topk.reshape(-1), minlength=E).to(torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)
    R = E * c["cap"] if c["cap"] else T * k
    codes = torch.randint(0, 256, (E, rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(E, rows, -(-K // G), generator=g, device="cuda") + 0.5).mul_(0.2 / math.sqrt(K)).to(torch.bfloat16)
    x, x_scales = _randn(g, R, K, dtype=torch.bfloat16), None
    if c["x"] != "bf16":  # as the dispatch quantises: blocks of 128 channels
        b = x.float().view(R, K // 128, 128)
        x_scales = b.abs().amax(2).clamp_min(1e-4) / 448
        if c["x"] == "ue8m0":
            e = torch.ceil(torch.log2(x_scales))
            x = (b * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(R, K)
            x_scales = (e + 127).to(torch.uint8)
        else:
            x = (b / x_scales[..., None]).to(torch.float8_e4m3fn).view(R, K)
    s = dict(c, x=x, x_scales=x_scales, counts=counts, offsets=offsets, R=R)
    if own:
        import combine_ep_get_04_gb300 as ep
        s["weights"] = ep.W4Weights(codes, scales, group=G, paired=c["paired"])
        s["out"] = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    else:
        s["codes"], s["scales"] = codes, scales
    return s


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = dict(c, h=_randn(g, T, H, scale=2.0, dtype=dtype), y=_randn(g, T, H, scale=0.5, dtype=torch.bfloat16),
             w_post=1 + _randn(g, H, scale=0.1) if c["post"] else None, w_pre=1 + _randn(g, H, scale=0.1), gate=None,
             case_gate=c["gate"], res_scale=None)
    if c["gate"] != "none":
        s["gate"] = 0.5 + _randn(g, H if c["gate"] == "channel" else T, scale=0.2)
    if c["scale"]:
        s["res_scale"] = 0.9 + 0.1 * torch.rand(1, generator=g, device="cuda")
    if c["train"]:
        s["d_h_out"] = (_randn(g, T, H) + 0.1 * s["h"].float()).to(dtype)
        s["d_n"] = _randn(g, T, H, dtype=torch.bfloat16)
    if own:
        import combine_ep_get_04_gb300 as ep
        s["norm"] = ep.BlockNorm(T, H, dtype=dtype, gate=None if c["gate"] == "none" else c["gate"], post=c["post"],
                                 scaled=c["scale"], eps=EPS, train=c["train"])
    return s


# ------------------------------------------------------------------- runs

def run(s):
    return {"route": _run_route, "w4": _run_w4, "norm": _run_norm}[s["op"]](s)


def _run_route(s):
    if own:
        r = s["router"]
        o = r.route(s["logits"], s["select_bias"], s["mask"], s["seq_offsets"])
        if not s["train"]:
            return {"topk_idx": o.topk_idx, "topk_w": o.topk_w}
        d = r.backward(s["logits"], s["d_topk_w"], s["d_losses"], s["seq_offsets"])
        return {"topk_idx": o.topk_idx, "topk_w": o.topk_w, "counts": o.counts, "prob_sums": o.prob_sums, "losses": o.losses,
                "d_logits": d}
    T, E, k, S, G = s["T"], s["E"], s["k"], s["seqs"], s["groups"]
    x = s["logits"].float()
    sel = x if s["select_bias"] is None else x + s["select_bias"]
    live = torch.isfinite(x).any(1)
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)
    sel = torch.where(live[:, None], sel, -math.inf)
    if G > 1:
        order = sel.view(T, G, -1).amax(2).sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order[:, : s["topk_groups"]], True)
        sel = torch.where(keep[:, :, None], sel.view(T, G, -1), -math.inf).view(T, E)
    ranked = sel.sort(dim=1, descending=True, stable=True)
    idx, got = ranked.indices[:, :k], ranked.values[:, :k] > -math.inf
    top = torch.where(live, x.amax(1), 0.0)
    lse = torch.where(live, top + torch.log(torch.exp(x - top[:, None]).sum(1)), 0.0)
    p = torch.where(live[:, None], torch.exp(x - lse[:, None]), 0.0)
    if s["full"]:
        w = torch.where(got, p.gather(1, idx), 0.0)
    else:
        chosen = torch.where(got, x.gather(1, idx), -math.inf)
        e = torch.where(got, torch.exp(chosen - chosen.amax(1, keepdim=True)), 0.0)
        w = torch.where(got, e / e.sum(1, keepdim=True), 0.0)
    topk_idx = torch.where(got, idx, -1).to(torch.int32)
    if not s["train"]:
        return {"topk_idx": topk_idx, "topk_w": w}
    if S > 1:
        seq = torch.searchsorted(s["seq_offsets"][1:].contiguous(), torch.arange(T, dtype=torch.int32, device=x.device), right=True)
    else:
        seq = torch.zeros(T, dtype=torch.int64, device=x.device)
    member = (seq[None] == torch.arange(S, device=x.device)[:, None]) & live
    n = member.sum(1).float()
    counts = torch.zeros(S * E, dtype=torch.int32, device=x.device)
    counts = counts.scatter_add_(0, (seq[:, None] * E + idx).reshape(-1), got.reshape(-1).to(torch.int32)).view(S, E)
    prob_sums = member.float() @ p
    share = E / (k * n.clamp_min(1) ** 2)
    full_seqs, tokens = (n > 0).sum().clamp_min(1), n.sum().clamp_min(1)
    balance = BALANCE * (share * (counts * prob_sums).sum(1)).sum() / full_seqs
    z = ZCOEF * (lse * lse).sum() / tokens
    da, dz = s["d_losses"][0], s["d_losses"][1]
    gp = (da * BALANCE / full_seqs * share)[seq][:, None] * counts[seq]
    if s["full"]:
        gp = gp.scatter_add(1, idx, torch.where(got, s["d_topk_w"], 0.0))
    d = p * (gp - (p * gp).sum(1, keepdim=True)) + (2 * ZCOEF * dz / tokens * lse)[:, None] * p
    if not s["full"]:
        dw = torch.where(got, s["d_topk_w"], 0.0)
        d = d.scatter_add(1, idx, w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"topk_idx": topk_idx, "topk_w": w, "counts": counts, "prob_sums": prob_sums, "losses": torch.stack([balance, z]),
            "d_logits": d.to(s["logits"].dtype)}


def _run_w4(s):
    if own:
        import combine_ep_get_04_gb300 as ep
        return ep.expert_w4(s["x"], s["weights"], s["counts"], s["offsets"], capacity=s["cap"] or None, x_scales=s["x_scales"],
                            max_rows=s["T"] * s["k"], out=s["out"])
    E, K, N, G, T, R = s["E"], s["K"], s["N"], s["group"], s["T"], s["R"]
    c = s["codes"]
    w = torch.stack([c & 15, c >> 4], dim=-1).reshape(E, -1, K).float()
    w -= 8
    w *= s["scales"].float().repeat_interleave(G, 2)[..., :K]
    x = s["x"].float()
    if s["x"].dtype != torch.bfloat16:
        xs = s["x_scales"]
        xs = torch.exp2(xs.float() - 127) if xs.dtype == torch.uint8 else xs
        x = (x.view(R, -1, 128) * xs[..., None]).view(R, K)
    at = torch.arange(T, device=x.device)
    start = (torch.arange(E, device=x.device) * s["cap"] if s["cap"] else s["offsets"][:E].long())[:, None] + at
    rows = torch.where(at < s["counts"][:, None], start, R)
    y = torch.bmm(x[rows.clamp_max(R - 1)], w.transpose(1, 2))
    if s["paired"]:
        gate, up = y[..., :N], y[..., N:]
        y = gate / (1 + torch.exp(-gate)) * up
    out = torch.zeros(R + 1, N, dtype=torch.bfloat16, device=x.device)
    return out.index_copy_(0, rows.reshape(-1), y.reshape(-1, N).to(torch.bfloat16))[:R]


def _run_norm(s):
    if own:
        m = s["norm"]
        h_out, n = m.forward(s["h"], s["y"], s["w_post"], s["w_pre"], s["gate"], s["res_scale"])
        out = {"h_out": h_out, "n": n}
        if s["train"]:
            d = m.backward(s["h"], s["y"], s["w_post"], s["w_pre"], s["gate"], s["res_scale"], s["d_h_out"], s["d_n"])
            out.update(d_h=d.d_h, d_y=d.d_y, d_w_pre=d.d_w_pre)
            if s["post"]:
                out["d_w_post"] = d.d_w_post
            if s["gate"] is not None:
                out["d_gate"] = d.d_gate
            if s["scale"]:
                out["d_res_scale"] = d.d_res_scale
        return out
    h, y = s["h"].float(), s["y"].float()
    if s["post"]:
        r1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        yn = y * r1
        u = yn * s["w_post"]
    else:
        u = y
    gate = 1.0 if s["gate"] is None else s["gate"] if s["case_gate"] == "channel" else s["gate"][:, None]
    a = 1.0 if s["res_scale"] is None else s["res_scale"]
    h2 = a * h + gate * u
    r2 = torch.rsqrt((h2 * h2).mean(1, keepdim=True) + EPS)
    hn = h2 * r2
    out = {"h_out": h2.to(s["h"].dtype), "n": (hn * s["w_pre"]).to(torch.bfloat16)}
    if not s["train"]:
        return out
    dn = s["d_n"].float()
    t = dn * s["w_pre"]
    dh2 = s["d_h_out"].float() + r2 * (t - hn * (t * hn).mean(1, keepdim=True))
    du = gate * dh2
    out["d_h"] = (a * dh2).to(s["h"].dtype)
    if s["post"]:
        t = du * s["w_post"]
        out["d_y"] = (r1 * (t - yn * (t * yn).mean(1, keepdim=True))).to(torch.bfloat16)
        out["d_w_post"] = (du * yn).sum(0)
    else:
        out["d_y"] = du.to(torch.bfloat16)
    out["d_w_pre"] = (dn * hn).sum(0)
    if s["gate"] is not None:
        out["d_gate"] = (dh2 * u).sum(0 if s["case_gate"] == "channel" else 1)
    if s["scale"]:
        out["d_res_scale"] = (dh2 * h).sum().view(1)
    return out


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        size = 4 if c["dtype"] == "f32" else 2
        b = T * E * size + 8 * T * k
        f = 5 * T * E
        if c["train"]:  # logits again, their gradient, the choice and its weights again with their gradient; counts and sums
            b += 2 * T * E * size + 12 * T * k + 8 * T + 16 * c["seqs"] * E
            f += 10 * T * E
        return {"bytes": b, "flops": f}
    if c["op"] == "w4":
        E, T, k, K, N = c["E"], c["T"], c["k"], c["K"], c["N"]
        rows = 2 * N if c["paired"] else N
        used = E * (1 - (1 - k / E) ** T)  # experts that some token chooses
        x = 2 * K if c["x"] == "bf16" else K + K // 128 * (4 if c["x"] == "fp8" else 1)
        return {"bytes": used * rows * (K / 2 + 2 * -(-K // c["group"])) + T * k * (x + 2 * N), "flops": 2.0 * T * k * rows * K}
    T, H = c["T"], c["H"]
    hs = 4 if c["dtype"] == "f32" else 2
    b = T * H * (2 * hs + 4)
    if c["train"]:
        b += T * H * (3 * hs + 6)
    return {"bytes": b, "flops": T * H * (32 if c["train"] else 12)}


# -------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "w4": _exact_w4, "norm": _exact_norm}[case["op"]](s)


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _exact_route(s):
    T, E, k, S = s["T"], s["E"], s["k"], s["seqs"]
    l = s["logits"].float().cpu().numpy()
    pick = l if s["select_bias"] is None else l + s["select_bias"].cpu().numpy()  # the rule adds in 32 bits
    l = l.astype(np.float64)
    live = (l > -np.inf).any(1)
    if s["mask"] is not None:
        live &= s["mask"].cpu().numpy() != 0
    pick = np.where(live[:, None], pick, -np.inf).astype(np.float64)
    if s["groups"] > 1:
        best = pick.reshape(T, s["groups"], -1).max(2)
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1, kind="stable")
        off = np.repeat(rank >= s["topk_groups"], E // s["groups"], axis=1)
        pick[off] = -np.inf
    idx = np.argsort(-pick, axis=1, kind="stable")[:, :k]
    got = np.take_along_axis(pick, idx, 1) > -np.inf
    top = np.where(live, l.max(1), 0.0)
    expd = np.where(live[:, None], np.exp(l - top[:, None]), 0.0)
    z = np.where(live, expd.sum(1), 1.0)
    p = expd / z[:, None]
    lse = np.where(live, top + np.log(z), 0.0)
    w = np.where(got, np.take_along_axis(p, idx, 1), 0.0)
    if not s["full"]:
        total = w.sum(1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    dev = s["logits"].device
    out = {"topk_idx": None, "topk_w": torch.from_numpy(w).to(dev)}
    if not s["train"]:
        return out
    bounds = [0, T] if S == 1 else s["seq_offsets"].cpu().tolist()
    da, dz = _np(s["d_losses"])
    dw = np.where(got, _np(s["d_topk_w"]), 0.0)
    sums, slope, balance = np.zeros((S, E)), np.zeros((T, E)), 0.0
    spans = [(a, b) for a, b in zip(bounds, bounds[1:])]
    filled, tokens = max(1, sum(bool(live[a:b].any()) for a, b in spans)), max(1, int(live.sum()))
    for i, (a, b) in enumerate(spans):
        m = int(live[a:b].sum())
        if m == 0:
            continue
        count = np.bincount(idx[a:b][got[a:b]], minlength=E)
        sums[i] = p[a:b].sum(0)
        c = BALANCE * E / (k * m * m * filled)
        balance += c * (count * sums[i]).sum()
        slope[a:b] = da * c * count
    at = np.arange(T)[:, None]
    if s["full"]:
        np.add.at(slope, (np.broadcast_to(at, idx.shape), idx), dw)
    d = p * (slope - (p * slope).sum(1, keepdims=True)) + (2 * ZCOEF * dz / tokens * lse)[:, None] * p
    if not s["full"]:
        np.add.at(d, (np.broadcast_to(at, idx.shape), idx), w * (dw - (w * dw).sum(1, keepdims=True)))
    out.update(counts=None, prob_sums=torch.from_numpy(sums).to(dev),
               losses=torch.tensor([balance, ZCOEF * (lse ** 2).sum() / tokens], dtype=torch.float64, device=dev),
               d_logits=torch.from_numpy(d).to(dev))
    return out


def _exact_w4(s):
    N, K, G = s["N"], s["K"], s["group"]
    out = torch.zeros(s["R"], N, dtype=torch.float64, device="cuda")
    counts, offsets = s["counts"].tolist(), s["offsets"].tolist()
    channel = torch.arange(K, device="cuda")
    for e in range(s["E"]):
        if counts[e] == 0:
            continue
        a = e * s["cap"] if s["cap"] else offsets[e]
        x = s["x"][a:a + counts[e]].to(torch.float32).double()
        if s["x_scales"] is not None:
            xs = s["x_scales"][a:a + counts[e]].double()
            xs = 2.0 ** (xs - 127) if s["x_scales"].dtype == torch.uint8 else xs
            x = x * xs[:, channel // 128]
        byte = s["codes"][e][:, channel // 2].int()
        q = torch.where(channel % 2 == 0, byte % 16, byte // 16).double() - 8
        y = x @ (q * s["scales"][e].double()[:, channel // G]).t()
        out[a:a + counts[e]] = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:] if s["paired"] else y
    return out


def _exact_norm(s):
    T, H = s["T"], s["H"]
    part = 2048  # rows at a time
    keep = {}
    a = 1.0 if s["res_scale"] is None else s["res_scale"].double()
    wp, wq = s["w_pre"].double(), None if s["w_post"] is None else s["w_post"].double()
    sums = {"d_w_pre": 0.0, "d_w_post": 0.0, "d_gate": 0.0, "d_res_scale": 0.0}
    for t in range(0, T, part):
        h, y = s["h"][t:t + part].double(), s["y"][t:t + part].double()
        gate = torch.ones((), dtype=torch.float64, device="cuda")
        if s["gate"] is not None:
            gate = s["gate"].double() if s["case_gate"] == "channel" else s["gate"][t:t + part, None].double()
        sy = (y.pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
        v = y / sy if wq is not None else y
        u = v * wq if wq is not None else v
        hh = a * h + gate * u
        sh = (hh.pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
        piece = {"h_out": hh, "n": hh / sh * wp}
        if s["train"]:
            dn = s["d_n"][t:t + part].double()
            lead = dn * wp
            dhh = s["d_h_out"][t:t + part].double() + lead / sh - hh * (lead * hh).sum(1, keepdim=True) / (H * sh ** 3)
            du = gate * dhh
            piece["d_h"] = a * dhh
            if wq is not None:
                lead = du * wq
                piece["d_y"] = lead / sy - y * (lead * y).sum(1, keepdim=True) / (H * sy ** 3)
                sums["d_w_post"] = sums["d_w_post"] + (du * v).sum(0)
            else:
                piece["d_y"] = du
            sums["d_w_pre"] = sums["d_w_pre"] + (dn * hh / sh).sum(0)
            if s["case_gate"] == "channel":
                sums["d_gate"] = sums["d_gate"] + (dhh * u).sum(0)
            elif s["case_gate"] == "token":
                piece["d_gate"] = (dhh * u).sum(1)
            sums["d_res_scale"] = sums["d_res_scale"] + (dhh * h).sum().view(1)
        for name, v in piece.items():
            keep.setdefault(name, []).append(v)
    out = {name: torch.cat(v) for name, v in keep.items()}
    if s["train"]:
        out["d_w_pre"] = sums["d_w_pre"]
        if wq is not None:
            out["d_w_post"] = sums["d_w_post"]
        if s["case_gate"] == "channel":
            out["d_gate"] = sums["d_gate"]
        if s["res_scale"] is not None:
            out["d_res_scale"] = sums["d_res_scale"]
    return out
