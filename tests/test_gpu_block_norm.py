"""ep_block_norm and its gradients against a plain 64-bit implementation.

The bounds come from the formulas (block_reference.bound): a row's sums have H
terms, sums over rows T terms, each result is rounded once to its type.
"""
import os
import subprocess

import numpy as np
import pytest
import torch

import block_reference as ref
import combine_ep_get_04_gb300 as ep

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(T, H, dtype, gate, post, pre, scaled, block=True, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dt=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    def rows(dt, scale):   # rows `pad` elements further apart than their length
        return rand(T, H + pad, dt=dt, scale=scale)[:, :H] if pad else rand(T, H, dt=dt, scale=scale)

    return dict(h=rows(dtype, 2.0), y=rows(torch.bfloat16, 0.5) if block else None,
                w_post=1 + rand(H, scale=0.1) if post else None, w_pre=1 + rand(H, scale=0.1) if pre else None,
                gate=None if gate is None else 0.5 + rand(H if gate == "channel" else T, scale=0.2),
                res_scale=torch.full((1,), 0.9, device="cuda") if scaled else None), \
        dict(d_h_out=rand(T, H, dt=dtype), d_n=rand(T, H, dt=torch.bfloat16) if pre else None)


def check(T, H, dtype, gate, post, pre, scaled, block=True, pad=0, edit=None, d_h_out=True):
    inputs, grads = make(T, H, dtype, gate, post, pre, scaled, block, pad=pad)
    if not d_h_out:
        grads["d_h_out"] = None
    if edit is not None:
        edit(inputs)
    m = ep.BlockNorm(T, H, dtype, gate=gate, post=post, pre=pre, scaled=scaled, block=block, eps=EPS, train=True)
    h_out, n = m.forward(**inputs)
    d = m.backward(**inputs, **grads)
    got = dict(h_out=h_out, n=n, d_h=d.d_h, d_y=d.d_y, d_w_post=d.d_w_post, d_w_pre=d.d_w_pre, d_gate=d.d_gate,
               d_res_scale=d.d_res_scale)
    torch.cuda.synchronize()
    r = {k: f64(v) for k, v in inputs.items()}
    if gate == "token":
        r["gate"] = r["gate"][:, None]
    r["res_scale"] = 1.0 if r["res_scale"] is None else r["res_scale"][0]
    v, z = ref.block_norm(**r, eps=EPS, **{k: f64(x) for k, x in grads.items()})
    for name, x in got.items():
        if x is None:
            continue
        terms = {"d_w_post": H + T, "d_w_pre": H + T, "d_res_scale": T * H}.get(name, H + T if gate == "channel" and name == "d_gate" else H)
        b = ref.bound(v[name], z[name], terms, x.dtype == torch.bfloat16)
        off = np.abs(f64(x) - v[name])
        assert (off <= b).all(), f"{name}: {(off > b).sum()} of {off.size} beyond the bound, worst {(off - b).max():.3g} past it"
    return got


SIZES = [(1, 8), (1, 7168), (2, 16), (3, 256), (5, 264), (7, 512), (9, 520), (130, 1000), (333, 1024), (40, 2056), (64, 4096),
         (131, 7168), (17, 8192), (9, 8200), (6, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H, dtype):
    check(T, H, dtype, "channel", True, True, True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("scaled", [False, True])
def test_forms(dtype, gate, post, pre, scaled):
    for T, H in ((37, 1000), (200, 264)):
        check(T, H, dtype, gate, post, pre, scaled)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_first_norm_of_a_network(dtype):
    check(37, 1000, dtype, None, False, True, False, block=False)
    check(37, 1000, dtype, None, False, True, True, block=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_further_apart_than_their_length(dtype):
    check(33, 1000, dtype, "token", True, True, True, pad=24)


def test_no_gradient_of_the_stream():
    check(33, 1000, torch.bfloat16, "channel", True, True, True, d_h_out=False)


def test_more_rows_than_the_grid_holds():
    check(4099, 64, torch.float32, "channel", True, True, True)
    check(2051, 2048, torch.bfloat16, "token", True, True, True)


@pytest.mark.parametrize("T,H,dtype,gate,post,pre,scaled,block,pad", [
    (3040, 4104, torch.bfloat16, "channel", True, True, True, True, 0), (3041, 4096, torch.float32, "token", True, True, True, True, 0),
    (6100, 4104, torch.bfloat16, "token", True, True, True, True, 24), (3200, 7936, torch.float32, "channel", True, True, False, True, 8),
    (3333, 7168, torch.bfloat16, None, True, True, False, True, 0), (3100, 5000, torch.float32, "token", False, True, True, True, 0),
    (3100, 5000, torch.bfloat16, "channel", True, False, True, True, 0), (3100, 4800, torch.float32, "channel", False, False, True, True, 0),
    (3100, 6008, torch.bfloat16, None, False, True, True, False, 0), (4000, 7944, torch.bfloat16, "token", True, True, True, True, 0)])
def test_many_wide_rows(T, H, dtype, gate, post, pre, scaled, block, pad):
    """The first and the last rows, all of some CTAs' and some of the others'."""
    inputs, _ = make(T, H, dtype, gate, post, pre, scaled, block, pad=pad)
    m = ep.BlockNorm(T, H, dtype, gate=gate, post=post, pre=pre, scaled=scaled, block=block, eps=EPS, train=True)
    m.h_out.fill_(float("nan"))
    h_out, n = m.forward(**inputs)
    rows = torch.tensor(sorted({t for t in range(T) if t < 4 or t >= T - 160 or t % 152 in (5, 151) or t % 53 == 0}), device="cuda")
    r = {k: v if k in ("w_post", "w_pre", "res_scale") or (k == "gate" and gate != "token") or v is None else v[rows] for k, v in inputs.items()}
    r = {k: f64(v) for k, v in r.items()}
    if gate == "token":
        r["gate"] = r["gate"][:, None]
    r["res_scale"] = 1.0 if r["res_scale"] is None else r["res_scale"][0]
    v, z = ref.block_norm(**r, eps=EPS)
    for name, x in dict(h_out=h_out, n=n).items():
        if x is None:
            continue
        b = ref.bound(v[name], z[name], H, x.dtype == torch.bfloat16)
        off = np.abs(f64(x[rows]) - v[name])
        assert (off <= b).all(), f"{name}: {(off > b).sum()} of {off.size} beyond the bound, worst {(off - b).max():.3g} past it"
    assert torch.isfinite(h_out).all() and (n is None or torch.isfinite(n).all())
    # a root's relative error is half its argument's
    for i, (there, x) in enumerate(((post, r["y"]), (pre, v["h_out"]))):
        if there:
            want = 1 / np.sqrt((x * x).mean(1) + EPS)
            slack = np.sqrt((z["h_out"] ** 2).mean(1) / (x * x).mean(1)) if i else 1.0
            assert (np.abs(f64(m.rstd[i][rows]) / want - 1) <= (H + 64) * ref.EPS32 * slack).all()
    want = [None if x is None else x.clone() for x in (h_out, n)]
    m.forward(**inputs)
    assert torch.equal(m.h_out, want[0]) and (n is None or torch.equal(m.n, want[1]))
    if not pad:
        m.h_out = inputs["h"]                        # in place
        m.forward(**inputs)
        assert torch.equal(inputs["h"], want[0]) and (n is None or torch.equal(m.n, want[1]))


def test_rows_of_zeros():
    """A row of zeros has mean square 0: eps alone stands under the root."""
    def edit(i):
        i["h"][3].zero_()
        i["y"][3].zero_()
        i["y"][5].zero_()
    got = check(9, 1000, torch.float32, "channel", True, True, True, edit=edit)
    assert not got["h_out"][3].any() and not got["n"][3].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_stays_alone(bad):
    inputs, grads = make(12, 1000, torch.bfloat16, "token", True, True, True)
    m = ep.BlockNorm(12, 1000, gate="token", scaled=True, eps=EPS)
    clean = [t.clone() for t in m.forward(**inputs)]
    inputs["y"][4, 7] = bad
    h_out, n = m.forward(**inputs)
    others = [t for t in range(12) if t != 4]
    assert torch.equal(h_out[others], clean[0][others]) and torch.equal(n[others], clean[1][others])
    assert torch.isnan(n[4].float()).any()


def test_same_bits_twice_and_on_another_stream():
    inputs, grads = make(1000, 7168, torch.bfloat16, "channel", True, True, True)
    m = ep.BlockNorm(1000, 7168, gate="channel", scaled=True, eps=EPS, train=True)

    def run(stream=None):
        m.forward(**inputs, stream=stream)
        g = m.backward(**inputs, **grads, stream=stream)
        if stream is not None:
            stream.synchronize()
        torch.cuda.synchronize()
        return [t.clone() for t in (m.h_out, m.n, g.d_h, g.d_y, g.d_w_post, g.d_w_pre, g.d_gate, g.d_res_scale)]

    a = run()
    for b in (run(), run(torch.cuda.Stream())):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_h_out_in_place_of_h():
    inputs, _ = make(50, 1000, torch.float32, "channel", True, True, True)
    m = ep.BlockNorm(50, 1000, torch.float32, gate="channel", scaled=True, eps=EPS)
    want = [t.clone() for t in m.forward(**inputs)]
    m.h_out = inputs["h"]
    m.forward(**inputs)
    assert torch.equal(inputs["h"], want[0]) and torch.equal(m.n, want[1])


def test_no_rows():
    m = ep.BlockNorm(0, 64, gate="channel", scaled=True, train=True)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    a = torch.ones(1, device="cuda")
    m.forward(e, e, w, w, w, a)
    for t in (m.grads.d_w_post, m.grads.d_w_pre, m.grads.d_gate, m.grads.d_res_scale):
        t.fill_(7)
    g = m.backward(e, e, w, w, w, a, e, e)
    assert not any(t.any() for t in (g.d_w_post, g.d_w_pre, g.d_gate, g.d_res_scale))


def test_refusals():
    m = ep.BlockNorm(4, 64, gate="token", scaled=True)
    i, _ = make(4, 64, torch.bfloat16, "token", True, True, True)
    with pytest.raises(ValueError):
        m.forward(**{**i, "gate": None})
    with pytest.raises(ValueError):
        m.forward(**{**i, "h": i["h"][:, :32]})
    with pytest.raises(TypeError):
        m.forward(**{**i, "h": i["h"].float()})
    with pytest.raises(ValueError):
        m.forward(**{**i, "y": i["y"].cpu()})
    with pytest.raises(ValueError):
        m.forward(**{**i, "gate": torch.ones(64, device="cuda")})
    wide = torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ep.EPError):                     # rows 68 elements apart: not 16-byte aligned
        m.forward(**{**i, "h": wide[:, :64]})
    shifted = torch.zeros(4 * 72 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 72)
    with pytest.raises(ep.EPError):
        m.forward(**{**i, "h": shifted[:, :64]})
    with pytest.raises(ValueError):
        m.backward(**i)
    with pytest.raises(ep.EPError):
        ep.BlockNorm(4, 60)
    with pytest.raises(ep.EPError):
        ep.BlockNorm(4, 16392)
    with pytest.raises(ep.EPError):
        ep.BlockNorm(4, 64, eps=0.0)


def test_an_sm_holds_the_ctas_that_the_backward_pass_plans(tmp_path):
    from combine_ep_get_04_gb300 import build as B
    here = os.path.dirname(os.path.abspath(__file__))
    exe = tmp_path / "norm_occupancy"
    subprocess.run([B.nvcc(), *B.ARCH, *B.NVCC_FLAGS, os.path.join(here, "norm_occupancy.cu"), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr


def test_the_smallest_eps():
    """Rows of zeros: the reciprocal roots are as large as they get, and their
    products stay finite."""
    T, H = 6, 264
    inputs, grads = make(T, H, torch.float32, "channel", True, True, True)
    for t in (1, 4):
        inputs["h"][t], inputs["y"][t] = 0, 0
    m = ep.BlockNorm(T, H, torch.float32, gate="channel", scaled=True, eps=1e-30, train=True)
    h_out, n = m.forward(**inputs)
    grads["d_h_out"][[1, 4]] *= 1e-20            # the gradient of a row of zeros is eps^-1/2 times the one behind it
    grads["d_n"][[1, 4]] *= 1e-20
    d = m.backward(**inputs, **grads)
    r = {k: f64(v) for k, v in inputs.items()}
    r["res_scale"] = r["res_scale"][0]
    v, z = ref.block_norm(**r, eps=1e-30, **{k: f64(x) for k, x in grads.items()})
    for name, x in dict(h_out=h_out, n=n, d_h=d.d_h, d_y=d.d_y, d_w_post=d.d_w_post, d_w_pre=d.d_w_pre, d_gate=d.d_gate).items():
        b = ref.bound(v[name], z[name], H + T, x.dtype == torch.bfloat16)
        assert (np.abs(f64(x) - v[name]) <= b).all(), name
