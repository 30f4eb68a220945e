"""ep_layer_norm and its gradients over many rows, against the plain 64-bit
implementations and the bounds of layer_reference."""
import numpy as np
import pytest
import torch

import combine_ep_get_04_gb300 as ep
import layer_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def near(name, got, value, error):
    error = ref.stored(value, error, got.dtype == BF16)
    off = np.abs(f64(got) - value)
    assert (off <= error).all(), f"{name}: {(~(off <= error)).sum()} of {off.size} beyond the bound, worst {np.nanmax(off - error):.3g} past it"


def test_as_many_rows_as_there_are_numbers():
    """2^31 - 1 rows of 8 channels: every row is written, and some all over the buffer are compared."""
    T, H = 2 ** 31 - 1, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 * 2 ** 30:
        pytest.skip("the largest buffers do not fit")
    g = torch.Generator(device="cuda").manual_seed(0)
    h, d_n = (torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(2))
    w, b = 1 + 0.1 * torch.randn(H, generator=g, device="cuda"), 0.1 * torch.randn(H, generator=g, device="cuda")
    m = ep.LayerNorm(T, H, BF16, block=False, eps=EPS, train=True)
    m.n.fill_(float("nan"))
    m.grads.d_h.fill_(float("nan"))
    _, n = m.forward(h, w=w, b=b)
    d = m.backward(h, w, d_n)
    torch.cuda.synchronize()
    assert int(m.err_flags) == 0
    for a in range(0, T, 2 ** 26):
        assert not n[a:a + 2 ** 26].isnan().any() and not d.d_h[a:a + 2 ** 26].isnan().any(), a
    for a in (0, 2 ** 30 - 500, T - 1000):
        at = slice(a, a + 1000)
        n_v, n_e, s = ref.layer_norm(f64(h[at]), f64(w), f64(b), EPS)
        near("n", n[at], n_v, n_e)
        near("d_h", d.d_h[at], *ref.layer_norm_gradients(s, f64(d_n[at]), None, 1.0)["d_h"])
    assert torch.isfinite(d.d_w).all() and torch.isfinite(d.d_b).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [256, 520, 1032, 2056, 4104, 8200])
def test_an_infinite_gradient_by_its_place(H, dtype):
    """An infinity in d_n leaves in a row what the formula makes of it, infinities of either sign and NaN, whichever
    channel it stands in: swapping two channels of all inputs swaps them in all results."""
    T, place = 3, 123
    g = torch.Generator(device="cuda").manual_seed(H)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")     # noqa: E731
    h, d_n, dh, w = rand(T, H).to(dtype), rand(T, H).bfloat16(), rand(T, H).to(dtype), 1 + 0.1 * rand(H)
    h[:, 0] = 1.0                        # away from the mean, so that d_n times the normed value is an infinity too
    d_n[1, 0], d_n[2, 0] = float("inf"), float("-inf")
    swap = torch.arange(H, device="cuda")
    swap[0], swap[place] = place, 0
    m = ep.LayerNorm(T, H, dtype, bias=False, block=False, eps=EPS, train=True)
    x = d_n.double() * w.double()

    def run(at):
        hs = h[:, at].contiguous()
        m.forward(hs, w=w[at].contiguous())
        return m.backward(hs, w[at].contiguous(), d_n[:, at].contiguous(), dh[:, at].contiguous()).d_h.clone()

    first, other = run(torch.arange(H, device="cuda")), run(swap)[:, swap]
    v = h.double()
    xn = (v - v.mean(1, keepdim=True)) / (v.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
    want = x - x.mean(1, keepdim=True) - xn * (x * xn).mean(1, keepdim=True)
    assert want[1:].isinf().any() and torch.isfinite(want[0]).all()
    for got in (first, other):
        assert torch.isfinite(got[0]).all()
        for sign in (float("inf"), float("-inf")):
            assert torch.equal(got[1:] == sign, want[1:] == sign)
        assert torch.equal(got[1:].isnan(), want[1:].isnan())


def ring(T, H, row_bytes, sms):
    """CTAs of a call whose rows come through a ring, and its stages."""
    nv = 1 if H <= 4096 else 2 if H <= 8192 else 4
    warps = -(-H // 8 // (32 * nv))
    per_sm = 1 if nv > 1 else max(1, min(8, 20 // (warps + 1)))
    return min(T, sms * per_sm), max(1, min(8, (212 * 1024 // per_sm - 2048) // row_bytes))


@pytest.mark.parametrize("T,H,dtype", [(3 * 25 * 152, 1040, BF16), (2 * 25 * 152, 2048, BF16), (26 * 152, 7168, BF16), (27 * 152, 4096, F32),
                                       (16 * 152 + 7, 8192, F32), (10 * 152 + 3, 16384, BF16), (25 * 152, 5000, BF16)])
def test_many_rounds_of_the_ring(T, H, dtype):
    """Every stage, slot and barrier is used at least three times in both directions; all rows and the sums over them
    are compared.  The sums' bound counts the kernel's own chain of additions, the rows of a CTA, every 16th CTA and 16
    warps, so that any lost or doubled row lies outside it."""
    sms, size = torch.cuda.get_device_properties(0).multi_processor_count, 2 if dtype == BF16 else 4
    for row_bytes in (H * (size + 2), H * (2 * size + 2)):
        ctas, stages = ring(T, H, row_bytes, sms)
        assert T // ctas >= 3 * stages
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *shape, scale=1.0: torch.randn(*shape, generator=g, device="cuda") * scale     # noqa: E731
    h, y, d_n, dh = rand(T, H, scale=1.5).to(dtype), rand(T, H, scale=0.5).bfloat16(), rand(T, H).bfloat16(), rand(T, H).to(dtype)
    w, b, rng = 1 + rand(H, scale=0.1), rand(H, scale=0.1), torch.tensor([5, 6], device="cuda")
    m = ep.LayerNorm(T, H, dtype, p=0.1, site=2, eps=EPS, train=True)
    h_out, n = m.forward(h, y, w, b, rng)
    d = m.backward(h_out, w, d_n, dh, rng)
    torch.cuda.synchronize()
    assert int(m.err_flags) == 0
    f = ref.factors(T, H, 0.1, (5, 6), 2)
    near("h_out", h_out, *ref.dropped_sum(f64(y), f, f64(h)))
    n_v, n_e, s = ref.layer_norm(f64(h_out), f64(w), f64(b), EPS)
    near("n", n, n_v, n_e)
    dn = f64(d_n)
    grads = ref.layer_norm_gradients(s, dn, f64(dh), f)
    near("d_h", d.d_h, *grads["d_h"])
    near("d_y", d.d_y, *grads["d_y"])
    chain = -(-T // ctas) + ctas // 16 + 1 + 17
    for name, got, terms, off in (("d_w", d.d_w, np.abs(dn * s["xn"]), (np.abs(dn) * s["e_xn"]).sum(0)), ("d_b", d.d_b, np.abs(dn), 0.0)):
        error = off + (chain + 2) * ref.U * terms.sum(0)
        near(name, got, grads[name][0], error)
        assert (terms > error).any(1).all(), "a lost row would not show"


def test_gradients_are_those_of_the_last_forward():
    """From h_out or a copy of it; two batches on their way at once have a norm each."""
    T, H = 40, 1040
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda: torch.randn(T, H, generator=g, device="cuda")          # noqa: E731
    batches = [(rand() * (i + 1), rand().bfloat16(), rand().bfloat16()) for i in range(2)]
    w, rng = 1 + 0.1 * rand()[0], torch.tensor([1, 2], device="cuda")
    make = lambda: ep.LayerNorm(T, H, F32, p=0.1, bias=False, train=True)  # noqa: E731
    want = []
    for h, y, d_n in batches:
        m = make()
        copy = m.forward(h, y, w, rng=rng)[0].clone()
        want.append([t.clone() for t in (m.backward(m.h_out, w, d_n, rng=rng).d_h, m.grads.d_w)])
        d = m.backward(copy, w, d_n, rng=rng)
        assert torch.equal(d.d_h, want[-1][0]) and torch.equal(d.d_w, want[-1][1])
    norms = [make(), make()]
    outs = [m.forward(h, y, w, rng=rng)[0] for m, (h, y, _) in zip(norms, batches)]
    for m, h_out, (_, _, d_n), (d_h, d_w) in zip(norms, outs, batches, want):
        d = m.backward(h_out, w, d_n, rng=rng)
        assert torch.equal(d.d_h, d_h) and torch.equal(d.d_w, d_w)
