"""ep_layer_norm, its gradients and ep_dropout against plain 64-bit
implementations, within the bounds of layer_reference.  The norm is compared on
the h_out that the call stored, as it is defined."""
import numpy as np
import pytest
import torch

import combine_ep_get_04_gb300 as ep
import layer_reference as ref

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def near(name, got, value, error, rows=None):
    error = ref.stored(value, error, got.dtype == BF16)
    got = f64(got if rows is None else got[rows])
    off = np.abs(got - value)
    assert (off <= error).all(), f"{name}: {(~(off <= error)).sum()} of {off.size} beyond the bound, worst {np.nanmax(off - error):.3g} past it"


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows_of(g, T, H, dtype, scale=1.0, shift=0.0, pad=0):
    t = (torch.randn(T, H + pad, generator=g, device="cuda") * scale + shift).to(dtype)
    return t[:, :H] if pad else t


def words(*v):
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in v], device="cuda")


def check(T, H, dtype=BF16, p=0.1, weight=True, bias=True, block=True, d_h_out=True, pad=0, shift=0.3, site=3, seed=0, edit=None, rows=None,
          rng=True):
    """Forward and backward against the reference, all rows or some (the sums over rows only with all)."""
    g = generator(seed)
    h, y = rows_of(g, T, H, dtype, 1.5, shift, pad), rows_of(g, T, H, BF16, 0.5, pad=pad) if block else None
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda") if weight else None
    b = 0.1 * torch.randn(H, generator=g, device="cuda") if bias else None
    d_n, dh = rows_of(g, T, H, BF16), rows_of(g, T, H, dtype) if d_h_out else None
    if edit is not None:
        edit(h, y)
    words_ = words(0xFEDCBA9876543210, 2 ** 64 - 2) if rng and p else None
    m = ep.LayerNorm(T, H, dtype, p=p if block else 0.0, site=site, weight=weight, bias=bias, block=block, eps=EPS, train=True)
    h_out, n = m.forward(h, y, w, b, words_)
    d = m.backward(h_out, w, d_n, dh, words_)
    torch.cuda.synchronize()
    assert int(m.err_flags) == 0
    at = slice(None) if rows is None else torch.as_tensor(rows, device="cuda")
    f = ref.factors(T, H, p, words_.tolist() if words_ is not None else None, site, rows)
    if block:
        v, e = ref.dropped_sum(f64(y[at]), f, f64(h[at]))
        near("h_out", h_out, v, e, at)
    else:
        assert h_out is h
    n_v, n_e, s = ref.layer_norm(f64(h_out[at]), f64(w), f64(b), EPS)
    near("n", n, n_v, n_e, at)
    assert (np.abs(f64(m.stats[1][at]) / s["r"][:, 0] - 1) <= s["e_r"][:, 0]).all()
    grads = ref.layer_norm_gradients(s, f64(d_n[at]), None if dh is None else f64(dh[at]), f)
    for name, x in (("d_h", d.d_h), ("d_y", d.d_y), ("d_w", d.d_w), ("d_b", d.d_b)):
        if x is None or (rows is not None and x.dim() == 1):
            continue
        near(name, x, *grads[name], rows=at if x.dim() == 2 else None)
    return h_out, n, d, m


SIZES = [(1, 8), (1, 7168), (2, 16), (3, 256), (5, 264), (7, 512), (9, 520), (130, 1000), (333, 1024), (40, 2056), (64, 4096), (11, 4104),
         (131, 7168), (17, 8192), (9, 8200), (5, 12008), (6, 16384)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H, dtype):
    check(T, H, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("weight,bias", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("d_h_out", [True, False])
def test_forms(dtype, p, weight, bias, d_h_out):
    for T, H in ((37, 1000), (200, 264)):
        check(T, H, dtype, p, weight, bias, d_h_out=d_h_out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_first_norm_of_a_network(dtype):
    check(37, 1000, dtype, 0.0, block=False)
    check(37, 1000, dtype, 0.0, block=False, pad=24)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_further_apart_than_their_length(dtype):
    check(33, 1000, dtype, pad=24)


@pytest.mark.parametrize("T,H,dtype", [(4099, 64, F32), (2051, 2048, BF16), (1300, 4096, F32), (700, 7168, BF16), (500, 8192, F32),
                                       (330, 16384, F32), (400, 12000, BF16)])
def test_more_rows_than_the_grid_holds(T, H, dtype):
    check(T, H, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_far_from_zero(dtype):
    """The mean is a hundred deviations off: squares of the channels themselves would leave little of the variance."""
    check(41, 1032, dtype, shift=150.0)
    check(9, 7168, dtype, shift=-150.0)


def test_rows_without_a_spread():
    """A row of one value has variance 0: eps alone stands under the root."""
    def edit(h, y):
        h[3], y[3] = 2.0, 0.0
        h[4], y[4] = 0.0, 0.0
    h_out, n, _, m = check(9, 1000, F32, 0.0, bias=False, edit=edit)
    assert not n[3].any() and not n[4].any() and (m.stats[0][3] == 2).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_stays_alone(bad):
    def run(edit):
        g = generator(1)
        h, y = rows_of(g, 40, 1000, F32), rows_of(g, 40, 1000, BF16)
        w, d_n = torch.ones(1000, device="cuda"), rows_of(g, 40, 1000, BF16)
        if edit:
            h[7, 500] = bad
            y[9, 3] = bad
        m = ep.LayerNorm(40, 1000, F32, train=True)
        h_out, n = m.forward(h, y, w, w)
        d = m.backward(h_out, w, d_n)
        return h_out, n, d.d_h, d.d_y
    clean, got = run(False), run(True)
    rest = [t for t in range(40) if t not in (7, 9)]
    for a, b in zip(clean, got):
        assert torch.equal(a[rest], b[rest])
    assert got[1][[7, 9]].isnan().all() and got[2][[7, 9]].isnan().all()


def test_what_is_dropped_does_not_count():
    """Infinities and NaN where an element is dropped change nothing."""
    T, H, p, rng = 20, 264, 0.5, words(5, 6)
    f = torch.from_numpy(ref.factors(T, H, p, rng.tolist(), 0)).cuda()
    g = generator(0)
    h, y = rows_of(g, T, H, BF16), rows_of(g, T, H, BF16)
    m = ep.LayerNorm(T, H, p=p, weight=False, bias=False)
    want = [t.clone() for t in m.forward(h, y, rng=rng)]
    for bad in (float("nan"), float("inf")):
        z = torch.where(f == 0, torch.full_like(y, bad), y)
        for a, b in zip(want, m.forward(h, z, rng=rng)):
            assert torch.equal(a, b)
        assert torch.equal(ep.dropout(z, p, rng), ep.dropout(y, p, rng))
    assert torch.equal(ep.dropout(y, p, rng, residual=h), want[0])


def test_everything_and_nothing_dropped():
    g = generator(0)
    h, y, d_n = rows_of(g, 9, 64, F32), rows_of(g, 9, 64, BF16), rows_of(g, 9, 64, BF16)
    for p, rng in ((1.0, words(1, 2)), (0.3, None), (0.0, words(1, 2)), (2.0 ** -18, words(1, 2))):
        m = ep.LayerNorm(9, 64, F32, p=p, weight=False, bias=False, train=True)
        h_out, _ = m.forward(h, y, rng=rng)
        d = m.backward(h_out, None, d_n, h, rng)
        if p == 1.0:
            assert torch.equal(h_out, h) and not d.d_y.any()
        else:
            assert torch.equal(h_out, h + y.float()) and torch.equal(d.d_y, d.d_h.bfloat16())


def test_dropout_where_nothing_is_dropped():
    g = generator(3)
    x, res = rows_of(g, 33, 1001, BF16), rows_of(g, 33, 1001, BF16)
    for p, rng in ((0.4, None), (0.0, words(1, 2))):
        assert torch.equal(ep.dropout(x, p, rng), x)
        assert torch.equal(ep.dropout(x[:, :1000], p, rng, residual=res[:, :1000]), (x.float() + res.float()).bfloat16()[:, :1000])
    assert torch.equal(ep.dropout(x, 1.0, words(1, 2), residual=res), res) and not ep.dropout(x, 1.0, words(1, 2)).any()


def test_seed_step_and_site():
    """Each changes the mask; a step with a site is the step that many later."""
    x = torch.ones(64, 128, device="cuda")
    base = ep.dropout(x, 0.5, words(1, 10))
    for rng, site in ((words(2, 10), 0), (words(1 + 2 ** 32, 10), 0), (words(1, 11), 0), (words(1, 10 + 2 ** 32), 0), (words(1, 10), 1),
                      (words(1, 10), 2 ** 40)):
        assert (ep.dropout(x, 0.5, rng, site) != base).float().mean() > 0.4
    assert torch.equal(ep.dropout(x, 0.5, words(1, 4), 6), base)
    assert torch.equal(ep.dropout(x, 0.5, words(1, 2 ** 64 - 1), 11), base)          # modulo 2^64
    assert torch.equal(ep.dropout(x, 0.5, words(1, 11), -1), base)


def drop_check(T, H, dtype, p=0.3, pad=0, residual=False, first=0, site=2):
    g = generator(T + H)
    rng = words(77, 2 ** 63 + 5)

    def buffer():          # rows start `first` elements into an allocation
        return (torch.randn(T * (H + pad) + first, generator=g, device="cuda") * 2).to(dtype)[first:].view(T, H + pad)[:, :H]

    x, res, out = buffer(), buffer() if residual else None, buffer()
    around = out.as_strided((T, H + pad), (H + pad, 1))[:, H:].clone()
    got = ep.dropout(x, p, rng, site, residual=res, out=out)
    f = ref.factors(T, H, p, rng.tolist(), site)
    v, e = ref.dropped_sum(f64(x), f, f64(res) if residual else 0.0)
    near("y", got, v, e)
    assert got is out and torch.equal(out.as_strided((T, H + pad), (H + pad, 1))[:, H:], around), "written beside the rows"
    assert ((f64(got) == 0) == (f == 0))[f64(x) != 0].all() or residual
    assert torch.equal(ep.dropout(x, p, rng, site, residual=res), out)
    x_before = x.clone()
    if residual:
        assert ep.dropout(x, p, rng, site, residual=res, out=res) is res and torch.equal(res, out) and torch.equal(x, x_before)
    else:
        assert ep.dropout(x, p, rng, site, out=x) is x and torch.equal(x, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7), (3, 8), (5, 9), (1, 4096), (17, 1000), (777, 1001), (300, 31), (4000, 8), (70000, 3), (2, 100003)])
def test_dropout_sizes(T, H, dtype):
    drop_check(T, H, dtype)
    drop_check(T, H, dtype, residual=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,pad,first", [(1000, 8, 0), (1000, 3, 0), (64, 0, 1), (64, 64, 4), (1001, 7, 3), (24, 8, 8)])
def test_dropout_of_rows_that_lie_apart(H, pad, first, dtype):
    drop_check(70, H, dtype, pad=pad, first=first)
    drop_check(70, H, dtype, pad=pad, first=first, residual=True)


def test_dropout_of_more_than_2_to_the_31_elements():
    """The last rows of 2^18 + 3 rows of 8200 bf16 channels."""
    T, H, rng = 2 ** 18 + 3, 8200, words(3, 4)
    x = torch.ones(T, H, dtype=BF16, device="cuda")
    ep.dropout(x, 0.25, rng, out=x)
    rows = [0, 1, 2 ** 17, T - 2, T - 1]
    want = ref.factors(T, H, 0.25, rng.tolist(), 0, rows)
    assert np.array_equal(f64(x[torch.tensor(rows, device="cuda")]), f64(torch.from_numpy(want).to(BF16)))


def test_layer_norm_of_more_than_2_to_the_31_elements():
    T, H = 2 ** 17 + 5, 16384
    rows = [0, 151, 2 ** 17 - 1, 2 ** 17, T - 1]
    h_out, n, d, m = check(T, H, BF16, rows=rows)
    assert torch.isfinite(d.d_w).all() and torch.isfinite(d.d_b).all()


def test_one_mask_in_all_calls():
    """The norm's dropout, its gradient's and the function's are one."""
    T, H, p, site, rng = 70, 520, 0.4, 9, words(11, 12)
    one = torch.ones(T, H, dtype=BF16, device="cuda")
    mask = ep.dropout(one, p, rng, site) != 0
    m = ep.LayerNorm(T, H, p=p, site=site, weight=False, bias=False, train=True)
    h_out, _ = m.forward(torch.zeros_like(one), one, rng=rng)
    d = m.backward(h_out, None, torch.zeros_like(one), one, rng)
    assert torch.equal(h_out != 0, mask) and torch.equal(d.d_y != 0, mask) and torch.equal(d.d_y, ep.dropout(one, p, rng, site))


@pytest.mark.parametrize("H", [256, 520, 2056, 8200])
def test_in_place(H):
    g = generator(0)
    h, y, d_n, dh = rows_of(g, 700, H, F32), rows_of(g, 700, H, BF16), rows_of(g, 700, H, BF16), rows_of(g, 700, H, F32)
    m = ep.LayerNorm(700, H, F32, p=0.1, weight=False, bias=False, train=True)
    rng = words(1, 2)
    h_out, n = (t.clone() for t in m.forward(h, y, rng=rng))
    d_h = m.backward(h_out, None, d_n, dh, rng).d_h.clone()
    lib, stream = ep.load(), torch.cuda.current_stream().cuda_stream
    assert lib.ep_layer_norm(m._ref, h.data_ptr(), H, y.data_ptr(), H, None, None, rng.data_ptr(), h.data_ptr(), m.n.data_ptr(), None, None,
                             stream) == 0
    assert torch.equal(h, h_out) and torch.equal(m.n, n)
    assert lib.ep_layer_norm_backward(m._ref, h.data_ptr(), H, None, rng.data_ptr(), m.stats.data_ptr(), dh.data_ptr(), d_n.data_ptr(),
                                      dh.data_ptr(), None, None, None, m.workspace.data_ptr(), m.workspace_bytes, None, stream) == 0
    assert torch.equal(dh, d_h)


def test_no_rows():
    m = ep.LayerNorm(0, 64, p=0.1, train=True)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    m.forward(e, e, w, w, words(1, 2))
    d = m.backward(e, w, e, e, words(1, 2))
    assert not d.d_w.any() and not d.d_b.any() and d.d_h.shape == (0, 64)
    assert ep.dropout(e, 0.5, words(1, 2)).shape == (0, 64)


def test_same_bits_twice_and_on_another_stream():
    for T, H, dtype in ((900, 1000, BF16), (300, 7168, F32)):
        g = generator(0)
        h, y, d_n, dh = rows_of(g, T, H, dtype), rows_of(g, T, H, BF16), rows_of(g, T, H, BF16), rows_of(g, T, H, dtype)
        w, rng = torch.ones(H, device="cuda"), words(3, 4)

        def run(stream=None):
            m = ep.LayerNorm(T, H, dtype, p=0.1, train=True)
            torch.cuda.synchronize()
            h_out, n = m.forward(h, y, w, w, rng, stream=stream)
            d = m.backward(h_out, w, d_n, dh, rng, stream=stream)
            x = ep.dropout(h, 0.2, rng, stream=stream)
            torch.cuda.synchronize()
            return h_out, n, d.d_h, d.d_y, d.d_w, d.d_b, x
        a = run()
        for b in (run(), run(torch.cuda.Stream())):
            assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_captured_and_replayed_with_the_step_counted_up():
    T, H, p = 64, 512, 0.3
    g = generator(0)
    h, y, d_n = rows_of(g, T, H, BF16), rows_of(g, T, H, BF16), rows_of(g, T, H, BF16)
    w, rng = torch.ones(H, device="cuda"), words(21, 100)
    m, x = ep.LayerNorm(T, H, p=p, site=7, train=True), torch.empty_like(h)

    def step():
        h_out, _ = m.forward(h, y, w, w, rng)
        m.backward(h_out, w, d_n, h, rng)
        ep.dropout(y, p, rng, 8, out=x)
        rng[1] += 1

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        rng[1] = 100
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    seen = []
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        f = torch.from_numpy(ref.factors(T, H, p, (21, 100 + i), 7)).cuda()
        assert torch.equal(m.grads.d_y != 0, (f != 0) & (m.grads.d_h != 0))
        assert torch.equal(x, ep.dropout(y, p, words(21, 100 + i), 8))
        seen.append(x.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_gradients_by_differences():
    """The loss along a random direction, f32 stream: by central differences of step s the error is s^2 of third
    derivatives and bf16's rounding of n over s; both are far below 5 % here, which the directional derivative has to
    be within."""
    T, H, p, rng = 16, 64, 0.25, words(8, 9)
    g = generator(2)
    h, w, b = rows_of(g, T, H, F32), 1 + 0.1 * rows_of(g, 1, H, F32)[0], rows_of(g, 1, H, F32)[0]
    y, d_n, dh = rows_of(g, T, H, BF16), rows_of(g, T, H, BF16), rows_of(g, T, H, F32)
    m = ep.LayerNorm(T, H, F32, p=p, train=True)

    def loss(h, w, b):
        h_out, n = m.forward(h, y, w, b, rng)
        return (n.double() * d_n.double()).sum() + (h_out.double() * dh.double()).sum()

    loss(h, w, b)
    d = m.backward(m.h_out.clone(), w, d_n, dh, rng)
    s = 0.05
    for at, grad in ((0, d.d_h), (1, d.d_w), (2, d.d_b)):
        args = [h, w, b]
        way = grad / grad.norm()          # along the gradient: the derivative is its norm
        hi, lo = (loss(*(a + sign * s * way if i == at else a for i, a in enumerate(args))) for sign in (1, -1))
        assert abs((hi - lo) / (2 * s) / grad.double().norm() - 1) < 0.05, at


def test_refusals():
    m = ep.LayerNorm(4, 64, p=0.1, train=True)
    x, w, rng = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda"), words(1, 2)
    for bad in (dict(y=None), dict(w=None), dict(b=None), dict(h=x[:3]), dict(y=x.t().contiguous().t()), dict(w=w[:32])):
        with pytest.raises(ValueError):
            m.forward(**{**dict(h=x, y=x, w=w, b=w, rng=rng), **bad})
    for bad in (dict(h=x.float()), dict(y=x.float()), dict(w=w.double()), dict(rng=rng.int())):
        with pytest.raises(TypeError):
            m.forward(**{**dict(h=x, y=x, w=w, b=w, rng=rng), **bad})
    with pytest.raises(ValueError):
        m.forward(x, x, w, w, rng.repeat(2))
    with pytest.raises(ValueError):
        ep.LayerNorm(4, 64).backward(x, w, x)
    with pytest.raises(ValueError):
        ep.LayerNorm(4, 64, p=0.1, block=False)
    with pytest.raises(ep.EPError):
        m.backward(x, w, None)
    for bad in (dict(H=12), dict(eps=0.0), dict(p=1.5), dict(H=16392)):
        with pytest.raises(ep.EPError):
            ep.LayerNorm(**{**dict(T=4, H=64), **bad})
    with pytest.raises(TypeError):
        ep.LayerNorm(4, 64, torch.float16)
    with pytest.raises(TypeError):
        ep.dropout(x.half(), 0.1, rng)
    with pytest.raises(TypeError):
        ep.dropout(x, 0.1, rng, residual=x.float())
    with pytest.raises(TypeError):
        ep.dropout(x, 0.1, rng.int())
    with pytest.raises(ValueError):
        ep.dropout(x, 0.1, rng.cpu())
    with pytest.raises(ValueError):
        ep.dropout(x[0], 0.1, rng)
    with pytest.raises(ValueError):
        ep.dropout(x, 0.1, rng, out=x[:2])
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ep.EPError):
            ep.dropout(x, p, rng)
