"""ep_route and its gradient against a plain 64-bit implementation.

The choice, the counts and the live tokens are equal; what is computed is
within a bound taken from the formulas: exponentials of arguments up to
`reach` (their rounding grows with the argument), sums over E experts, over k
places and over the tokens (in runs, so their chains are n / 64 long and a few
more).
"""
import numpy as np
import pytest
import torch

import block_reference as ref
import combine_ep_get_04_gb300 as ep

pytestmark = pytest.mark.gpu

BALANCE, Z = 0.3, 0.2


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def make(T, E, dtype, seed=0, pad=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, E + pad, generator=g, device="cuda") * scale
    return x.to(dtype)[:, :E]


def check(logits, k, groups=1, topk_groups=1, full=False, bias=None, mask=None, bounds=None, d_w=True, d_losses=(0.7, -0.4)):
    T, E = logits.shape
    S = 1 if bounds is None else len(bounds) - 1
    seq = None if bounds is None else torch.tensor(bounds, dtype=torch.int32, device="cuda")
    r = ep.Router(T, E, k, groups, topk_groups, full, logits.dtype, S, BALANCE, Z, train=True)
    dw = torch.randn(T, k, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda") if d_w else None
    dl = None if d_losses is None else torch.tensor(d_losses, device="cuda")
    o = r.route(logits, bias, mask, seq)
    d = r.backward(logits, dw, dl, seq)
    torch.cuda.synchronize()
    l32 = logits.float().cpu().numpy()
    idx, live = ref.choose(l32, None if bias is None else bias.cpu().numpy(), None if mask is None else mask.cpu().numpy(), k, groups,
                           topk_groups)
    l64 = l32.astype(np.float64)
    v, z = ref.route(l64, idx, live, np.array([0, T] if bounds is None else bounds), full, BALANCE, Z,
                     None if dw is None else dw.double().cpu().numpy(), dl.double().cpu().numpy() if dl is not None else (0.0, 0.0))
    np.testing.assert_array_equal(o.topk_idx.cpu().numpy(), idx)
    np.testing.assert_array_equal(o.counts.cpu().numpy(), v["counts"])
    np.testing.assert_array_equal(o.seq_tokens.cpu().numpy(), v["seq_tokens"])
    assert int(o.err_flags) == 0
    # arguments of exponentials that do not underflow, and the largest logits themselves
    tops = l64[live].max(1, keepdims=True) if live.any() else np.zeros((1, 1))
    reach = float(np.abs(tops).max() + min(104.0, np.max(tops - l64[live], initial=0.0)))
    for name, x in (("topk_w", o.topk_w), ("lse", o.lse), ("prob_sums", o.prob_sums), ("losses", o.losses), ("d_logits", d)):
        terms = 128 + 8 * reach + E / 16 + k + (T / 64 if name in ("prob_sums", "losses", "d_logits") else 0)
        got, want = x.double().cpu().numpy(), v[name]
        if name == "lse":
            np.testing.assert_array_equal(got == -np.inf, ~live)
            got, want, size = got[live], want[live], z[name][live]
        else:
            size = z[name]
        b = ref.bound(want, size, terms, x.dtype == torch.bfloat16) + 1e-37   # where probabilities underflow
        off = np.abs(got - want)
        assert (off <= b).all(), f"{name}: {(off > b).sum()} of {off.size} beyond the bound, worst {(off / b).max():.3g} of it"
    serve = ep.Router(T, E, k, groups, topk_groups, full, logits.dtype)
    s = serve.route(logits, bias, mask)
    assert torch.equal(s.topk_idx, o.topk_idx) and torch.equal(s.topk_w, o.topk_w) and s.losses is None
    return o, d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (2, 3, 2), (5, 31, 4), (9, 32, 32), (17, 33, 5), (100, 60, 4), (77, 64, 8),
                                   (40, 65, 6), (130, 128, 8), (33, 160, 6), (128, 256, 8), (31, 257, 3), (20, 512, 10),
                                   (19, 1000, 8), (25, 1024, 32)])
def test_sizes(T, E, k, dtype):
    check(make(T, E, dtype, seed=E), k)
    check(make(T, E, dtype, seed=E + 1), k, full=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(128, 8, 4, 8), (256, 8, 4, 8), (60, 4, 2, 5), (96, 32, 3, 8), (64, 2, 1, 32),
                                                    (1024, 16, 5, 8), (32, 32, 4, 8)])
def test_groups(E, groups, topk_groups, k, dtype):
    """k may exceed what the groups hold: (32, 32, 4, 8) leaves four places empty."""
    check(make(200, E, dtype, seed=E), k, groups, topk_groups)


@pytest.mark.parametrize("T", [8, 4864, 5000, 9729, 40000])
def test_runs_of_more_tokens(T):
    check(make(T, 64, torch.float32, seed=T), 4)
    check(make(T, 24, torch.bfloat16, seed=T), 4, bounds=[0, 1, 3, 3, T // 2, T, T])


@pytest.mark.parametrize("bounds", [[0, 0, 100], [0, 100, 100], [0, 0, 0, 100, 100], [0, 8, 16, 24, 100], [0, 1, 2, 3, 4, 5, 6, 100],
                                    list(range(101))])
def test_sequences(bounds):
    check(make(100, 48, torch.float32), 3, bounds=bounds)


def test_ties_go_to_the_lower_index():
    x = torch.zeros(40, 300, device="cuda")
    x[1::2, 100:] = 1.0
    x[2, :] = -0.0
    x[3, ::2] = 0.0
    x[3, 1::2] = -0.0
    o, _ = check(x, 7, full=True)
    assert o.topk_idx[0].tolist() == list(range(7)) and o.topk_idx[1].tolist() == list(range(100, 107))
    assert o.topk_idx[2].tolist() == list(range(7)) and o.topk_idx[3].tolist() == list(range(7))
    check(torch.randint(-2, 3, (200, 128), device="cuda").float(), 8, 8, 3)
    check(torch.randint(-2, 3, (200, 160), device="cuda").bfloat16(), 8)


def test_bias_shifts_the_choice_alone():
    x = make(50, 64, torch.float32)
    bias = torch.linspace(2, -2, 64, device="cuda")
    o, _ = check(x, 6, bias=bias)
    c, _ = check(x, 6)
    assert not torch.equal(o.topk_idx, c.topk_idx)
    check(x.bfloat16(), 6, 4, 2, bias=bias)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
def test_masked_tokens_and_experts(full, groups, topk_groups):
    x = make(300, 64, torch.float32)
    x[::3] = torch.where(torch.rand(100, 64, device="cuda") < 0.7, float("-inf"), x[::3])
    x[5] = float("-inf")                         # nothing to choose
    x[7, 3:] = float("-inf")                     # less than k
    x[8, 4:] = torch.finfo(torch.float32).min    # the type's lowest value is a number like others
    mask = (torch.rand(300, device="cuda") < 0.8).to(torch.uint8)
    mask[[5, 7, 8]] = 1
    mask[[10, 11, 12]] = 0
    x[10], x[11], x[12, 3] = float("nan"), float("inf"), float("-inf")   # whatever a masked token holds
    o, d = check(x, 8, groups, topk_groups, full, mask=mask, bounds=[0, 50, 150, 300])
    assert o.topk_idx[5].tolist() == [-1] * 8 and not d[5].any() and not d[10].any() and not d[11].any()
    check(x, 8, groups, topk_groups, full, mask=mask.bool())


def test_no_live_token():
    mask = torch.zeros(30, dtype=torch.uint8, device="cuda")
    o, d = check(make(30, 16, torch.float32), 2, mask=mask)
    assert not o.losses.any() and not d.any() and not o.topk_w.any()
    check(make(30, 16, torch.bfloat16), 2, mask=mask, bounds=[0, 10, 30])


def test_large_logits():
    check(make(64, 128, torch.float32, scale=60.0), 8)
    check(make(64, 128, torch.float32, scale=60.0) + 1000.0, 8, full=True)


def test_nan_stays_in_its_row_and_is_not_chosen():
    x = make(40, 64, torch.float32)
    r = ep.Router(40, 64, 4, train=True, full_softmax=True)
    before = r.route(x).topk_idx.clone()
    x[9, 20] = float("nan")
    o = r.route(x)
    rows = [t for t in range(40) if t != 9]
    assert torch.equal(o.topk_idx[rows], before[rows]) and 20 not in o.topk_idx[9].tolist()
    assert torch.isnan(o.topk_w[9]).all() and not torch.isnan(o.topk_w[rows]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_further_apart_and_odd_addresses(dtype):
    check(make(50, 61, dtype, pad=3), 5)
    flat = torch.randn(50 * 64 + 1, device="cuda").to(dtype)
    check(flat[1:].view(50, 64)[:, :63], 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 0), (2, 2), (0, 1), (0, 4)])
@pytest.mark.parametrize("E,groups,topk_groups", [(256, 1, 1), (256, 8, 4), (128, 32, 5), (160, 8, 3), (512, 8, 2), (1024, 2, 1), (56, 7, 2)])
def test_groups_and_rows_at_any_place(E, groups, topk_groups, pad, shift, dtype):
    """Groups of whole lanes and others, rows that wide accesses can and cannot read."""
    flat = make(1, 40 * (E + pad) + shift, dtype, seed=E + pad)[0]
    x = flat[shift:].view(40, E + pad)[:, :E]
    check(x, 8, groups, topk_groups, bias=torch.linspace(-0.1, 0.1, E, device="cuda"))


def test_gradient_parts():
    x = make(60, 48, torch.float32)
    _, d = check(x, 4, d_w=False, d_losses=None)
    assert not d.any()
    check(x, 4, d_w=False)
    check(x, 4, d_losses=None)
    check(x, 4, full=True, d_losses=None)


def test_same_bits_twice_and_on_another_stream():
    x = make(20000, 96, torch.float32)
    dw, dl = torch.randn(20000, 6, device="cuda"), torch.ones(2, device="cuda")
    seq = torch.tensor([0, 123, 9000, 20000], dtype=torch.int32, device="cuda")
    r = ep.Router(20000, 96, 6, num_seqs=3, balance_coef=1.0, z_coef=1.0, train=True)
    torch.cuda.synchronize()

    def run(stream=None):
        o = r.route(x, seq_offsets=seq, stream=stream)
        d = r.backward(x, dw, dl, seq, stream=stream)
        torch.cuda.synchronize()
        return [t.clone() for t in (o.topk_idx, o.topk_w, o.lse, o.counts, o.prob_sums, o.losses, d)]

    a = run()
    for b in (run(), run(torch.cuda.Stream())):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_bad_sequences_are_flagged():
    x = make(64, 16, torch.float32)
    r = ep.Router(64, 16, 2, num_seqs=2, balance_coef=1.0, train=True)
    for bad in ([0, 70, 64], [1, 10, 64], [0, 10, 63], [0, -5, 64], [0, 2 ** 31 - 1, -2 ** 31]):
        r.out.err_flags.zero_()
        r.route(x, seq_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert int(r.out.err_flags) == ep.ERRF_BAD_SEQ, bad


def test_no_tokens():
    r = ep.Router(0, 16, 2, balance_coef=1.0, z_coef=1.0, train=True)
    x = torch.empty(0, 16, device="cuda")
    o = r.route(x)
    assert not o.losses.any() and not o.counts.any() and not o.prob_sums.any() and not o.seq_tokens.any()
    assert r.backward(x, torch.empty(0, 2, device="cuda"), torch.ones(2, device="cuda")).shape == (0, 16)


def test_refusals():
    r = ep.Router(8, 16, 2, num_seqs=2, train=True)
    x, seq = make(8, 16, torch.float32), torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        r.route(x)
    with pytest.raises(TypeError):
        r.route(x.bfloat16(), seq_offsets=seq)
    with pytest.raises(ValueError):
        r.route(x[:, :8], seq_offsets=seq)
    with pytest.raises(ValueError):
        r.route(x.t().contiguous().t(), seq_offsets=seq)
    with pytest.raises(TypeError):
        r.route(x, seq_offsets=seq.long())
    with pytest.raises(ValueError):
        r.route(x, token_mask=torch.ones(7, dtype=torch.uint8, device="cuda"), seq_offsets=seq)
    with pytest.raises(ValueError):
        ep.Router(8, 16, 2).backward(x, None, None)
    for bad in (dict(E=1025), dict(k=17), dict(k=0), dict(groups=3), dict(groups=16, topk_groups=17), dict(num_seqs=0), dict(T=-1)):
        with pytest.raises((ep.EPError, RuntimeError)):
            ep.Router(**{**dict(T=8, E=16, k=2), **bad})


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (300, 32), (1024, 20)])
def test_logits_that_differ_in_their_last_bits(E, k, bias):
    """Neighbours that agree in all but their lowest bits, in stretches of a few
    and of more than a warp can hold, in any order of the experts."""
    g = torch.Generator(device="cuda").manual_seed(E + k)
    for width in (2, 5, 40, E):
        step = torch.rand(64, E, generator=g, device="cuda").argsort(1)             # a permutation in each row
        x = 1.0 + (step // width).float() * 0.01 + (step % width).float() * 2.0 ** -23
        b = torch.zeros(E, device="cuda") if bias else None
        check(x, k, bias=b)
        check(-x, k, bias=b)
        if E % 4 == 0:
            check(x, k, 4, 2, bias=b)


def test_the_largest_batch():
    """2^31 - 1 tokens of one expert: token numbers past the end of the last run
    do not fit a signed 32-bit number.  21 GB, with the losses and gradient 35."""
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB")
    x = torch.full((T, 1), 0.5, dtype=torch.bfloat16, device="cuda")

    def everywhere(t, want):
        flat = t.view(-1)
        return all(bool((part == want).all()) for part in flat.split(2 ** 28))

    serve = ep.Router(T, 1, 1, dtype=torch.bfloat16)
    serve.out.topk_idx.fill_(7)
    o = serve.route(x)
    assert everywhere(o.topk_idx, 0) and everywhere(o.topk_w, 1.0)
    del serve, o
    r = ep.Router(T, 1, 1, dtype=torch.bfloat16, balance_coef=1.0, z_coef=1.0, train=True)
    r.out.topk_idx.fill_(7)
    r.d_logits.fill_(7)
    o = r.route(x)
    assert everywhere(o.topk_idx, 0) and everywhere(o.topk_w, 1.0) and everywhere(o.lse, 0.5)
    assert o.counts.item() == T and o.seq_tokens.tolist() == [T, T, 1]
    # sums of 2^31 terms in runs of 256: chains of 256, 2^18 (a warp's runs) and 32 additions
    bound = (256 + 2 ** 18 + 32) * ref.EPS32
    assert abs(o.prob_sums.item() / T - 1) <= bound
    assert abs(o.losses[0].item() - 1) <= 2 * bound and abs(o.losses[1].item() / 0.25 - 1) <= bound
    # the probability is 1 and counts cancel: 2 lse / n of the z loss is left
    d = r.backward(x, None, torch.tensor([1.0, float(T)], device="cuda"))
    assert everywhere(d, 1.0)
    del r, o, d, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("E", [48, 128, 256, 512, 1000])
def test_small_probabilities_are_as_close_as_large_ones(E, full):
    """One expert far above the rest, by whole numbers from 24 to 80, so that each
    argument of an exponential is exact and the sum is 1 to within 2^-24: what
    is left of a probability's error is that of the exponential (at most two units
    in its last place, 4 x 2^-24) and of some roundings, at every size of the
    argument: 16 x 2^-24 for a probability, 24 x 2^-24 for a gradient."""
    T, k = 60, 4
    g = torch.Generator(device="cuda").manual_seed(E)
    x = -torch.randint(24 + (E > 300), 81, (T, E), generator=g, device="cuda").float()
    top = torch.randint(0, E, (T,), generator=g, device="cuda")
    x[torch.arange(T), top] = 0.0
    bounds = list(range(T + 1))                         # each token its own sequence: prob_sums are probabilities
    seq = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    r = ep.Router(T, E, k, full_softmax=full, num_seqs=T, balance_coef=BALANCE, z_coef=Z, train=True)
    dl = torch.tensor([0.7, 0.0], device="cuda")
    o = r.route(x, seq_offsets=seq)
    d = r.backward(x, None, dl, seq).double().cpu().numpy()
    idx, live = ref.choose(x.cpu().numpy(), None, None, k, 1, 1)
    np.testing.assert_array_equal(o.topk_idx.cpu().numpy(), idx)
    v, z = ref.route(x.double().cpu().numpy(), idx, live, np.array(bounds), full, BALANCE, Z, None, dl.double().cpu().numpy())
    p = v["prob_sums"]
    assert (p < 1e-30).sum() > T                        # down to exp(-80)
    for name, got, size, units in (("prob_sums", o.prob_sums.double().cpu().numpy(), p, 16), ("d_logits", d, z["d_logits"], 24)):
        off = np.abs(got - v[name]) / (units * ref.EPS32 * size)
        assert (off <= 1).all(), f"{name}: {(off > 1).sum()} of {off.size} beyond the bound, worst {off.max():.3g} of it"
