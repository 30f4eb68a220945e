"""ep_expert_i8 and ep_quant_i8 against plain 64-bit implementations.

Products: sums of codes' products are whole numbers, exact in fp32 below 2^24;
beyond, K terms of which each may be cut off at 2^-23 of the sum so far.  Three
more roundings for the scales, and one to bf16.  Codes: equal.
"""
import threading

import numpy as np
import pytest
import torch

import block_reference as bounds
import combine_ep_get_04_gb300 as ep
import layer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def make_weights(E, N, K, paired, g):
    rows = 2 * N if paired else N
    codes = torch.randint(-128, 128, (E, rows, K), generator=g, device="cuda", dtype=torch.int8)
    scales = (torch.rand(E, rows, generator=g, device="cuda") + 0.5) * (0.02 / K ** 0.5)
    return codes, scales


def make_rows(R, K, g):
    return (torch.randint(-128, 128, (R, K), generator=g, device="cuda", dtype=torch.int8),
            (torch.rand(R, generator=g, device="cuda") + 0.5) * 0.02)


def check(counts, N, K, paired=False, capacity=None, seed=0, max_rows=None, bare=False, edit=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    codes, scales = make_weights(E, N, K, paired, g)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    R = E * capacity if capacity else int(offsets[-1])
    x, xs = make_rows(R, K, g)
    if edit is not None:
        edit(codes, x)
    w = ep.I8Weights(codes, scales, paired)
    kept = [min(c, capacity) if capacity else c for c in counts]
    spans = [(e, e * capacity if capacity else int(offsets[e]), n) for e, n in enumerate(kept)]
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = dict(dtype=torch.int32, device="cuda")
    layout = {} if bare else dict(counts=torch.tensor(counts, **dev), offsets=torch.tensor(offsets, **dev))
    got = ep.expert_i8(x, xs, w, **layout, capacity=capacity, max_rows=max_rows, out=out, err_flags=err)
    torch.cuda.synchronize()
    assert got is out and int(err) == 0
    live, y, size = ref.expert_i8(x.cpu().numpy(), xs.double().cpu().numpy(), codes.cpu().numpy(), scales.double().cpu().numpy(), paired, spans)
    got = out.double().cpu().numpy()
    assert (got[~live] == 7.0).all(), "rows without a copy were written"
    b = bounds.bound(y, size, 2 * K if K * 128 * 128 > 2 ** 24 else 0, True)[live]
    off = np.abs(got - y)[live]
    assert (off <= b).all(), f"{(~(off <= b)).sum()} of {off.size} beyond the bound, worst {np.nanmax(off - b):.3g} past it"


@pytest.mark.parametrize("K", [16, 48, 64, 112, 128, 144, 1008, 4096, 7168])
@pytest.mark.parametrize("N", [8, 24, 64, 72, 128, 136, 1000])
@pytest.mark.parametrize("paired", [False, True])
def test_one_matrix(K, N, paired):
    for rows in (1, 3, 16):
        check([rows], N, K, paired, bare=rows == 3)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_rows_of_one_matrix(rows):
    check([rows], 72, 512, True)
    check([rows], 200, 272)


@pytest.mark.parametrize("K", [16, 48, 64, 112, 128, 144, 1008, 4096, 7168])
@pytest.mark.parametrize("paired", [False, True])
def test_wide_matrices(K, paired):
    """As much work as goes in tiles, in shares of K too."""
    N = 1032 if paired else 2056
    check([100], N, K, paired, bare=K == 64)
    check([3, 0, 60, 17], N, K, paired)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 159, 160, 161, 255, 256, 257, 300, 320, 321])
def test_rows_of_a_wide_matrix(rows):
    check([rows], 20008, 144)
    check([rows], 10008, 80, True)


@pytest.mark.parametrize("K", [2 ** 16, 2 ** 16 + 16])
def test_largest_sums_of_integers(K):
    """The longest sums that 32-bit integers hold, and the next, which go in fp32: all terms at an end, of either sign.
    The integers are exact up to three roundings (2^-24 each) and bf16's."""
    codes = torch.full((1, 16, K), -128, dtype=torch.int8, device="cuda")
    codes[:, 8:] = 127
    x = torch.full((4, K), -128, dtype=torch.int8, device="cuda")
    x[1::2] = 127
    w = ep.I8Weights(codes, torch.ones(1, 16, device="cuda"))
    got = ep.expert_i8(x, torch.ones(4, device="cuda"), w).double().cpu()
    want = x[:, :1].double().cpu() @ codes[0, :, :1].double().cpu().t() * K
    # in fp32 K terms, each cut off at 2^-23 of the sum at most
    bound = want.abs() * (2.0 ** -8 + 2.0 ** -22 + (0 if K <= 2 ** 16 else K * 2.0 ** -23))
    assert ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("capacity", [None, 12])
def test_experts_with_few_rows(capacity):
    counts = [3, 0, 1, 12, 0, 0, 5, 9, 8, 2, 1, 4, 0]
    check(counts, 136, 384, False, capacity, max_rows=sum(counts))
    check(counts, 72, 256, True, capacity, max_rows=sum(counts))


@pytest.mark.parametrize("capacity", [None, 40])
def test_uneven_experts(capacity):
    check([70, 0, 1, 2, 0, 3], 64, 256, capacity=capacity)
    check([0, 0, 129, 2], 64, 256, True, capacity=capacity)
    check([40, 40, 39, 33, 64], 64, 256, capacity=capacity)
    check([70, 0, 1, 2, 0, 3], 2600, 256, capacity=capacity)
    check([0, 0, 129, 2], 1304, 256, True, capacity=capacity)


def test_many_experts():
    rng = np.random.default_rng(4)
    check(rng.poisson(0.7, 1024).tolist(), 16, 128)
    check(rng.poisson(2.0, 333).tolist(), 16, 128, True)
    check(rng.poisson(2.0, 33).tolist(), 24, 144, False, capacity=3)


@pytest.mark.parametrize("counts,N,K,paired", [([1024], 4096, 512, True), ([700], 3000, 272, False), ([64, 70, 100, 65] * 4, 4096, 256, False),
                                               ([128, 0, 513, 64, 96, 1], 2048, 384, True), ([90] * 30, 1000, 640, False), ([140] * 9, 520, 1024, True)])
def test_prompt_batches(counts, N, K, paired):
    """Many tiles of rows an expert."""
    check(counts, N, K, paired, max_rows=sum(counts))


def test_many_row_blocks():
    check(np.random.default_rng(0).integers(0, 9, 240).tolist(), 2680, 208)
    check([1] * 8, 20008, 144)


@pytest.mark.parametrize("K,rows", [(128, 5), (1024, 40), (16384, 3), (16384, 200)])
@pytest.mark.parametrize("N", [72, 2056])
def test_largest_codes(K, rows, N):
    """All codes at an end: sums of up to 2^14 K, a power of two times a sum of powers of two, held exactly."""
    def edit(codes, x):
        codes.fill_(-128)
        x.fill_(-128)
        x[1::2] = 127
    check([rows], N, K, edit=edit)


@pytest.mark.parametrize("N,paired", [(2056, False), (1032, True)])
@pytest.mark.parametrize("K", [272, 7168])
def test_a_row_is_the_same_in_every_batch(N, paired, K):
    """Sums below 2^24 are exact in integers and in fp32, in whatever shares."""
    g = torch.Generator(device="cuda").manual_seed(0)
    codes, scales = make_weights(1, N, K, paired, g)
    w = ep.I8Weights(codes, scales, paired)
    x, xs = make_rows(700, K, g)
    xs *= 30 / K ** 0.5                                       # gates on both sides of 0, not all far out
    assert (x.float() @ codes[0].float().t()).abs().max() < 2 ** 24
    whole = ep.expert_i8(x, xs, w)
    for rows in (1, 5, 33, 100):
        assert torch.equal(ep.expert_i8(x[:rows], xs[:rows], w), whole[:rows]), rows


def test_long_sums():
    """Many steps of K, shared by clusters and not."""
    check([3], 16, 2 ** 18)
    check([40], 24, 2 ** 16 + 16, True)
    check([5, 0, 33, 2], 1000, 2 ** 14, max_rows=40)


@pytest.mark.parametrize("N", [16, 20008])
@pytest.mark.parametrize("K", [128, 4096])
def test_more_rows_than_promised(K, N):
    """All rows are computed, or what is not is left as it was and flagged."""
    g = torch.Generator(device="cuda").manual_seed(0)
    w = ep.I8Weights(*make_weights(3, N, K, False, g))
    x, xs = make_rows(12, K, g)
    o, err = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = ep.expert_i8(x, xs, w, offsets=o)
    out = ep.expert_i8(x, xs, w, offsets=o, max_rows=1, out=torch.full_like(want, 7.0), err_flags=err)
    assert int(err) in (0, ep.ERRF_CAPACITY)
    there = (out == want).all(1)
    assert there.all() if int(err) == 0 else (there[:4].all() and (out[4:] == 7).all())


@pytest.mark.parametrize("N", [72, 2056])
def test_rows_past_2_to_the_31_bytes(N):
    """The second expert of a capacity buffer, 2^31 bytes and more behind its start."""
    K, cap = 4096, 2 ** 19 + 40
    g = torch.Generator(device="cuda").manual_seed(0)
    w = ep.I8Weights(*make_weights(2, N, K, False, g))
    x, xs = torch.zeros(2 * cap, K, dtype=torch.int8, device="cuda"), torch.zeros(2 * cap, device="cuda")
    few, few_s = make_rows(2 * 30, K, g)
    at = torch.tensor([*range(30), *range(cap, cap + 30)], device="cuda")
    x[at], xs[at] = few, few_s
    counts = torch.tensor([30, 30], dtype=torch.int32, device="cuda")
    y = ep.expert_i8(x, xs, w, counts, capacity=cap, max_rows=60, out=torch.full((2 * cap, N), 7.0, dtype=torch.bfloat16, device="cuda"))
    want = ep.expert_i8(few, few_s, w, offsets=torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda"))
    assert torch.equal(y[at], want)
    y[at] = 7.0
    assert (y == 7.0).all()
    del x
    z = torch.zeros(2 * cap, K, dtype=torch.bfloat16, device="cuda")
    z[at] = torch.randn(60, K, generator=g, device="cuda").bfloat16()
    q, s = ep.quant_i8(z, counts, capacity=cap)
    want = ep.quant_i8(z[at])
    assert torch.equal(q[at], want[0]) and torch.equal(s[at], want[1])


def test_no_rows():
    check([0, 0, 0], 16, 128, capacity=4, max_rows=5)
    w = ep.I8Weights(*make_weights(3, 16, 128, False, torch.Generator(device="cuda").manual_seed(0)))
    i32 = dict(dtype=torch.int32, device="cuda")
    y = ep.expert_i8(torch.empty(0, 128, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"), w, torch.zeros(3, **i32), torch.zeros(4, **i32))
    assert y.shape == (0, 16)


@pytest.mark.parametrize("N", [64, 20008])
def test_a_row_without_a_scale_stays_alone(N):
    """What quantisation makes of a row that holds an infinity: NaN throughout, its neighbours untouched."""
    g = torch.Generator(device="cuda").manual_seed(0)
    w = ep.I8Weights(*make_weights(1, N, 208, False, g))
    x = torch.randn(6, 208, generator=g, device="cuda").bfloat16()
    clean = ep.expert_i8(*ep.quant_i8(x), w).clone()
    x[2, 100], x[4, 207] = float("inf"), float("nan")
    y = ep.expert_i8(*ep.quant_i8(x), w)
    assert torch.equal(y[[0, 1, 3, 5]], clean[[0, 1, 3, 5]]) and y[[2, 4]].isnan().all()


def test_same_bits_twice_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(0)
    for counts, N, K in (([1], 4096, 4096), ([4] * 40, 512, 1024), ([200] * 3, 640, 7168)):
        w = ep.I8Weights(*make_weights(len(counts), N, K, False, g))
        x, xs = make_rows(sum(counts), K, g)
        o = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        a = ep.expert_i8(x, xs, w, offsets=o).clone()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        b = ep.expert_i8(x, xs, w, offsets=o, stream=s)
        s.synchronize()
        assert torch.equal(a, b) and torch.equal(a, ep.expert_i8(x, xs, w, offsets=o))


def test_calls_of_several_threads():
    jobs, errors = [], []
    for i, (rows, K) in enumerate(((4, 128), (600, 4096), (1, 7168))):
        g = torch.Generator(device="cuda").manual_seed(i)
        w = ep.I8Weights(*make_weights(1, 264, K, False, g))
        x, xs = make_rows(rows, K, g)
        jobs.append((w, x, xs, ep.expert_i8(x, xs, w).clone()))
    torch.cuda.synchronize()

    def run(w, x, xs, want):
        stream, got = torch.cuda.Stream(), torch.full_like(want, 7.0)
        torch.cuda.synchronize()
        try:
            for _ in range(100):
                ep.expert_i8(x, xs, w, out=got, stream=stream)
            stream.synchronize()
            assert torch.equal(got, want)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("N", [16, 5200])
def test_bad_layouts_are_flagged_and_skipped(N):
    g = torch.Generator(device="cuda").manual_seed(0)
    w = ep.I8Weights(*make_weights(3, N, 128, False, g))
    x, xs = make_rows(12, 128, g)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(offsets, **more):
        out = torch.full((12, N), 7.0, dtype=torch.bfloat16, device="cuda")
        err.zero_()
        ep.expert_i8(x, xs, w, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out, err_flags=err, **more)
        return out, int(err)

    good, flags = run([0, 4, 8, 12])
    assert flags == 0
    out, flags = run([0, 4, 8, 13])
    assert flags == ep.ERRF_BAD_SLOT and torch.equal(out[:8], good[:8]) and (out[8:] == 7).all()
    out, flags = run([-2, 4, 8, 12])
    assert flags == ep.ERRF_BAD_SLOT and (out[:4] == 7).all() and torch.equal(out[4:], good[4:])
    out, flags = run([0, 12, 8, 12])              # falls: expert 1 has no rows
    assert flags == 0 and torch.equal(out[:4], good[:4])


def test_gates_of_any_size():
    """y = silu(gate) * up for gates and ups from one exact product each: an exponential, a quotient and three
    products, 24 u in all, beside the steps of subnormal numbers and the rounding to bf16."""
    gates = torch.linspace(-110, 110, 881, device="cuda")
    ups = torch.tensor([1.0, -3.0, 100.0], device="cuda")
    x = torch.zeros(gates.numel() * 3, 16, dtype=torch.int8, device="cuda")
    x[:, 0], x[:, 1] = 1, ups.repeat(gates.numel()).to(torch.int8)
    xs = gates.repeat_interleave(3).contiguous()
    codes = torch.zeros(1, 16, 16, dtype=torch.int8, device="cuda")
    codes[0, :8, 0], codes[0, 8:, 1] = 1, 1
    w = ep.I8Weights(codes, torch.ones(1, 16, device="cuda"), True)
    g = xs.double().cpu().numpy()[:, None]
    u = g * x[:, 1:2].double().cpu().numpy()                 # the row's scale is in both
    want = g / (1 + np.exp(-g)) * u
    bound = bounds.HALF_ULP_BF16 * np.abs(want) + 24 * bounds.EPS32 * np.abs(want) + (np.abs(g) + 1) * 2.0 ** -149 * np.abs(u) + 2.0 ** -133
    for rows in (5, 40, 300, x.shape[0]):
        for at in range(0, x.shape[0], rows):
            got = ep.expert_i8(x[at:at + rows], xs[at:at + rows], w).double().cpu().numpy()
            assert (np.abs(got - want[at:at + rows]) <= bound[at:at + rows]).all(), (rows, at)


def quant_check(R, K, held=None, seed=0, pad=0, edit=None, **layout):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(R, K + pad, generator=g, device="cuda") * torch.exp(2 * torch.randn(R, 1, generator=g, device="cuda"))).bfloat16()[:, :K]
    if edit is not None:
        edit(x)
    q, s = torch.full((R, K), 77, dtype=torch.int8, device="cuda"), torch.full((R,), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ep.quant_i8(x, out=q, scales=s, err_flags=err, **layout)
    assert got[0] is q and got[1] is s
    held = np.ones(R, bool) if held is None else held
    want_q, want_s = ref.quant_i8(x.double().cpu().numpy())
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(q[held], want_q[held])
    assert np.array_equal(s[held], want_s[held].astype(np.float32), equal_nan=True)     # one division, correctly rounded
    assert (q[~held] == 77).all() and (s[~held] == 7).all(), "rows without a copy were written"
    return int(err)


@pytest.mark.parametrize("K", [16, 48, 256, 272, 1008, 1024, 1040, 2048, 4096, 7168, 16384])
def test_quant_widths(K):
    quant_check(9, K)
    quant_check(3, K, pad=8)


def test_quant_of_many_rows():
    quant_check(40000, 64)
    quant_check(5000, 2048)


def test_quant_of_halves_zeros_and_the_unfit():
    def edit(x):
        x[0] = 0
        x[1] = 0
        x[1, 3] = -1.0
        x[1, 4] = 0.5                     # 63.5: to the even 64
        x[2, 5] = float("inf")
        x[3, 6] = float("nan")
        x[4, 0] = -float("inf")
        x[5] = 2.0 ** -133                # the smallest bf16
        x[6] = 3.3895e38                  # the largest
        x[7] = -0.0
        x[8] = torch.arange(64, device="cuda") * 2.0 ** -130
    quant_check(12, 64, edit=edit)
    # every quotient of two bf16 mantissas, two binades down
    for m in range(0, 128, 8):
        def fill(x):
            x[:, 0] = torch.arange(128, 128 + 8 * 16, 16, device="cuda")[: x.shape[0]] + m % 16
            x[:, 1:] = torch.linspace(-127, 127, 1023, device="cuda")[:, None].t()[:, : x.shape[1] - 1].repeat(x.shape[0], 1).bfloat16()
        quant_check(8, 1024, edit=fill)


@pytest.mark.parametrize("counts", [[3, 0, 1, 12, 0, 40], [0, 0], [5] * 300])
def test_quant_of_rows_in_use(counts):
    E, cap, i32 = len(counts), 10, dict(dtype=torch.int32, device="cuda")
    c, o = torch.tensor(counts, **i32), torch.tensor(np.concatenate([[0], np.cumsum(counts)]), **i32)
    held = np.concatenate([np.arange(cap) < n for n in counts])
    assert quant_check(E * cap, 80, held, counts=c, offsets=o, capacity=cap) == 0
    R = sum(counts) + 5
    assert quant_check(R, 80, np.arange(R) < sum(counts), counts=c, offsets=o) == 0
    if sum(counts) > 5:
        R = sum(counts) - 2
        assert quant_check(R, 80, offsets=o) == ep.ERRF_BAD_SLOT
    negative = torch.full_like(c, -3)
    assert quant_check(E * cap, 80, np.zeros(E * cap, bool), counts=negative, capacity=cap) == 0


def test_quant_on_streams_and_in_graphs():
    x = torch.randn(50, 512, device="cuda").bfloat16()
    want = [t.clone() for t in ep.quant_i8(x)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ep.quant_i8(x, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    w = ep.I8Weights(*make_weights(1, 72, 512, True, torch.Generator(device="cuda").manual_seed(0)), True)
    q, sc, y = torch.empty(50, 512, dtype=torch.int8, device="cuda"), torch.empty(50, device="cuda"), torch.empty(50, 72, dtype=torch.bfloat16, device="cuda")
    ep.expert_i8(*ep.quant_i8(x, out=q, scales=sc), w, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.expert_i8(*ep.quant_i8(x, out=q, scales=sc), w, out=y)
    for i in range(3):
        x.copy_(torch.randn(50, 512, device="cuda"))
        graph.replay()
        assert torch.equal(y, ep.expert_i8(*ep.quant_i8(x), w))


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(0)
    codes, scales = make_weights(2, 16, 128, False, g)
    w = ep.I8Weights(codes, scales)
    x, xs = make_rows(4, 128, g)
    o = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for error, call in (
            (ValueError, lambda: ep.expert_i8(x, xs, w)), (ValueError, lambda: ep.expert_i8(x[:, :64], xs, w, offsets=o)),
            (TypeError, lambda: ep.expert_i8(x.view(torch.uint8), xs, w, offsets=o)), (ValueError, lambda: ep.expert_i8(x, xs, w, offsets=o[:2])),
            (ValueError, lambda: ep.expert_i8(x, xs[:2], w, offsets=o)), (TypeError, lambda: ep.expert_i8(x, xs.half(), w, offsets=o)),
            (ep.EPError, lambda: ep.expert_i8(x, xs, w, counts=o[:2], capacity=3)), (ep.EPError, lambda: ep.expert_i8(x, xs, w, counts=o[:2])),
            (ValueError, lambda: ep.expert_i8(x, xs, w, offsets=o, out=torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"))),
            (ep.EPError, lambda: ep.I8Weights(codes[:, :, :120].contiguous(), scales)), (ep.EPError, lambda: ep.I8Weights(codes[:, :12].contiguous(), scales[:, :12].contiguous())),
            (ValueError, lambda: ep.I8Weights(codes, scales[:1])), (TypeError, lambda: ep.I8Weights(codes, scales.half())),
            (TypeError, lambda: ep.I8Weights(codes.view(torch.uint8), scales)), (ValueError, lambda: ep.I8Weights(codes[0], scales)),
            (TypeError, lambda: ep.quant_i8(x)), (ValueError, lambda: ep.quant_i8(x.bfloat16()[0])), (ep.EPError, lambda: ep.quant_i8(x.bfloat16()[:, :40].contiguous())),
            (ValueError, lambda: ep.quant_i8(x.bfloat16(), capacity=2)), (ValueError, lambda: ep.quant_i8(x.bfloat16(), counts=o[:2])),
            (ep.EPError, lambda: ep.quant_i8(x.bfloat16(), counts=o[:2], capacity=3)), (ep.EPError, lambda: ep.quant_i8(x.bfloat16()[:, 4:116][:, :112].as_strided((4, 112), (128, 1), 4)))):
        with pytest.raises(error):
            call()
