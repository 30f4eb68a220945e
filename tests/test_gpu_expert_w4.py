"""ep_expert_w4 against a plain 64-bit implementation.

Bound: K products a sum, fp32 (the matrix instructions may cut off where a
fused multiply-add rounds, so two units of 2^-24 a term), one rounding to bf16.
"""
import threading

import numpy as np
import pytest
import torch

import block_reference as ref
import combine_ep_get_04_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def make_weights(E, N, K, group, paired, g):
    rows = 2 * N if paired else N
    codes = torch.randint(0, 256, (E, rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(E, rows, -(-K // group), generator=g, device="cuda") + 0.5) * 0.3 / K ** 0.5).bfloat16()
    return codes, scales


def make_rows(R, K, kind, g):
    x = torch.randn(R, K, generator=g, device="cuda")
    if kind == "bf16":
        x = x.bfloat16()
        return x, None, x.double().cpu().numpy()
    b = x.view(R, K // 128, 128)
    s = b.abs().amax(2).clamp_min(1e-4) / 448
    if kind == "ue8m0":
        e = torch.ceil(torch.log2(s))
        q = (b * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        value = q.double() * torch.exp2(e.double())[..., None]
        s = (e + 127).to(torch.uint8)
    else:
        q = (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        value = q.double() * s.double()[..., None]
    return q.view(R, K), s, value.view(R, K).cpu().numpy()


def check(counts, N, K, group=128, paired=False, kind="bf16", capacity=None, seed=0, max_rows=None, bare=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    codes, scales = make_weights(E, N, K, group, paired, g)
    w = ep.W4Weights(codes, scales, group, paired)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    R = E * capacity if capacity else int(offsets[-1])
    x, xs, value = make_rows(R, K, kind, g)
    kept = [min(c, capacity) if capacity else c for c in counts]
    spans = [(e, e * capacity if capacity else int(offsets[e]), n) for e, n in enumerate(kept)]
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = dict(dtype=torch.int32, device="cuda")
    layout = {} if bare else dict(counts=torch.tensor(counts, **dev), offsets=torch.tensor(offsets, **dev))
    got = ep.expert_w4(x, w, **layout, capacity=capacity, x_scales=xs, max_rows=max_rows, out=out, err_flags=err)
    torch.cuda.synchronize()
    assert got is out and int(err) == 0
    live, y, size = ref.expert_w4(value, codes.cpu().numpy(), scales.double().cpu().numpy(), group, paired, spans)
    got = out.double().cpu().numpy()
    assert (got[~live] == 7.0).all(), "rows without a copy were written"
    b = ref.bound(y, size, 2 * K, True)[live]
    off = np.abs(got - y)[live]
    assert (off <= b).all(), f"{(off > b).sum()} of {off.size} beyond the bound, worst {(off - b).max():.3g} past it"


@pytest.mark.parametrize("kind,K", [("bf16", 8), ("bf16", 72), ("bf16", 128), ("bf16", 200), ("bf16", 1000), ("bf16", 4096),
                                    ("fp8", 128), ("fp8", 640), ("ue8m0", 384), ("fp8", 7168)])
@pytest.mark.parametrize("N", [8, 24, 128, 136, 1000])
@pytest.mark.parametrize("paired", [False, True])
def test_one_matrix(kind, K, N, paired):
    for group, rows in ((32, 1), (64, 3), (128, 8)):
        check([rows], N, K, group, paired, kind, bare=rows == 3)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 130, 300])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "ue8m0"])
def test_rows_of_one_matrix(rows, kind):
    check([rows], 72, 512, 64, True, kind)
    check([rows], 200, 256, 128, False, kind)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "ue8m0"])
@pytest.mark.parametrize("capacity", [None, 12])
def test_experts_with_few_rows(group, kind, capacity):
    counts = [3, 0, 1, 12, 0, 0, 5, 9, 8, 2, 1, 4, 0]
    check(counts, 136, 384, group, False, kind, capacity, max_rows=sum(counts))
    check(counts, 72, 256, group, True, kind, capacity, max_rows=sum(counts))


@pytest.mark.parametrize("capacity", [None, 40])
def test_uneven_experts(capacity):
    """Shares of 8, 16 and more rows an expert take tiles of other sizes; one expert has most rows."""
    check([70, 0, 1, 2, 0, 3], 64, 256, capacity=capacity)
    check([0, 0, 129, 2], 64, 256, 64, True, "fp8", capacity=capacity)
    check([40, 40, 39, 33, 64], 64, 256, 32, capacity=capacity)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind,K", [("bf16", 264), ("bf16", 1000), ("fp8", 384), ("ue8m0", 640)])
@pytest.mark.parametrize("paired", [False, True])
def test_wide_tiles_in_many_ctas(group, kind, K, paired):
    check([0, 1, 30, 33, 17, 8, 24, 64, 25, 40, 12, 9, 31, 2, 16, 50, 7, 32, 13, 21, 26, 19], 2040, K, group, paired, kind)


def test_many_experts():
    rng = np.random.default_rng(4)
    check(rng.poisson(0.7, 1024).tolist(), 16, 128, 32)
    check(rng.poisson(2.0, 333).tolist(), 16, 128, 128, True, "fp8")
    check(rng.poisson(2.0, 33).tolist(), 24, 136, 64, False, capacity=3)


def test_no_rows():
    check([0, 0, 0], 16, 128, capacity=4, max_rows=5)
    w = ep.W4Weights(*make_weights(3, 16, 128, 128, False, torch.Generator(device="cuda").manual_seed(0)))
    i32 = dict(dtype=torch.int32, device="cuda")
    y = ep.expert_w4(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), w, torch.zeros(3, **i32), torch.zeros(4, **i32))
    assert y.shape == (0, 16)


def test_a_bad_row_stays_alone():
    """Infinities and NaN reach the outputs of their own row only, also past
    the end of a short last step of K."""
    g = torch.Generator(device="cuda").manual_seed(0)
    codes, scales = make_weights(1, 64, 200, 64, False, g)
    w = ep.W4Weights(codes, scales, 64)
    x = torch.randn(6, 200, generator=g, device="cuda").bfloat16()
    clean = ep.expert_w4(x, w).clone()
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[2, 100] = bad
        z[4, 199] = bad
        y = ep.expert_w4(z, w)
        rows = [0, 1, 3, 5]
        assert torch.equal(y[rows], clean[rows])
        for r, k in ((2, 100), (4, 199)):
            code = (codes[0, :, k // 2] >> (4 * (k % 2))) & 15
            finite = torch.isfinite(y[r].float())
            # inf times a zero weight is NaN too
            assert not finite.any(), (bad, r, code[finite])


def test_same_bits_twice_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(0)
    for counts, N, K in (([1], 4096, 4096), ([4] * 40, 512, 1024)):
        codes, scales = make_weights(len(counts), N, K, 128, False, g)
        w = ep.W4Weights(codes, scales)
        x = torch.randn(sum(counts), K, generator=g, device="cuda").bfloat16()
        o = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        a = ep.expert_w4(x, w, offsets=o).clone()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        b = ep.expert_w4(x, w, offsets=o, stream=s)
        s.synchronize()
        assert torch.equal(a, b) and torch.equal(a, ep.expert_w4(x, w, offsets=o))


def test_calls_of_several_threads():
    """Forms that need little and much shared memory, from two threads at once."""
    jobs, errors = [], []
    for i, K in enumerate((128, 16384)):
        g = torch.Generator(device="cuda").manual_seed(i)
        w = ep.W4Weights(*make_weights(1, 64, K, 128, False, g), 128, False)
        x, xs, _ = make_rows(4, K, "fp8", g)
        jobs.append((w, x, xs, ep.expert_w4(x, w, x_scales=xs).clone()))
    torch.cuda.synchronize()

    def run(w, x, xs, want):
        stream, got = torch.cuda.Stream(), torch.full_like(want, 7.0)
        torch.cuda.synchronize()
        try:
            for _ in range(300):
                ep.expert_w4(x, w, x_scales=xs, out=got, stream=stream)
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


def test_bad_layouts_are_flagged_and_skipped():
    g = torch.Generator(device="cuda").manual_seed(0)
    codes, scales = make_weights(3, 16, 128, 128, False, g)
    w = ep.W4Weights(codes, scales)
    x = torch.randn(12, 128, generator=g, device="cuda").bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(offsets, **more):
        out = torch.full((12, 16), 7.0, dtype=torch.bfloat16, device="cuda")
        err.zero_()
        ep.expert_w4(x, w, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out, err_flags=err, **more)
        return out, int(err)

    good, flags = run([0, 4, 8, 12])
    assert flags == 0
    out, flags = run([0, 4, 8, 13])
    assert flags == ep.ERRF_BAD_SLOT and torch.equal(out[:8], good[:8]) and (out[8:] == 7).all()
    out, flags = run([-2, 4, 8, 12])
    assert flags == ep.ERRF_BAD_SLOT and (out[:4] == 7).all() and torch.equal(out[4:], good[4:])
    out, flags = run([0, 12, 8, 12])              # falls: expert 1 has no rows
    assert flags == 0 and torch.equal(out[:4], good[:4])
    _, flags = run([0, 4, 8, 12], max_rows=1)     # room for one expert's tile
    assert flags == ep.ERRF_CAPACITY
    x, out = x[:12], None


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(0)
    codes, scales = make_weights(2, 16, 128, 128, False, g)
    w = ep.W4Weights(codes, scales)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ep.expert_w4(x, w)
    with pytest.raises(ValueError):
        ep.expert_w4(x[:, :64], w, offsets=o)
    with pytest.raises(TypeError):
        ep.expert_w4(x.float(), w, offsets=o)
    with pytest.raises(ValueError):
        ep.expert_w4(x, w, offsets=o[:2])
    with pytest.raises(TypeError):
        ep.expert_w4(x, w, offsets=o, x_scales=torch.ones(4, 1, device="cuda"))
    with pytest.raises(TypeError):
        ep.expert_w4(x.to(torch.float8_e4m3fn), w, offsets=o, x_scales=torch.ones(4, 1, device="cuda").half())
    with pytest.raises(ValueError):
        ep.expert_w4(x.to(torch.float8_e4m3fn), w, offsets=o, x_scales=torch.ones(4, 2, device="cuda"))
    with pytest.raises(ep.EPError):
        ep.expert_w4(x, w, counts=o[:2], capacity=3)      # needs 6 rows
    with pytest.raises(ep.EPError):
        ep.expert_w4(x, w, counts=o[:2])                   # packed rows need offsets
    with pytest.raises(ValueError):
        ep.expert_w4(x, w, offsets=o, out=torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"))
    for bad in (dict(group=96), dict(codes=codes[:, :, :62], scales=scales), dict(codes=codes[:, :12], scales=scales[:, :12])):
        with pytest.raises(ep.EPError):
            ep.W4Weights(**{**dict(codes=codes, scales=scales), **bad})
    with pytest.raises(ValueError):
        ep.W4Weights(codes, scales, group=64)
    with pytest.raises(TypeError):
        ep.W4Weights(codes, scales.float())
    odd = ep.W4Weights(codes[:, :, :60].contiguous(), scales)   # K = 120: no fp8 rows
    with pytest.raises(ep.EPError):
        ep.expert_w4(x.to(torch.float8_e4m3fn)[:, :120].contiguous(), odd, offsets=o, x_scales=torch.ones(4, 0, device="cuda"))


@pytest.mark.parametrize("K", [8, 40, 72, 200, 264, 1000])
@pytest.mark.parametrize("rows", [33, 50, 95])
def test_short_last_step_with_many_rows(K, rows):
    """Rows end inside a box of channels, and the last tile past the buffer's end."""
    check([rows], 72, K, 32, True)
    check([rows, 3, 40], 24, K, 128, False)
    check([rows, 0, 40], 24, K, 64, False, capacity=45)


def test_memory_of_a_call_on_another_stream():
    """What a call on a stream allocates is that stream's: it is not what other
    work may still be reading, nor handed out while the call runs; codes and
    scales may be dropped at once.  (Seen from the addresses: nothing here would
    read or write memory in use even if it were not so.)"""
    g = torch.Generator(device="cuda").manual_seed(0)
    codes, scales = make_weights(1, 4096, 1024, 128, False, g)
    kept = ep.W4Weights(codes, scales)
    x = torch.randn(256, 1024, generator=g, device="cuda").bfloat16()
    want = ep.expert_w4(x, kept).clone()
    s = torch.cuda.Stream()

    def block(nbytes):
        """A block of the current stream, freed: the next of its size there."""
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda").data_ptr()

    freed = block(want.numel() * 2)
    assert freed == torch.empty(want.numel() * 2, dtype=torch.uint8, device="cuda").data_ptr()
    y = ep.expert_w4(x, kept, stream=s)
    assert y.data_ptr() != freed
    s.synchronize()
    assert torch.equal(y, want)
    y = y.data_ptr()                                    # dropped: memory of s
    assert torch.empty(want.numel() * 2, dtype=torch.uint8, device="cuda").data_ptr() != y

    freed = block(kept.packed.numel())
    w = ep.W4Weights(codes, scales, stream=s)
    assert w.packed.data_ptr() != freed
    s.synchronize()
    assert torch.equal(w.packed, kept.packed)

    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mine = [t.clone() for t in (codes, scales)]
    places = [(t.data_ptr(), t.numel() * t.element_size()) for t in mine]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(600_000_000)                  # some 300 ms
    w = ep.W4Weights(*mine, stream=s)
    packed = torch.cuda.Event()
    packed.record(s)
    del mine
    again = [torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr() for _, n in places]
    assert not packed.query(), "the packing was over before the addresses were looked at"
    assert not {p for p, _ in places} & set(again)
    s.synchronize()
    assert torch.equal(w.packed, kept.packed)


def spread(E, few, seed=0):
    """Rows of E experts, up to `few` each, some none."""
    return np.random.default_rng(seed).integers(0, few + 1, E).tolist()


@pytest.mark.parametrize("counts,N,K,group,paired,kind", [
    (spread(240, 8), 2680, 200, 64, False, "bf16"),       # 2 steps of K, the second short: 21 row blocks, two to a CTA
    (spread(240, 8, 1), 2680, 264, 128, False, "bf16"),   # 3 steps: a stage of two and a short one
    (spread(240, 8, 2), 1336, 136, 32, True, "bf16"),
    (spread(240, 14, 3), 2680, 72, 64, False, "bf16"),    # one short step; some experts with two columns of tokens
    (spread(240, 8, 4), 2680, 384, 128, False, "fp8"),
    (spread(240, 8, 5), 1336, 128, 64, True, "ue8m0"),
    (spread(470, 8, 6), 2680, 136, 64, False, "bf16"),    # four to a CTA, the last CTA with one
    ([1] * 8, 78088, 136, 128, False, "bf16"),            # no more than 8 rows in all
    ([20, 3, 33, 9] * 20, 9752, 136, 128, False, "bf16"), # rows by tensor copies
])
def test_several_row_blocks_a_cta(counts, N, K, group, paired, kind):
    """At least 32 x 152 products of 128 weight rows, so that a CTA takes several
    and its ring runs on from one to the next, over a short last step of K too."""
    check(counts, N, K, group, paired, kind, max_rows=sum(counts))


def test_one_byte_rows_of_another_type_are_refused():
    g = torch.Generator(device="cuda").manual_seed(0)
    w = ep.W4Weights(*make_weights(1, 16, 128, 128, False, g))
    x, xs, _ = make_rows(4, 128, "fp8", g)
    want = ep.expert_w4(x, w, x_scales=xs)
    assert torch.equal(ep.expert_w4(x.view(torch.uint8), w, x_scales=xs), want)       # codes as bytes
    for other in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.int8, torch.bool):
        with pytest.raises(TypeError):
            ep.expert_w4(x.view(other), w, x_scales=xs)


def test_gates_of_any_size():
    """y = silu(gate) * up for exact gates and ups (one weight of 1 each): two
    units in the last place of an exponential, a quotient and a product, 16 x
    2^-24 in all, beside the steps of numbers below fp32's normal range and the
    rounding to bf16."""
    gates = torch.linspace(-110, 110, 881, device="cuda").bfloat16()
    ups = torch.tensor([1.0, -3.0, 1e30, 1e-6], device="cuda").bfloat16()
    x = torch.zeros(gates.numel() * 4, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = gates.repeat_interleave(4), ups.repeat(gates.numel())
    codes = torch.full((1, 16, 4), 0x88, dtype=torch.uint8, device="cuda")
    codes[0, :8, 0], codes[0, 8:, 0] = 0x89, 0x98
    w = ep.W4Weights(codes, torch.ones(1, 16, 1, dtype=torch.bfloat16, device="cuda"), 32, True)
    g, u = (x[:, i].double().cpu().numpy()[:, None] for i in (0, 1))
    want = g / (1 + np.exp(-g)) * u
    bound = ref.HALF_ULP_BF16 * np.abs(want) + 16 * ref.EPS32 * np.abs(want) + (np.abs(g) + 1) * 2.0 ** -149 * np.abs(u) + 2.0 ** -133
    for rows in (5, 8, 40, x.shape[0]):          # every form
        for at in range(0, x.shape[0], rows):
            got = ep.expert_w4(x[at:at + rows], w).double().cpu().numpy()
            off = np.abs(got - want[at:at + rows])
            assert (off <= bound[at:at + rows]).all(), (rows, g[at:at + rows][(off > bound[at:at + rows]).any(1)])


def test_rows_too_long_for_a_wide_tile():
    """A call whose own form holds a row's scales is answered, whatever the
    others could; one whose form does not is refused."""
    check([2], 16, 2 ** 18, 128, False, "fp8", bare=True)
    check([3, 0, 8, 7, 2], 24, 2 ** 18, 64, True, "ue8m0")
    g = torch.Generator(device="cuda").manual_seed(0)
    w = ep.W4Weights(*make_weights(1, 16, 2 ** 18, 128, False, g))
    x, xs, _ = make_rows(40, 2 ** 18, "fp8", g)
    with pytest.raises(ep.EPError):
        ep.expert_w4(x, w, x_scales=xs)


@pytest.mark.parametrize("counts,N,K,group,paired,kind", [
    ([1024], 4096, 512, 128, True, "fp8"), ([700], 3000, 264, 32, False, "bf16"), ([64, 70, 100, 65] * 4, 4096, 256, 128, False, "bf16"),
    ([128, 0, 513, 64, 96, 1], 2048, 384, 64, True, "ue8m0"), ([90] * 30, 1000, 640, 128, False, "fp8")])
def test_prompt_batches(counts, N, K, group, paired, kind):
    """Many tiles of rows an expert."""
    check(counts, N, K, group, paired, kind, max_rows=sum(counts))


@pytest.mark.parametrize("kind", ["fp8", "ue8m0"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 5, 8, 12, 40])
@pytest.mark.parametrize("large", [1, 4])
def test_small_channels_beside_a_large_one(rows, group, kind, large):
    """One or four channels of each 128 at e4m3's largest value, with zero weights,
    the others at multiples of its smallest, 2^-9.  Every product is a multiple of
    2^-9, and sums of them stay below 2^14 even where the codes are taken as 0 to
    15 and 8 times the row is taken off: 24 bits hold all of them exactly."""
    K, N = 640, 72
    g = torch.Generator(device="cuda").manual_seed(rows + group)
    codes, _ = make_weights(1, N, K, group, False, g)
    at = (torch.rand(K // 128, 128, generator=g, device="cuda").argsort(1)[:, :large] + 128 * torch.arange(K // 128, device="cuda")[:, None]).view(-1)
    for parity in (0, 1):                       # two channels of one byte one after the other
        here = at[at % 2 == parity]
        half = codes[0, :, here // 2]
        codes[0, :, here // 2] = (half & 0x0f) | 0x80 if parity else (half & 0xf0) | 8
    scales = torch.ones(1, N, K // group, dtype=torch.bfloat16, device="cuda")
    x = torch.randint(-7, 8, (rows, K), generator=g, device="cuda") * 2.0 ** -9
    x[:, at] = 448.0 * (1 - 2 * torch.randint(0, 2, (rows, at.numel()), generator=g, device="cuda"))
    x = x.to(torch.float8_e4m3fn)
    xs = torch.full((rows, K // 128), 127, dtype=torch.uint8, device="cuda") if kind == "ue8m0" else torch.ones(rows, K // 128, device="cuda")
    got = ep.expert_w4(x, ep.W4Weights(codes, scales, group), x_scales=xs).double().cpu().numpy()
    _, y, size = ref.expert_w4(x.double().cpu().numpy(), codes.cpu().numpy(), scales.double().cpu().numpy(), group, False, [(0, 0, rows)])
    b = ref.bound(y, size, 0, True)
    off = np.abs(got - y)
    assert (off <= b).all(), f"{(off > b).sum()} of {off.size} beyond the bound, worst {np.max(off / np.abs(y).mean()):.3g} of a mean result"
