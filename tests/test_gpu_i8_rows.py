"""ep_expert_i8 over as many rows as it accepts.  Rows are compared on the device,
a part at a time: sums of 16 products of codes are exact, two scales and bf16
are rounded (2 u and half a step), and every row of the buffer is looked at.
"""
import pytest
import torch

import combine_ep_get_04_gb300 as ep

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1
K, N = 16, 8


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


@pytest.fixture(scope="module")
def buffers():
    """The largest receive buffer: 34 GB of codes, 9 GB of scales and 34 GB of results."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 * 2 ** 30:
        pytest.skip("the largest buffers do not fit")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(MOST, K, dtype=torch.int8, device="cuda")
    scales = torch.empty(MOST, device="cuda")
    for a in range(0, MOST, 2 ** 26):
        n = min(2 ** 26, MOST - a)
        x[a:a + n] = torch.randint(-128, 128, (n, K), generator=g, device="cuda", dtype=torch.int8)
        scales[a:a + n] = torch.rand(n, generator=g, device="cuda") + 0.5
    yield x, scales, torch.empty(MOST, N, dtype=torch.bfloat16, device="cuda")
    del x, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E,max_rows", [(1, None), (300, 300)])
def test_the_largest_buffer(buffers, E, max_rows):
    """All rows of one expert; and all but 299 with the first of 300 experts, of
    which 300 rows were promised: tiles of 32, more than 2^26 of them."""
    x, scales, out = buffers
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    w_scales = torch.rand(E, N, generator=g, device="cuda") + 0.5
    w = ep.I8Weights(codes, w_scales)
    first = MOST - (E - 1)
    offsets = torch.tensor([0] + [first + e for e in range(E)], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out.fill_(float("nan"))
    ep.expert_i8(x, scales, w, offsets=offsets, max_rows=max_rows, out=out, err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    step = 2 ** 24
    for a in [*range(0, first, step), first]:
        b = min(a + step, first) if a < first else MOST
        if a == b:
            continue
        rows = x[a:b].float()
        sums = rows @ codes[0].float().t() if a < first else (rows[:, None, :] * codes[1:].float()).sum(2)
        of = w_scales[:1] if a < first else w_scales[1:]
        want = sums.double() * of.double() * scales[a:b, None].double()
        off = (out[a:b].double() - want).abs()
        # not <=: a row that was not written is a NaN
        bad = ~(off <= want.abs() * (2.0 ** -8 + 2.0 ** -22))
        assert not bad.any(), f"{int(bad.any(1).sum())} of rows {a} to {b}"
