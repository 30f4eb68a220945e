"""Which dropouts of successive steps share their random numbers: those whose sums
of step and site are equal, and no two where steps and sites are counted as the
interface asks."""
import itertools

import numpy as np
import pytest
import torch

import layer_reference as ref

T, H, P, SEED, SITES, STEPS = 6, 1000, 0.5, 77, 5, 6

# step counted by more than the largest site; sites further apart than the steps reach; near the end of the numbers too
COUNTED = {"by the number of sites": [(n * SITES, i) for n in range(STEPS) for i in range(SITES)],
           "by 1, sites far apart": [(n, i << 32) for n in range(STEPS) for i in range(SITES)],
           "by 1 up to 2^32": [(2 ** 32 - STEPS + n, i << 32) for n in range(STEPS) for i in range(SITES)],
           "past 2^64": [((2 ** 64 - 10 + n * SITES) % 2 ** 64, i) for n in range(STEPS) for i in range(SITES)]}


def mask(step, site):
    return ref.factors(T, H, P, (SEED, step), site) != 0


@pytest.mark.parametrize("how", COUNTED)
def test_no_mask_is_used_twice(how):
    """Independent masks of n elements differ in half of them, five deviations sqrt(n) / 2 off at most."""
    masks = [mask(*at) for at in COUNTED[how]]
    n = T * H
    for a, b in itertools.combinations(masks, 2):
        assert abs((a != b).sum() - n / 2) < 5 * n ** 0.5 / 2


def test_steps_counted_by_one_walk_through_close_sites():
    for step, site in itertools.product(range(3), range(1, SITES)):
        assert np.array_equal(mask(step, site), mask(step + 1, site - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("how", COUNTED)
def test_the_kernels_masks(how):
    """The function's and the norm's, which are the reference's, bit by bit: a captured step that counts itself up."""
    import combine_ep_get_04_gb300 as ep
    at = COUNTED[how]
    signed = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v     # noqa: E731
    rng = torch.tensor([SEED, signed(at[0][0])], device="cuda")
    by = at[SITES][0] - at[0][0]
    sites = [site for _, site in at[:SITES]]
    ones = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    norms = [ep.LayerNorm(T, H, p=P, site=site, weight=False, bias=False) for site in sites]
    drops = [torch.empty_like(ones) for _ in sites]

    def step():
        for site, norm, out in zip(sites, norms, drops):
            norm.forward(torch.zeros_like(ones), ones, rng=rng)
            ep.dropout(ones, P, rng, site, out=out)
        rng[1] += by

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    rng[1] = signed(at[0][0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for n in range(STEPS):
        graph.replay()
        torch.cuda.synchronize()
        for (step_no, site), norm, out in zip(at[n * SITES:(n + 1) * SITES], norms, drops):
            want = torch.from_numpy(mask(step_no, site)).cuda()
            assert torch.equal(norm.h_out != 0, want) and torch.equal(out != 0, want), (n, site)
