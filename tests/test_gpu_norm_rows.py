"""Gradients of ep_block_norm where every CTA has many rows: the slots of the
rows' sums, the ring's stages and the barriers' phases are all used again, and
sums over rows come from every CTA.  Bounds in norm_cases.
"""
import numpy as np
import pytest
import torch

import combine_ep_get_04_gb300 as ep
import norm_cases

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def check(T, H, dtype, gate, post, pre, scaled, d_h_out=True):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    inputs, grads = norm_cases.make(T, H, dtype, gate, post, pre, scaled, d_h_out)
    v, z = norm_cases.reference(inputs, grads)
    on = lambda d: {k: None if x is None else x.cuda() for k, x in d.items()}      # noqa: E731
    inputs, grads = on(inputs), on(grads)
    m = ep.BlockNorm(T, H, dtype, gate=gate, post=post, pre=pre, scaled=scaled, eps=norm_cases.EPS, train=True)
    h_out, n = m.forward(**inputs)
    d = m.backward(**inputs, **grads)
    torch.cuda.synchronize()
    assert int(m.err_flags) == 0
    got = dict(h_out=h_out, n=n, d_h=d.d_h, d_y=d.d_y, d_w_post=d.d_w_post, d_w_pre=d.d_w_pre, d_gate=d.d_gate, d_res_scale=d.d_res_scale)
    for name, x in got.items():
        if x is None:
            continue
        b = norm_cases.bound(name, v[name], z[name], T, H, gate, sms, x.dtype == BF16)
        off = np.abs(x.double().cpu().numpy() - v[name])
        assert (off <= b).all(), f"{name}: {(off > b).sum()} of {off.size} beyond the bound, worst {(off / b).max():.3g} of it"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,gate,post,pre,scaled,d_h_out", [
    (18300, 256, "channel", True, True, True, True),       # six CTAs an SM
    (16000, 512, "token", True, True, True, True),         # five
    (9200, 1024, "channel", True, True, True, True),       # three
    (6400, 1152, "token", True, True, True, True),         # two
    (4000, 4096, "channel", True, True, True, True),       # one, with two or three rows of lag
    (3301, 2600, "token", True, True, True, False),
    (3300, 2600, "channel", True, False, True, True),
    (3300, 2600, None, False, True, False, True),
    (2000, 7168, "channel", True, True, True, True),       # rows shared by two CTAs
    (1999, 7168, "token", False, True, True, False),
    (1000, 8200, "channel", True, True, True, True),       # by four
    (777, 16384, "token", True, True, True, True),
])
def test_gradients_of_many_rows(T, H, gate, post, pre, scaled, d_h_out, dtype):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T / norm_cases.clusters(T, H, sms)[0] >= 20
    check(T, H, dtype, gate, post, pre, scaled, d_h_out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,gate", [(1, 8, "channel"), (37, 1000, "channel"), (200, 264, "token"), (130, 1000, None), (333, 1024, "channel"),
                                      (64, 4096, "token"), (131, 7168, "channel"), (17, 8192, "token"), (2051, 2048, "token"),
                                      (4099, 64, "channel"), (6, 16384, "channel")])
def test_sums_over_few_rows(T, H, gate, dtype):
    check(T, H, dtype, gate, True, True, True)
