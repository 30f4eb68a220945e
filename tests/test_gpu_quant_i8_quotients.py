"""ep_quant_i8's codes over every quotient of bf16 magnitudes that leaves a code
other than 0: rows of all 128 mantissas of the largest magnitude, with every
mantissa below it in every binade, and the halves between two codes."""
import numpy as np
import pytest
import torch

import combine_ep_get_04_gb300 as ep
import layer_reference as ref

pytestmark = pytest.mark.gpu

BINADES = 9         # a quotient of 1 / 512 has code 0 (127 / 512 is below a half)
K = 2 * 128 * BINADES + 16


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    ep.load()


def rows(exponent):
    """[128, K]: the row's largest magnitude first, then +-m 2^-b of every mantissa m and binade b, times 2^exponent, as
    far as it is not larger (else 0), shuffled."""
    top = np.arange(128, 256, dtype=np.float64)[:, None]
    m = (np.arange(128, 256, dtype=np.float64)[None, :] * 2.0 ** -np.arange(BINADES)[:, None]).reshape(1, -1)
    x = np.zeros((128, K))
    x[:, 1:1 + m.size] = np.where(m <= top, m, 0.0)
    x[:, 1 + m.size:1 + 2 * m.size] = -np.where(m <= top, m, 0.0)
    x[:, 0] = top[:, 0] * np.where(np.arange(128) % 2, -1.0, 1.0)
    order = np.random.default_rng(exponent % 2 ** 16).permutation(K)
    return np.ascontiguousarray(x[:, order]) * 2.0 ** exponent


@pytest.mark.parametrize("exponent", [0, -7, 56, 57, 58, 63, 64, 100, 120, -70, -71, -72, -73, -100, -118, -120, -126, -130, -133])
def test_every_quotient(exponent):
    """Beside each border of the scaling (2^64 and 2^-64: a top of 128 to 255 times 2^57 and 2^-71), at the largest and
    the smallest numbers, where part of a row is no bf16 any more (those become 0)."""
    x = rows(exponent)
    t = torch.from_numpy(x).float().bfloat16()
    x = np.where(t.double().numpy() == x, x, 0.0)        # what bf16 has no number for
    t = torch.from_numpy(x).float().bfloat16()
    assert np.array_equal(t.double().numpy(), x)
    want, scales = ref.quant_i8(x)
    q, s = ep.quant_i8(t.cuda())
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(s.cpu().numpy(), scales.astype(np.float32))
    if exponent == 0:
        assert set(np.unique(want)) == set(range(-127, 128))


def test_every_half():
    """127 x / top is a half of an odd number where top is 127 x 2 / odd: top = 127 a, x = a (n + 1/2), for all such n."""
    x = np.zeros((12, 272))
    for i, a in enumerate((1.0, 2.0, -1.0, 2.0 ** 50, 2.0 ** -50, 2.0 ** 60, 2.0 ** -80, 2.0 ** 58, 2.0 ** -71, 2.0 ** 57, 2.0 ** -70, 2.0 ** 110)):
        x[i, 0] = 127 * a
        x[i, 1:128] = a * (np.arange(127) + 0.5)
        x[i, 128:255] = -a * (np.arange(127) + 0.5)
    t = torch.from_numpy(x).float().bfloat16()
    exact = t.double().numpy() == x
    x = np.where(exact, x, 0.0)
    assert exact[:, :128].all()                           # n + 1/2 below 127 has 8 bits
    want, _ = ref.quant_i8(x)
    assert (want[:, 1:128] == np.where(x[:, :1] != 0, np.sign(x[:, 1:128]) * 2 * np.round((np.arange(127) + 0.5) / 2), 0)).all()
    q, _ = ep.quant_i8(torch.from_numpy(x).float().bfloat16().cuda())
    assert np.array_equal(q.cpu().numpy(), want)
