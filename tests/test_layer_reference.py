"""The plain implementations themselves: the generator's published vectors, and
gradients against differences."""
import numpy as np
import pytest

import layer_reference as ref


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_published_vectors_of_the_generator(counter, key, want):
    assert ref.philox(np.array([counter], dtype=np.uint64), key)[0].tolist() == list(want)


def test_a_mask_by_hand():
    """Element j of block i: half j % 2 of word j // 2 of the counter (i, 0, step + site, 0)."""
    f = ref.factors(3, 20, 0.3, (7 << 32 | 5, 2 ** 64 - 2), site=4)
    assert f.shape == (3, 20)
    limit = round(0.3 * 65536)
    for row, col in ((0, 0), (0, 19), (2, 9), (1, 16)):
        words = ref.philox(np.array([[row * 3 + col // 8, 0, 2, 0]], dtype=np.uint64), (5, 7))[0]
        bits = int(words[col % 8 // 2]) >> (16 * (col % 2)) & 0xFFFF
        assert f[row, col] == (65536 / (65536 - limit) if bits >= limit else 0.0)
    assert not ref.factors(2, 8, 1.0, (1, 2), 0).any() and (ref.factors(2, 8, 0.0, (1, 2), 0) == 1).all()


def test_share_that_stays():
    """10^6 independent elements: within five deviations, 5 sqrt(p (1 - p) / n)."""
    for p in (0.1, 0.5):
        f = ref.factors(1000, 1000, p, (123, 456), 0)
        assert abs((f == 0).mean() - p) < 5 * (p * (1 - p) / 1e6) ** 0.5 + 2.0 ** -17


@pytest.mark.parametrize("affine", [False, True])
def test_gradients_against_differences(affine):
    rng = np.random.default_rng(0)
    T, H, eps, step = 3, 16, 1e-5, 1e-6
    h, y, d_n, d_h = (rng.standard_normal((T, H)) for _ in range(4))
    w, b = (1 + 0.1 * rng.standard_normal(H), rng.standard_normal(H)) if affine else (None, None)
    f = ref.factors(T, H, 0.25, (9, 9), 1)

    def loss(h, y, w, b):
        x = h + y * f
        return (ref.layer_norm(x, w, b, eps)[0] * d_n).sum() + (x * d_h).sum()

    got = ref.layer_norm_gradients(ref.layer_norm(h + y * f, w, b, eps)[2], d_n, d_h, f)
    for name, at in (("d_h", 0), ("d_y", 1), ("d_w", 2), ("d_b", 3)):
        if at > 1 and not affine:
            continue
        args = [h, y, w, b]
        diff = np.zeros_like(args[at])
        for i in np.ndindex(diff.shape):
            d = []
            for sign in (1, -1):
                moved = args[at].copy()
                moved[i] += sign * step
                d.append(loss(*(moved if j == at else a for j, a in enumerate(args))))
            diff[i] = (d[0] - d[1]) / (2 * step)
        # central differences: third derivatives times step^2, and the losses' own rounding over the step
        assert np.abs(diff - got[name][0]).max() < 1e-7, name


def test_codes_by_hand():
    q, s = ref.quant_i8(np.array([[1.0, -0.5, 0.25, 0.0], [0.0, 0.0, 0.0, 0.0], [2.0, np.inf, 0.0, 1.0]]))
    assert q[0].tolist() == [127, -64, 32, 0] and q[1:].tolist() == [[0] * 4] * 2      # -63.5 to the even -64, 31.75 to 32
    assert s[0] == 1 / 127 and s[1] == 0 and np.isnan(s[2])
