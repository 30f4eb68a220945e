"""The 64-bit references of the block operators, checked on the CPU: their
gradients against central differences."""
import numpy as np
import pytest

import block_reference as ref


def differences(f, x, step=1e-5):
    """Central differences of the scalar f at every entry of x."""
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        down = f()
        x[i] = keep
        d[i] = (up - down) / (2 * step)
    return d


@pytest.mark.parametrize("gate_kind", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre,block", [(True, True, True), (False, True, True), (True, False, True), (False, True, False)])
def test_block_norm_gradients(gate_kind, post, pre, block):
    if not block and gate_kind != "none":
        return
    rng = np.random.default_rng(3)
    T, H, eps = 3, 8, 1e-6
    h, y = rng.standard_normal((T, H)), rng.standard_normal((T, H)) if block else None
    w_post = 1 + 0.1 * rng.standard_normal(H) if post else None
    w_pre = 1 + 0.1 * rng.standard_normal(H) if pre else None
    gate = {"none": None, "channel": rng.standard_normal(H), "token": rng.standard_normal((T, 1))}[gate_kind]
    a = np.array([0.8])
    d_h_out, d_n = rng.standard_normal((T, H)), rng.standard_normal((T, H)) if pre else None

    def loss():
        v, _ = ref.block_norm(h, y, w_post, w_pre, gate, a[0], eps)
        return (v["h_out"] * d_h_out).sum() + ((v["n"] * d_n).sum() if pre else 0.0)

    v, _ = ref.block_norm(h, y, w_post, w_pre, gate, a[0], eps, d_h_out, d_n)
    for name, x in (("d_h", h), ("d_y", y), ("d_w_post", w_post), ("d_w_pre", w_pre), ("d_gate", gate), ("d_res_scale", a)):
        if x is None:
            assert name not in v
            continue
        np.testing.assert_allclose(v[name].reshape(x.shape), differences(loss, x), rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_route_gradients(full, masked):
    """The choice and the counts are held while the logits move."""
    rng = np.random.default_rng(5)
    T, E, k, bounds = 7, 6, 3, np.array([0, 3, 3, 7])
    logits = rng.standard_normal((T, E))
    mask = (np.arange(T) != 4) if masked else None
    idx, live = ref.choose(logits.astype(np.float32), None, mask, k, 2, 1)
    assert (idx[:, 2] >= 0).sum() == live.sum()
    dw, dl = rng.standard_normal((T, k)), (1.3, 0.7)

    def loss():
        v, _ = ref.route(logits, idx, live, bounds, full, 0.5, 0.25)
        return (v["topk_w"] * dw).sum() + (v["losses"] * dl).sum()

    v, _ = ref.route(logits, idx, live, bounds, full, 0.5, 0.25, dw, dl)
    np.testing.assert_allclose(v["d_logits"], differences(loss, logits), rtol=1e-6, atol=1e-8)


def test_choice_by_hand():
    logits = np.array([[1, 3, 3, 2], [0, 0, 0, 0], [-np.inf, 5, -np.inf, np.nan], [-np.inf] * 4], np.float32)
    idx, live = ref.choose(logits, None, None, 2, 1, 1)
    assert idx.tolist() == [[1, 2], [0, 1], [1, -1], [-1, -1]] and live.tolist() == [True, True, True, False]
    idx, _ = ref.choose(logits, np.array([0, 0, 0, 2], np.float32), None, 2, 2, 1)
    assert idx.tolist() == [[3, 2], [3, 2], [1, -1], [-1, -1]]


def test_losses_by_hand():
    """Two tokens, two experts, both choose expert 0: c = (2, 0); equal logits
    give p = 1/2, so prob_sums = (1, 1) and the balance is E/(k n^2) * 2 = 1."""
    idx = np.zeros((2, 1), np.int64)
    v, _ = ref.route(np.zeros((2, 2)), idx, np.ones(2, bool), np.array([0, 2]), False, 1.0, 1.0)
    np.testing.assert_allclose(v["losses"], [1.0, np.log(2) ** 2])


def test_expert_w4_by_hand():
    codes = np.array([[[0x9f, 0x08], [0x71, 0xe8]]], np.uint8)        # codes 15 9 8 0 / 1 7 8 14
    scales = np.array([[[2.0], [0.5]]])
    x = np.array([[1.0, 2.0, 3.0, 1.0]])
    live, y, _ = ref.expert_w4(x, codes, scales, 32, False, [(0, 0, 1)])
    np.testing.assert_allclose(y, [[2 * (7 + 2 - 8), 0.5 * (-7 - 2 + 6)]])
    _, y, _ = ref.expert_w4(x, codes, scales, 32, True, [(0, 0, 1)])
    np.testing.assert_allclose(y, [[2 / (1 + np.exp(-2)) * -1.5]])
    assert live.all()
