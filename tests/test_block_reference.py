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
