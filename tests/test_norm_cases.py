"""The bounds on sums over rows tell a wrong sum from a right one (CPU)."""
import numpy as np
import pytest
import torch

import norm_cases


@pytest.mark.parametrize("T,H,gate", [(37, 1000, "channel"), (200, 264, "token"), (131, 7168, "channel"), (4099, 64, "channel"),
                                      (17, 8192, "channel"), (700, 2048, "token")])
@pytest.mark.parametrize("d_h_out", [True, False])
def test_a_lost_row_is_outside_the_bounds(T, H, gate, d_h_out):
    inputs, grads = norm_cases.make(T, H, torch.bfloat16, gate, True, True, True, d_h_out)
    v, z = norm_cases.reference(inputs, grads)
    one = {k: (x if x is None or k in ("w_post", "w_pre", "res_scale") or (k == "gate" and gate == "channel") else x[5:6])
           for k, x in inputs.items()}
    share, _ = norm_cases.reference(one, {k: None if x is None else x[5:6] for k, x in grads.items()})
    for name in ("d_res_scale", "d_w_post", "d_w_pre") + (("d_gate",) if gate == "channel" else ()):
        b = norm_cases.bound(name, v[name], z[name], T, H, gate, 152, False)
        # one column's share of a row may be next to nothing, but a lost row is lost to all columns
        assert np.mean(np.abs(v[name]) > b) > 0.95, f"{name}: 0 passes"
        assert np.mean(np.abs(share[name]) > b) > 0.5, f"{name}: a sum without one row passes"
