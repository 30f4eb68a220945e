"""Calls of the layer-normed block's functions that are refused before any
tensor's address is taken, so this runs without a GPU."""
import pytest
import torch

import combine_ep_get_04_gb300 as ep


class Weights:                           # what expert_i8 looks at before the library
    E, N, K = 1, 8, 16


def test_counts_of_one_matrix_need_offsets():
    """Packed rows are found by offsets: counts alone would leave the rows behind the last one written."""
    meta = dict(device="meta")
    x, scales, counts = torch.empty(4, 16, dtype=torch.int8, **meta), torch.empty(4, **meta), torch.empty(1, dtype=torch.int32, **meta)
    with pytest.raises(ValueError, match="need the layout's offsets"):
        ep.expert_i8(x, scales, Weights, counts)
    with pytest.raises(ValueError, match="need the layout's offsets"):
        ep.quant_i8(x.bfloat16(), counts)
