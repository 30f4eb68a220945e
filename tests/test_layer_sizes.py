"""Sizes that the C structures hold in 32 bits: larger ones are refused, not cut
to their low words.  On tensors without memory, so this runs without a GPU."""
import pytest
import torch

import combine_ep_get_04_gb300 as ep
from combine_ep_get_04_gb300 import build as epbuild

PAST = 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def built():
    epbuild.build()


def meta(*shape, dtype=torch.int8):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("T,H,name", [(PAST + 8, 8, "T"), (2 ** 31, 8, "T"), (4, PAST + 8, "H")])
def test_layer_norm(T, H, name):
    with pytest.raises(ValueError, match=f"{name} = "):
        ep.LayerNorm(T, H, block=False, device="meta")


@pytest.mark.parametrize("E,rows,K,name", [(1, 8, PAST + 16, "K"), (1, PAST + 8, 16, "N"), (PAST + 1, 8, 16, "E")])
def test_weights(E, rows, K, name):
    with pytest.raises(ValueError, match=f"{name} = "):
        ep.I8Weights(meta(E, rows, K), meta(E, rows, dtype=torch.float32))
    if name == "N":
        with pytest.raises(ValueError, match="N = "):
            ep.I8Weights(meta(E, 2 * rows, K), meta(E, 2 * rows, dtype=torch.float32), paired=True)


def test_rows():
    counts, x = meta(1, dtype=torch.int32), meta(4, PAST + 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="K = "):
        ep.quant_i8(x)
    with pytest.raises(ValueError, match="capacity = "):
        ep.quant_i8(meta(4, 16, dtype=torch.bfloat16), counts, capacity=PAST + 4)
    with pytest.raises(ValueError, match="E = "):
        ep.quant_i8(meta(4, 16, dtype=torch.bfloat16), meta(PAST + 1, dtype=torch.int32), capacity=4)


def test_capacity_of_products():
    class Weights:                       # what expert_i8 looks at before the library
        E, N, K = 1, 8, 16

    with pytest.raises(ValueError, match="capacity = "):
        ep.expert_i8(meta(4, 16), meta(4, dtype=torch.float32), Weights, meta(1, dtype=torch.int32), capacity=PAST + 4)
