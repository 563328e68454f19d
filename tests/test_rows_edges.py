"""Norm, rotary positions and the 4-bit cache without a GPU: calls at the ends of what is allowed."""
import numpy as np
import pytest

from sparse_attention_gemm_gb300 import build as dsa_build
from sparse_attention_gemm_gb300 import ops


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return ops.lib()


@pytest.mark.parametrize("first", [1, 3, 6, 7, 40, 201, 202, 4096])
@pytest.mark.parametrize("R,base,slow", [(64, 10000.0, 1.0), (16, 10.0, 2.0), (128, 500000.0, 1.0)])
def test_angles_of_pairs_beyond_the_blend(lib, first, R, base, slow):
    """A pair that makes fewer than beta_slow turns over the first positions is slowed by the whole factor, the
    first pair too; one that makes more than beta_fast keeps its angle."""
    factor = 8.0
    f, _ = ops.rotary_inv_freq(R, base, "yarn", factor, first, beta_fast=32.0, beta_slow=slow, device="cpu")
    plain, _ = ops.rotary_inv_freq(R, base, device="cpu")
    turns = first * plain.numpy() / (2 * np.pi)
    few, many = turns < slow, turns > 32.0
    ratio = f.numpy() / plain.numpy()
    # (the blend runs from pair floor(lo) to pair ceil(hi): those outside turns' bounds are outside it)
    assert np.allclose(ratio[few], 1 / factor, rtol=1e-13) and np.allclose(ratio[many], 1, rtol=1e-13)
