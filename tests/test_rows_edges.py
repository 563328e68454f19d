"""Norm, rotary positions and the 4-bit cache without a GPU: calls at the ends of what is allowed."""
import numpy as np
import pytest

from sparse_attention_gemm_gb300 import build as dsa_build
from sparse_attention_gemm_gb300 import ops
from test_kv8_abi import FAKE, ODD, attn_args
from test_rows_abi import FAR, FAR2, rotary_args


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


@pytest.mark.parametrize("bad", [
    dict(x2=FAR2, y2=FAR), dict(x2=FAR, y2=FAR2), dict(x2=FAR2, y2=FAKE), dict(x2=FAKE, y=FAKE, y2=FAKE),
    dict(x2=FAKE, y=FAKE, y2=FAR2)])
def test_rotary_refuses_one_tensor_in_two_places(lib, bad):
    """y and y2 in one place, or either in the place of the other tensor's input."""
    a = rotary_args(**{"H2": 8, "x2_token": 512, "x2_head": 64, "y2_token": 512, "y2_head": 64, **bad})
    assert lib.dsa_rotary(*a) == ops.DSA_ERR_VALUE
    assert b"dsa_rotary" in lib.dsa_last_error()


@pytest.mark.parametrize("bad", [dict(kv_scale=ODD), dict(Dqk=256, Dv=256, v8=FAKE, v_scale=ODD),
                                 dict(Dqk=256, Dv=256, v8=FAKE, v_scale=FAKE, kv_scale=ODD)])
def test_cache_attention_refuses_misaligned_scales(lib, bad):
    """A row's scale bytes are copied in words of up to 16 bytes."""
    assert lib.dsa_sparse_attn_fwd_kv4(*attn_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"v_scale" in lib.dsa_last_error() and b"16-byte" in lib.dsa_last_error()
