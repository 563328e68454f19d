"""Calls of the 8-bit block cache at the ends of their ranges."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, cu_from_lengths, dev, dev_bf16, f64
import kv8_ref as R
from sparse_attention_gemm_gb300 import ops
from sparse_attention_gemm_gb300 import workloads as W
from test_gpu_kv8 import Pages, cache_of, check_write, rows, same_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    ops.device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0, "a kernel raised a device status flag"


@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127])
def test_append_to_a_block_of_the_largest_scale(scale):
    """Codes are e4m3(x / s) where 1 / s has no exact fp32 form too; infinity is +-448, NaN stays NaN."""
    rng = np.random.default_rng(90)
    g = Pages(rng, [3, 4], [2, 5], 16)
    v = W.bf16_bits_to_f32(rows(rng, g.T, 2, 32)).copy()
    v *= np.float32(2.0 ** 123)
    v[1, 0, :3], v[5, 1, :2] = [np.inf, -np.inf, np.nan], [3.3895314e38, -3.3895314e38]
    codes, old = cache_of(rng, g.n_blocks, 16, 2, 32)
    old[:] = scale
    check_write(g, W.f32_to_bf16_bits(v), codes, old, 2, 32)
