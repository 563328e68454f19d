"""Calls of the 8-bit block cache at the ends of their ranges."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, cu_from_lengths, dev, dev_bf16, f64
import kv8_ref as R
from sparse_attention_gemm_gb300 import ops
from sparse_attention_gemm_gb300 import workloads as W
from test_gpu_kv8 import Pages, cache_of, check_write, rows, same_codes
from test_gpu_kv8_peaked import check

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


@pytest.mark.parametrize("block", [2, 16, 256])
def test_packed_rows_of_several_sequences_share_blocks(block):
    """Neither table nor positions: row t of the batch is row t of the cache, and blocks hold the end of one sequence
    and the start of the next; the same codes as of one sequence, call after call, and read back in place."""
    rng = np.random.default_rng(91)
    cu = cu_from_lengths([33, 16, 0, 1, 15, 2, 200, 7])
    T = int(cu[-1]) + 5  # and padding
    n_blocks = (T + block - 1) // block + 1
    x = rows(rng, T, 2, 64, 6.0)
    codes, scale = cache_of(rng, n_blocks, block, 2, 64, -14, -4)
    want, ws = R.write(f64(x), codes, scale, np.array([0, cu[-1]], np.int32), None, None)
    src = dev_bf16(x)
    for _ in range(3):
        c, s = dev(codes), dev(scale)
        ops.kv8_write(src, c, s, dev(cu))
        assert np.array_equal(s.cpu().numpy(), ws) and same_codes(c.cpu().numpy(), want)
    got = ops.kv8_read(c, s, dev(cu), T)[:int(cu[-1])].float().cpu().numpy()
    v = R.read(want, ws, np.array([0, cu[-1]], np.int32), T, None, None, np.zeros((T, 2, 64), np.float32))[:int(cu[-1])]
    assert np.array_equal(got, torch.from_numpy(v).to(torch.bfloat16).float().numpy())


def test_batches_of_nearly_2_to_the_31_rows():
    """Rows counted up to the int32 limit, all but a few of them padding."""
    T = 2 ** 31 - 10
    if torch.cuda.mem_get_info()[0] < T * 32 + (8 << 30):
        pytest.skip("needs 72 GB of device memory")
    rng = np.random.default_rng(92)
    x = rows(rng, 5, 1, 16)
    big = torch.empty((T, 1, 16), dtype=torch.bfloat16, device=DEV)
    big[:5] = dev_bf16(x)
    big[T - 1] = 7.0
    cu = dev(cu_from_lengths([2, 3]))
    c = torch.full((8, 1, 1, 16), 9, dtype=torch.uint8, device=DEV)
    s = torch.full((8, 1), 9.0, device=DEV)
    ops.kv8_write(big, c, s, cu)
    ref, rs = R.write(f64(x), np.full((8, 1, 1, 16), 9, np.uint8), np.full((8, 1), 9.0, np.float32), np.array([0, 5], np.int32), None, None)
    assert same_codes(c.cpu().numpy(), ref) and np.array_equal(s.cpu().numpy(), rs)
    ops.kv8_read(c, s, cu, T, out=big)
    v = R.read(ref, rs, np.array([0, 5], np.int32), 5, None, None, np.zeros((5, 1, 16), np.float32))
    assert np.array_equal(big[:5].float().cpu().numpy(), torch.from_numpy(v).to(torch.bfloat16).float().numpy())
    assert bool((big[T - 1] == 7.0).all())
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,H,K,narrow", [(200, 64, 130, False), (20, 64, 2048, False), (300, 12, 130, True), (1, 64, 2048, True)])
def test_values_near_the_largest_float(T, H, K, narrow):
    """Mean values fit where the sum of a row's, or of a split's, weighted values would not."""
    rng = np.random.default_rng(93)
    n_blocks, block = 40, 16
    k, ks = cache_of(rng, n_blocks, block, 1, 256)
    v, _ = cache_of(rng, n_blocks, block, 1, 256)
    q = rows(rng, T, H, 256)
    idx = rng.integers(0, n_blocks * block, (T, K)).astype(np.int32)
    check((256, 256), q, k, ks, idx, 1 / 16, narrow=narrow, v8=v, v_scale=np.full((n_blocks, 1), 2.0 ** 118, np.float32))
