"""The binding of the 8-bit cache refuses what is no tensor, on a machine without a GPU."""
import pytest
import torch

from sparse_attention_gemm_gb300 import ops


@pytest.mark.parametrize("bad", [None, [[0.0]], 3, torch.tensor(1.0, dtype=torch.bfloat16)])
def test_rows_that_are_no_rows(bad):
    cache, scale = torch.zeros(2, 4, 1, 32, dtype=torch.uint8), torch.ones(2, 1)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        ops.kv8_write(bad, cache, scale, cu)
    with pytest.raises((TypeError, ValueError)):
        ops.kv8_read(cache, scale, cu, 3, out=bad)
    with pytest.raises((TypeError, ValueError)):
        ops.sparse_attn_fwd_kv8(bad, cache, scale, cu, 0.1)
    with pytest.raises((TypeError, ValueError)):
        ops.kv8_write(torch.zeros(3, 1, 32, dtype=torch.bfloat16), bad, scale, cu)
