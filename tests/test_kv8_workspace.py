"""The workspace of the attention over the 8-bit cache, without a GPU: shapes
whose rows are split between CTAs need one, and are refused without it, with a
short one and with a misaligned one; others need none."""
import ctypes

import pytest

from sparse_attention_gemm_gb300 import build as dsa_build
from sparse_attention_gemm_gb300 import ops
from test_kv8_abi import FAKE, NULL, attn_args


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return ops.lib()


def args(shape, **kw):
    T, H, Hc, Dqk, Dv, K = shape
    v = dict(v8=FAKE, v_scale=FAKE) if Dqk == 256 else {}
    return attn_args(T=T, H=H, Hc=Hc, Dqk=Dqk, Dv=Dv, K=K, **v, **kw)


@pytest.mark.parametrize("shape", [(32, 128, 1, 576, 512, 2048), (20, 64, 1, 512, 512, 2048), (30, 64, 1, 256, 256, 1200),
                                   (1, 64, 1, 576, 512, 131072), (1, 16, 1, 576, 512, (1 << 20) + 1)])
def test_split_rows_are_refused_without_their_workspace(lib, shape):
    need = lib.dsa_sparse_attn_fwd_kv8_workspace_size(*shape)
    T, H, _, _, Dv, _ = shape
    assert need >= 2 * T * H * (Dv + 4) * 4  # two splits at least: a mean value and its sums each
    for bad in (dict(ws_bytes=need - 1), dict(ws_bytes=0), dict(workspace=NULL), dict(workspace=ctypes.c_void_p(4096 + 16)),
                dict(workspace=ctypes.c_void_p(4096 + 128))):
        assert lib.dsa_sparse_attn_fwd_kv8(*args(shape, **{"ws_bytes": need, **bad})) == ops.DSA_ERR_WORKSPACE, bad
        assert str(need).encode() in lib.dsa_last_error()


@pytest.mark.parametrize("shape", [(1, 64, 1, 576, 512, 2048), (3, 24, 2, 256, 256, 1027), (2048, 64, 1, 576, 512, 2048),
                                   (1024, 16, 1, 512, 512, 512), (1, 16, 1, 576, 512, 1 << 20)])
def test_other_shapes_need_none(lib, shape):
    assert lib.dsa_sparse_attn_fwd_kv8_workspace_size(*shape) == 0
