"""The 8-bit cache calls without a GPU: refusals of bad arguments before
anything is launched, and the tests' own 64-bit definitions against torch's
E4M3 conversion."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_ref as R
from sparse_attention_gemm_gb300 import build as dsa_build
from sparse_attention_gemm_gb300 import ops

NULL = None
FAKE = ctypes.c_void_p(4096)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return ops.lib()


def write_args(**kw):
    a = dict(src=FAKE, cu=FAKE, pos=NULL, table=NULL, n_seqs=2, T=8, Hc=1, D=576, block=64, n_blocks=10, max_blocks=0,
             cache=FAKE, scale=FAKE, stream=NULL)
    a.update(kw)
    return list(a.values())


def read_args(**kw):
    a = dict(cache=FAKE, scale=FAKE, cu=FAKE, pos=NULL, table=NULL, n_seqs=2, T=8, Hc=1, D=576, block=64, n_blocks=10,
             max_blocks=0, out=FAKE, stream=NULL)
    a.update(kw)
    return list(a.values())


def attn_args(**kw):
    a = dict(q=FAKE, kv8=FAKE, kv_scale=FAKE, v8=NULL, v_scale=NULL, idx=FAKE, topk_length=NULL, sink=NULL, cu=NULL,
             table=NULL, n_seqs=0, T=4, H=64, Hc=1, Dqk=576, Dv=512, K=128, block=64, n_blocks=10, max_blocks=0,
             scale=0.1, out=FAKE, lse=FAKE, lse_kv=NULL, max_logits=NULL, workspace=FAKE, ws_bytes=1 << 40, stream=NULL)
    a.update(kw)
    return list(a.values())


GEOMETRY = [dict(n_seqs=0), dict(T=-1), dict(Hc=0), dict(Hc=1025), dict(D=0), dict(D=24), dict(D=1040), dict(block=0),
            dict(block=48), dict(block=512), dict(n_blocks=0), dict(n_blocks=1 << 25), dict(table=FAKE, max_blocks=0),
            dict(cu=NULL), dict(cache=NULL), dict(scale=NULL), dict(cache=ODD)]


@pytest.mark.parametrize("bad", GEOMETRY + [dict(src=NULL), dict(src=ODD)])
def test_write_refuses(lib, bad):
    assert lib.dsa_kv8_write(*write_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_kv8_write" in lib.dsa_last_error()


@pytest.mark.parametrize("bad", GEOMETRY + [dict(out=NULL), dict(out=ODD)])
def test_read_refuses(lib, bad):
    assert lib.dsa_kv8_read(*read_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_kv8_read" in lib.dsa_last_error()


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=129), dict(H=64, Hc=3), dict(Hc=0), dict(K=-1), dict(K=(1 << 30) + 1), dict(K=(1 << 31) - 1), dict(Dqk=256), dict(Dv=256),
    dict(Dqk=256, Dv=256), dict(Dqk=256, Dv=256, v8=FAKE), dict(Dqk=256, Dv=256, v_scale=FAKE), dict(v8=FAKE, v_scale=FAKE),
    dict(v_scale=FAKE), dict(block=0), dict(block=3), dict(block=512), dict(n_blocks=0), dict(n_blocks=1 << 25),
    dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(q=NULL), dict(kv8=NULL), dict(kv_scale=NULL),
    dict(idx=NULL), dict(out=NULL), dict(lse=NULL), dict(q=ODD), dict(kv8=ODD), dict(out=ODD),
    dict(table=FAKE), dict(table=FAKE, cu=FAKE, n_seqs=0, max_blocks=4), dict(table=FAKE, cu=FAKE, n_seqs=2, max_blocks=0),
])
def test_attention_refuses(lib, bad):
    assert lib.dsa_sparse_attn_fwd_kv8(*attn_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_sparse_attn_fwd_kv8" in lib.dsa_last_error()


@pytest.mark.parametrize("shape", [(1, 64, 1, 576, 512, 2048), (3, 24, 2, 256, 256, 1027)])
def test_attention_checks_its_workspace(lib, shape):
    T, H, Hc, Dqk, Dv, K = shape
    need = lib.dsa_sparse_attn_fwd_kv8_workspace_size(*shape)
    v = dict(v8=FAKE, v_scale=FAKE) if Dqk == 256 else {}
    if need == 0:
        return
    for bad in (dict(ws_bytes=need - 1), dict(workspace=NULL), dict(workspace=ctypes.c_void_p(4096 + 16))):
        rc = lib.dsa_sparse_attn_fwd_kv8(*attn_args(T=T, H=H, Hc=Hc, Dqk=Dqk, Dv=Dv, K=K, **v, **{"ws_bytes": need, **bad}))
        assert rc == ops.DSA_ERR_WORKSPACE


def test_workspace_of_invalid_shapes_is_zero(lib):
    for shape in [(0, 64, 1, 576, 512, 64), (4, 0, 1, 576, 512, 64), (4, 64, 0, 576, 512, 64), (4, 64, 3, 576, 512, 64),
                  (4, 64, 1, 576, 512, 0), (-1, 64, 1, 576, 512, 64), (4, 64, 1, 100, 512, 64)]:
        assert lib.dsa_sparse_attn_fwd_kv8_workspace_size(*shape) == 0


def test_binding_refuses_cpu_tensors():
    cache, scale = torch.zeros(2, 4, 1, 32, dtype=torch.uint8), torch.ones(2, 1)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.kv8_write(torch.zeros(3, 1, 32, dtype=torch.bfloat16), cache, scale, cu)
    with pytest.raises(ValueError):
        ops.kv8_read(cache, scale, cu, 3)
    with pytest.raises(TypeError):
        ops.kv8_read(cache.float(), scale, cu, 3)


def test_reference_codes_are_torchs():
    x = np.concatenate([R.VALUES[np.isfinite(R.VALUES)], np.linspace(-500, 500, 20001), np.linspace(-0.05, 0.05, 20001)])
    got = R.to_codes(x)
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # the doubles of the grids are fp32-rounded for torch: compare where that changes nothing
    same = x.astype(np.float32).astype(np.float64) == x
    assert same.sum() > 250 and np.array_equal(R.VALUES[got[same]], R.VALUES[want[same]])
    assert np.abs(R.VALUES[got] - np.clip(x, -448, 448)).max() <= 16.0  # half a step at the top


def test_reference_scale_is_the_smallest_power_of_two():
    for a in [1e-45, 2.0 ** -126, 1.0, 447.9, 448.0, 448.1, 3.3e38]:
        s = R.scale_of(a)
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 448 * s / 2)
    assert R.scale_of(0.0) == 2.0 ** -126
