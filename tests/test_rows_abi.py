"""Norm, rotary positions and the 4-bit cache without a GPU: refusals before anything
is launched, the host's angles, and the tests' own definitions (gradients against
differences among them)."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref
import rows_ref as R
from sparse_attention_gemm_gb300 import build as dsa_build
from sparse_attention_gemm_gb300 import ops
from test_kv8_abi import FAKE, NULL, ODD, attn_args, read_args, write_args

FAR = ctypes.c_void_p(1 << 20)
FAR2 = ctypes.c_void_p(1 << 21)


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return ops.lib()


def fwd_args(**kw):
    a = dict(x=FAKE, ld_x=512, residual=NULL, ld_r=0, weight=FAKE, T=4, D=512, eps=1e-6, fmt=0, y=FAR, ld_y=512,
             y_scale=NULL, sum=NULL, ld_sum=0, rstd=NULL, stream=NULL)
    a.update(kw)
    return list(a.values())


def bwd_args(**kw):
    a = dict(dy=FAKE, ld_dy=512, x=FAR, ld_x=512, weight=FAKE, rstd=FAKE, d_sum=NULL, ld_ds=0, T=4, D=512, dx=FAR2,
             ld_dx=512, dweight=FAKE, workspace=FAKE, ws_bytes=1 << 40, stream=NULL)
    a.update(kw)
    return list(a.values())


def rotary_args(**kw):
    a = dict(x=FAKE, x_token=512, x_head=64, H=8, x2=NULL, x2_token=0, x2_head=0, H2=0, inv_freq=FAKE, cu=FAKE,
             pos=NULL, n_seqs=2, T=8, R=64, interleaved=1, inverse=0, mul=1.0, y=FAR, y_token=512, y_head=64, y2=NULL,
             y2_token=0, y2_head=0, stream=NULL)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(D=0), dict(D=12), dict(D=16392, ld_x=16392, ld_y=16392), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(fmt=3), dict(fmt=-1), dict(fmt=1, D=64, y_scale=FAKE),
    dict(fmt=2, D=48, y_scale=FAKE), dict(fmt=1), dict(fmt=2), dict(ld_x=504), dict(ld_x=516), dict(ld_y=500),
    dict(residual=FAR2, ld_r=8), dict(sum=FAR2, ld_sum=516), dict(x=NULL), dict(y=NULL), dict(weight=NULL), dict(x=ODD),
    dict(y=ODD), dict(weight=ODD), dict(residual=ODD, ld_r=512), dict(sum=ODD, ld_sum=512), dict(y=FAKE, ld_y=520),
    dict(y=FAKE, fmt=1, y_scale=FAKE), dict(sum=FAKE, ld_sum=520), dict(sum=FAR, ld_sum=512),
    dict(residual=FAR, ld_r=520), dict(residual=FAR2, ld_r=512, sum=FAR2, ld_sum=520)])
def test_norm_refuses(lib, bad):
    assert lib.dsa_rms_norm_fwd(*fwd_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_rms_norm_fwd" in lib.dsa_last_error()


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(D=0), dict(D=20), dict(D=1 << 20, ld_dy=1 << 20, ld_x=1 << 20, ld_dx=1 << 20), dict(ld_dy=504),
    dict(ld_x=516), dict(ld_dx=511), dict(d_sum=FAKE, ld_ds=4), dict(dy=NULL), dict(x=NULL), dict(weight=NULL),
    dict(rstd=NULL), dict(dx=NULL), dict(dy=ODD), dict(x=ODD), dict(dx=ODD), dict(d_sum=ODD, ld_ds=512),
    dict(dx=FAKE, ld_dx=520), dict(dx=FAR, ld_dx=520), dict(d_sum=FAR2, ld_ds=520)])
def test_norm_backward_refuses(lib, bad):
    assert lib.dsa_rms_norm_bwd(*bwd_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_rms_norm_bwd" in lib.dsa_last_error()


def test_norm_backward_workspace(lib):
    need = lib.dsa_rms_norm_bwd_workspace_size(4, 512)
    assert need >= 512 * 4 and lib.dsa_rms_norm_bwd_workspace_size(0, 512) == 0
    assert lib.dsa_rms_norm_bwd_workspace_size(4, 511) == 0
    for bad in (dict(ws_bytes=need - 1), dict(workspace=NULL), dict(workspace=ctypes.c_void_p(4096 + 128))):
        assert lib.dsa_rms_norm_bwd(*bwd_args(**{"ws_bytes": need, **bad})) == ops.DSA_ERR_WORKSPACE
    # the largest shapes do not overflow
    assert lib.dsa_rms_norm_bwd_workspace_size(2 ** 31 - 1, 16384) < 1 << 30


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(n_seqs=0), dict(H=0), dict(H2=-1), dict(H=1025), dict(H=1024, H2=1), dict(R=0), dict(R=8), dict(R=24),
    dict(R=1040), dict(mul=float("nan")), dict(mul=float("inf")), dict(x=NULL), dict(y=NULL), dict(inv_freq=NULL),
    dict(cu=NULL), dict(H2=1, x2=FAKE), dict(H2=1, y2=FAKE), dict(x_token=516), dict(x_head=65), dict(y_token=516),
    dict(y_head=60), dict(y_head=0), dict(y_head=32), dict(y_token=64), dict(y_token=0), dict(y_token=504, y_head=64),
    dict(y_token=64, y_head=504), dict(x=ODD), dict(y=ODD), dict(inv_freq=ctypes.c_void_p(4100)), dict(y=FAKE, y_token=520),
    dict(H2=2, x2=FAR2, x2_token=128, x2_head=64, y2=FAR2, y2_token=136, y2_head=64),
    dict(H2=2, x2=FAR2, x2_token=128, x2_head=64, y2=FAKE, y2_token=128, y2_head=8)])
def test_rotary_refuses(lib, bad):
    assert lib.dsa_rotary(*rotary_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_rotary" in lib.dsa_last_error()


@pytest.mark.parametrize("good", [dict(y_token=64, y_head=64 * 8), dict(x_head=0), dict(y_head=72, y_token=7 * 72 + 64)])
def test_rotary_layouts_that_are_not_refused(lib, good):
    """Heads before tokens, one row read for all heads, rows apart: no complaint about arguments."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    assert lib.dsa_rotary(*rotary_args(**good)) == ops.DSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("R_,base,scaling,factor,first", [
    (64, 10000.0, "plain", 1.0, 4096), (64, 10000.0, "yarn", 40.0, 4096), (128, 500000.0, "yarn", 8.0, 8192),
    (16, 10000.0, "linear", 4.0, 1), (256, 1e6, "ntk", 3.5, 1), (2, 10.0, "plain", 1.0, 1), (1024, 10000.0, "yarn", 1.0, 77)])
def test_angles_per_position(lib, R_, base, scaling, factor, first):
    f, mul = ops.rotary_inv_freq(R_, base, scaling, factor, first, device="cpu")
    want, want_mul = R.inv_freq(R_, base, scaling, factor, first)
    assert f.dtype == torch.float64 and np.allclose(f.numpy(), want, rtol=1e-13, atol=0)
    assert abs(mul - want_mul) <= 2.0 ** -24 * want_mul


@pytest.mark.parametrize("bad", [dict(R=0), dict(R=3), dict(R=1026), dict(base=1.0), dict(base=float("nan")),
                                 dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=float("inf")),
                                 dict(scaling="yarn", factor=2.0, first=0), dict(scaling="ntk", factor=2.0, R=2),
                                 dict(scaling="yarn", factor=2.0, beta_slow=0.0),
                                 dict(scaling="yarn", factor=2.0, beta_slow=32.0), dict(scaling="other")])
def test_angles_refuse(lib, bad):
    with pytest.raises(ValueError):
        ops.rotary_inv_freq(**{"R": 64, "device": "cpu", **bad})


GEOMETRY = [dict(n_seqs=0), dict(T=-1), dict(Hc=0), dict(Hc=1025), dict(D=0), dict(D=48), dict(D=1056), dict(block=0),
            dict(block=48), dict(block=512), dict(n_blocks=0), dict(n_blocks=1 << 25), dict(table=FAKE, max_blocks=0),
            dict(cu=NULL), dict(cache=NULL), dict(scale=NULL), dict(cache=ODD)]


@pytest.mark.parametrize("bad", GEOMETRY + [dict(src=NULL), dict(src=ODD)])
def test_cache_writer_refuses(lib, bad):
    assert lib.dsa_kv4_write(*write_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_kv4_write" in lib.dsa_last_error()


@pytest.mark.parametrize("bad", GEOMETRY + [dict(out=NULL), dict(out=ODD)])
def test_cache_reader_refuses(lib, bad):
    assert lib.dsa_kv4_read(*read_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_kv4_read" in lib.dsa_last_error()


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=129), dict(H=64, Hc=3), dict(Hc=0), dict(K=-1), dict(K=(1 << 30) + 1), dict(Dqk=256),
    dict(Dv=256), dict(Dqk=256, Dv=256), dict(Dqk=256, Dv=256, v8=FAKE), dict(Dqk=256, Dv=256, v_scale=FAKE),
    dict(v8=FAKE, v_scale=FAKE), dict(v_scale=FAKE), dict(block=0), dict(block=3), dict(block=512), dict(n_blocks=0),
    dict(n_blocks=1 << 25), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(q=NULL),
    dict(kv8=NULL), dict(kv_scale=NULL), dict(idx=NULL), dict(out=NULL), dict(lse=NULL), dict(q=ODD), dict(kv8=ODD),
    dict(out=ODD), dict(table=FAKE), dict(table=FAKE, cu=FAKE, n_seqs=0, max_blocks=4),
    dict(table=FAKE, cu=FAKE, n_seqs=2, max_blocks=0), dict(T=1 << 26, H=128)])
def test_cache_attention_refuses(lib, bad):
    assert lib.dsa_sparse_attn_fwd_kv4(*attn_args(**bad)) == ops.DSA_ERR_VALUE
    assert b"dsa_sparse_attn_fwd_kv4" in lib.dsa_last_error()


# (shape, block, blocks, paged, fewest bytes): rows in splits leave a mean value and its sums each; a cache that
# is widened once takes its rows in bf16, and the slots' rows with a block table
@pytest.mark.parametrize("shape,block,n_blocks,paged,least", [
    ((32, 128, 1, 576, 512, 2048), 64, 10, False, 2 * 32 * 128 * 516 * 4),
    ((20, 64, 1, 512, 512, 2048), 64, 10, False, 2 * 20 * 64 * 516 * 4),
    ((1, 64, 1, 576, 512, 131072), 64, 4096, False, 2 * 64 * 516 * 4),
    ((2048, 64, 1, 576, 512, 2048), 64, 256, False, 64 * 256 * 576 * 2),
    ((2048, 64, 1, 576, 512, 2048), 64, 256, True, 64 * 256 * 576 * 2 + 2048 * 2048 * 4),
    ((2048, 20, 1, 256, 256, 2048), 16, 1000, False, 16 * 1000 * 512 * 2),
])
def test_cache_attention_workspace(lib, shape, block, n_blocks, paged, least):
    need = lib.dsa_sparse_attn_fwd_kv4_workspace_size(*shape, block, n_blocks, 1 if paged else 0)
    assert need >= least
    T, H, Hc, Dqk, Dv, K = shape
    a = dict(T=T, H=H, Hc=Hc, Dqk=Dqk, Dv=Dv, K=K, block=block, n_blocks=n_blocks)
    if paged:
        a.update(table=FAKE, cu=FAKE, n_seqs=2, max_blocks=4)
    if Dqk == 256:
        a.update(v8=FAKE, v_scale=FAKE)
    for bad in (dict(ws_bytes=need - 1), dict(ws_bytes=0), dict(workspace=NULL),
                dict(workspace=ctypes.c_void_p(4096 + 128))):
        assert lib.dsa_sparse_attn_fwd_kv4(*attn_args(**{**a, "ws_bytes": need, **bad})) == ops.DSA_ERR_WORKSPACE
        assert str(need).encode() in lib.dsa_last_error()


@pytest.mark.parametrize("shape,block,n_blocks", [
    ((1, 64, 1, 576, 512, 2048), 64, 1024), ((2048, 64, 1, 576, 512, 2048), 64, 20000), ((96, 24, 2, 256, 256, 1027), 16, 9999),
    ((0, 64, 1, 576, 512, 64), 64, 10), ((4, 64, 1, 576, 512, 0), 64, 10), ((4, 64, 3, 576, 512, 64), 64, 10)])
def test_cache_attention_needs_no_workspace(lib, shape, block, n_blocks):
    assert lib.dsa_sparse_attn_fwd_kv4_workspace_size(*shape, block, n_blocks, 1) == 0


@pytest.mark.parametrize("bad", [None, [[0.0]], 3, torch.tensor(1.0, dtype=torch.bfloat16)])
def test_bindings_refuse_what_is_no_row(bad):
    cache, scale = torch.zeros(2, 4, 1, 16, dtype=torch.uint8), torch.ones(2, 4, 1, 1, dtype=torch.uint8)
    cu, w = torch.tensor([0, 3], dtype=torch.int32), torch.ones(64)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    for call in (lambda: ops.kv4_write(bad, cache, scale, cu), lambda: ops.kv4_read(cache, scale, cu, 3, out=bad),
                 lambda: ops.kv4_write(torch.zeros(3, 1, 32, dtype=torch.bfloat16), bad, scale, cu),
                 lambda: ops.sparse_attn_fwd_kv4(bad, cache, scale, cu, 0.1), lambda: ops.rms_norm_fwd(bad, w, 1e-6),
                 lambda: ops.rms_norm_fwd(x, bad, 1e-6), lambda: ops.rms_norm_bwd(bad, x, w, w[:3]),
                 lambda: ops.rms_norm_bwd(x, bad, w, w[:3]), lambda: ops.rotary(bad, w.double(), cu),
                 lambda: ops.rotary(x.view(3, 1, 64), bad, cu), lambda: ops.rms_norm_fwd(x, w, 1e-6, fmt="int8")):
        with pytest.raises((TypeError, ValueError)):
            call()


# ------------------------------------------------------- the definitions themselves
def test_norm_gradient_is_that_of_differences():
    rng = np.random.default_rng(1)
    x, r, w, dy, ds = (rng.standard_normal(s) for s in ((3, 24), (3, 24), 24, (3, 24), (3, 24)))
    h, rstd, _ = R.norm(x, w, 1e-3, r)
    dx, dw, _, _ = R.norm_back(dy, h, w, rstd, ds)

    def loss(x, r, w):
        h, _, y = R.norm(x, w, 1e-3, r)
        return (y * dy).sum() + (h * ds).sum()

    e = 1e-6
    for t, c in ((0, 0), (1, 7), (2, 23)):
        d = np.zeros_like(x)
        d[t, c] = e
        assert abs((loss(x + d, r, w) - loss(x - d, r, w)) / (2 * e) - dx[t, c]) < 1e-7
        assert abs((loss(x, r + d, w) - loss(x, r - d, w)) / (2 * e) - dx[t, c]) < 1e-7
        d = np.zeros_like(w)
        d[c] = e
        assert abs((loss(x, r, w + d) - loss(x, r, w - d)) / (2 * e) - dw[c]) < 1e-7


@pytest.mark.parametrize("pairs", [True, False])
def test_rotary_adjoint_is_that_of_differences(pairs):
    """The map is linear: <rotary(x), g> = <x, adjoint(g)>, and differences of the left side give the adjoint."""
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((4, 3, 16)), rng.standard_normal((4, 3, 16))
    f, at = R.inv_freq(16, 10000.0)[0], [0, 1, 700, 1 << 20]
    back = R.rotary(g, f, at, pairs, True, 1.5)[0]
    e = 1e-5
    for i in ((0, 0, 0), (1, 2, 15), (3, 1, 8)):
        d = np.zeros_like(x)
        d[i] = e
        up, down = (R.rotary(x + s * d, f, at, pairs, False, 1.5)[0] for s in (1, -1))
        assert abs(((up - down) * g).sum() / (2 * e) - back[i]) < 1e-8


def test_e2m1_rounding():
    """Every border and a little to both sides of it, in a block whose scale is 1."""
    for lo, hi in zip(kv4_ref.MAGNITUDES[:-1], kv4_ref.MAGNITUDES[1:]):
        mid = (lo + hi) / 2
        x = np.zeros(32)
        x[:4] = [6.0, mid * (1 - 1e-6), mid, mid * (1 + 1e-6)]
        c, s = kv4_ref.quantise(x)
        at = int(np.nonzero(kv4_ref.MAGNITUDES == lo)[0][0])
        assert s[0] == 127 and list(c[1:4]) == [at, at + (at % 2), at + 1]
    c, s = kv4_ref.quantise(np.array([-0.0, 6.0000001, np.inf, -np.inf] + [0.0] * 28))
    assert s[0] == 128 and list(c[:4]) == [8, 5, 7, 15]
    assert kv4_ref.quantise(np.zeros(32))[1][0] == 1 and kv4_ref.quantise(np.full(32, np.nan))[1][0] == 255
    assert kv4_ref.quantise(np.full(32, kv4_ref.BF16_MOST))[1][0] == 252
