"""Attention over the 8-bit block cache where the softmax is far from flat:
one early key far above the rest whose value is zero or small (as models
without a learned sink have it), and a block whose value scale is far above the
others' while its keys have no weight.  What remains of such a row is the sum of many
small weights, so every output is held to a bound relative to sum_j p_j |v_j|
that does not grow with the largest weight."""
import math

import numpy as np
import pytest
import torch

from gpu_util import DEV, cu_from_lengths, dev, dev_bf16, f64
import kv8_ref as R
from sparse_attention_gemm_gb300 import ops
from sparse_attention_gemm_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    ops.device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0, "a kernel raised a device status flag"


def definition(q, k, ks, count, sm, v8=None, v_scale=None, sink=None, narrow=False):
    """out, lse and how far each may be off, in float64, for rows that select every cache row r count[t, r] times.

    Scores are fp32 sums of exact products of bf16 queries and codes: off by at most Dqk * 2^-24 of
    the products' magnitudes and 2^-21 of the score (scale, log2(e), the reference); d is the largest such error of a
    row's slots, and enters a weight and its norm: 2 d.  A weight is rounded to bf16 (2^-8).  The value product adds 16
    slots at a time to an fp32 sum, each time off by 2^-23 of it at most: n / 16 * 2^-23 over n slots.  2^-16:
    exp and the fp32 operations of the norm.  out is rounded to bf16 (2^-8).
    In groups of 16 heads a query element is off by at most 2^-22 of its head's largest, and a
    weight, held as 14 times itself against a reference less than a factor of two above the largest (scales being
    powers of two), is
    an E4M3 and an E5M2 term of a half: off by 2^-8 + 2^-11, or by 2^-14 (half the last step where the E4M3
    term has none) in the place of weights times 2^14: 2^-28 / 7 of the largest weight times its scale."""
    T, H, dqk = q.shape
    n_blocks, block, heads, _ = k.shape
    group, rows = H // heads, n_blocks * block
    blk = np.arange(rows) // block
    dv = 512 if v8 is None else v8.shape[3]
    out, tol = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    lse, ltol = np.zeros((T, H)), np.zeros((T, H))
    for g in range(heads):
        hs = slice(g * group, (g + 1) * group)
        kk = R.VALUES[k.reshape(rows, heads, dqk)[:, g]] * ks[blk, g].astype(np.float64)[:, None]
        sv = (ks if v8 is None else v_scale)[blk, g].astype(np.float64)
        code = R.VALUES[(k if v8 is None else v8).reshape(rows, heads, -1)[:, g, :dv]]
        vv = code * sv[:, None]
        for t in range(T):
            used = count[t] > 0
            c = count[t, used].astype(np.float64)
            s = sm * (q[t, hs] @ kk[used].T)
            d = sm * dqk * 2.0 ** -24 * (np.abs(q[t, hs]) @ np.abs(kk[used]).T) + 2.0 ** -21 * np.abs(s)
            if narrow:
                d += sm * 2.0 ** -22 * np.abs(q[t, hs]).max(1)[:, None] * np.abs(kk[used]).sum(1)[None, :]
            d = d.max(1)
            sk = np.full(s.shape[0], -np.inf) if sink is None else sink[hs].astype(np.float64)
            m = np.maximum(s.max(1), sk)
            e = np.exp(s - m[:, None]) * c
            z = e.sum(1) + np.exp(sk - m)
            p = e / z[:, None]
            out[t, hs] = p @ vv[used]
            lse[t, hs] = m + np.log(z)
            n = c.sum()
            tol[t, hs] = (2.0 ** -8 * np.abs(out[t, hs]) +
                          (2.0 ** -8 + 2 * d[:, None] + n * 2.0 ** -27 + 2.0 ** -16) * (p @ np.abs(vv[used])))
            if narrow:
                tol[t, hs] += 2.0 ** -11 * (p @ np.abs(vv[used]))
                tol[t, hs] += (2.0 ** -28 / 7) * ((p / c) * sv[used]).max(1)[:, None] * (c @ np.abs(code[used]))[None, :]
            ltol[t, hs] = d + n * 2.0 ** -28 + 2.0 ** -19 + 2.0 ** -21 * (np.abs(lse[t, hs]) + 16)
    return out, tol, lse, ltol


def code_of(x):
    return R.to_codes(np.asarray(x, np.float64))


def finite_codes(rng, shape):
    c = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 127) == 127, c & 0x80, c).astype(np.uint8)


def check(form, q, k, ks, idx, sm, table=False, narrow=False, **kw):
    dqk, dv = form
    rows = k.shape[0] * k.shape[1]
    count = np.stack([np.bincount(i, minlength=rows) for i in idx])
    out, tol, lse, ltol = definition(f64(q), k, ks, count, sm, narrow=narrow, **kw)
    d = {n: dev(a) for n, a in kw.items() if n != "sink"}
    if "sink" in kw:
        d["sink"] = dev(kw["sink"])
    if table:  # one sequence whose pages are the cache's blocks in order
        d["block_table"] = dev(np.arange(k.shape[0], dtype=np.int32)[None])
        d["cu_seqlens"] = dev(cu_from_lengths([idx.shape[0]]))
    got = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, **d)
    o = got["out"].float().cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all()
    far = np.abs(o - out) / np.maximum(tol, 1e-300)
    assert not (far > 1).any(), f"{(far > 1).mean():.1%} of the outputs out of tolerance, the farthest {far.max():.1f} times"
    l = got["lse"].cpu().numpy().astype(np.float64)
    assert not (np.abs(l - lse) > ltol).any()
    return got, out, tol


def peaked(rng, form, T, H, heads, K, block, n, small, where, lo=6.0, hi=28.0):
    """Row 0 of the cache lies lo .. hi nats (from the first head to the last) above the others; its value is zero, or
    `small`: codes of the smallest steps.  The last key dim tells it from the others."""
    dqk, dv = form
    n_blocks = n // block
    k = finite_codes(rng, (n_blocks, block, heads, dqk))
    k[..., -1] = 0
    ks = np.exp2(rng.integers(-8, -5, (n_blocks, heads))).astype(np.float32)
    kw = {}
    if dqk == 256:
        kw["v8"], kw["v_scale"] = finite_codes(rng, (n_blocks, block, heads, dv)), np.exp2(rng.integers(-8, -5, (n_blocks, heads))).astype(np.float32)
        kw["v8"][0, 0] = rng.integers(0, 8, (heads, dv)) if small else 0
    k[0, 0] = rng.integers(0, 8, (heads, dqk)) if small else 0
    k[0, 0, :, -1] = code_of(448.0)
    sm = 1.0 / math.sqrt(dqk)
    q = rng.standard_normal((T, H, dqk)) * 0.3
    group = H // heads
    for h in range(H):
        gap = lo + (hi - lo) * (h % group) / max(group - 1, 1)
        q[:, h, -1] = gap / (sm * 448.0 * float(ks[0, h // group]))
    idx = rng.integers(1, n_blocks * block, (T, K)).astype(np.int32)
    at = {"first": 0, "middle": K // 2, "last": K - 1}[where]
    idx[:, at] = 0
    return W.f32_to_bf16_bits(q.astype(np.float32)), k, ks, idx, sm, kw


# (T, H, heads, K): whole rows and rows in splits
WIDE = [(40, 64, 1, 2048), (200, 40, 1, 512), (90, 128, 1, 300), (1, 64, 1, 131072), (1, 16, 1, 1100000)]
NARROW = [(1, 64, 1, 2048), (3, 16, 1, 16384), (2, 24, 2, 700), (5, 16, 1, 64), (300, 12, 1, 130), (1, 16, 1, 131072), (70, 32, 1, 512)]
FORMS = [(576, 512), (512, 512), (256, 256)]


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,heads,K", WIDE)
def test_peaked_rows_wide(form, T, H, heads, K, small, where):
    rng = np.random.default_rng(K + H + T + form[0])
    q, k, ks, idx, sm, kw = peaked(rng, form, T, H, heads, K, 16, 4096, small, where)
    check(form, q, k, ks, idx, sm, table=where == "middle", **kw)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("up", [8, 14, 40])
@pytest.mark.parametrize("T,H,heads,K", WIDE[:3])
def test_unused_block_of_large_scale_wide(form, T, H, heads, K, up):
    unused_block(form, T, H, heads, K, up)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,heads,K", NARROW)
def test_peaked_rows_narrow(form, T, H, heads, K, small, where):
    rng = np.random.default_rng(K + H + T + form[0])
    q, k, ks, idx, sm, kw = peaked(rng, form, T, H, heads, K, 16, 4096, small, where, hi=16.0)
    check(form, q, k, ks, idx, sm, table=where == "middle", narrow=True, **kw)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("up", [8, 14, 40])
@pytest.mark.parametrize("T,H,heads,K", NARROW[:5])
def test_unused_block_of_large_scale_narrow(form, T, H, heads, K, up):
    unused_block(form, T, H, heads, K, up, narrow=True)


def unused_block(form, T, H, heads, K, up, narrow=False):
    """One block's scale is 2^up times the others', and its keys have no weight."""
    rng = np.random.default_rng(K + H + T + up)
    dqk, dv = form
    block, n_blocks, group = 16, 64, H // heads
    k = finite_codes(rng, (n_blocks, block, heads, dqk))
    k[..., -1] = rng.integers(0, 0x70, k.shape[:3])  # 0 .. 120
    k[7, ..., -1] = code_of(-448.0)
    ks = np.full((n_blocks, heads), 2.0 ** -6, np.float32)
    kw = {}
    if dqk == 256:
        kw["v8"], kw["v_scale"] = finite_codes(rng, (n_blocks, block, heads, dv)), np.full((n_blocks, heads), 2.0 ** -6, np.float32)
        kw["v_scale"][7] *= 2.0 ** up
    else:
        ks[7] *= 2.0 ** up
    q = np.zeros((T, H, dqk))
    sm = 1.0 / math.sqrt(dqk)
    q[..., -1] = np.linspace(0.5, 3.0, H) / (sm * 2.0 ** -6 * 120)  # the others' scores: 0 .. 3 nats
    if dqk == 256:
        q[..., -1] *= 40  # 0 .. 120 nats, the block at -448
    idx = rng.integers(0, n_blocks * block, (T, K)).astype(np.int32)
    idx[:, 5] = 7 * block + 3
    check(form, W.f32_to_bf16_bits(q.astype(np.float32)), k, ks, idx, sm, narrow=narrow, **kw)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,K,narrow", [(40, 64, 2048, False), (1, 64, 131072, False), (1, 64, 2048, True), (3, 16, 16384, True)])
def test_peaked_rows_as_the_bf16_call_on_values_read_back(form, T, H, K, narrow):
    """Powers of two as scales: the values read back are the cache's, and each call is within its bound of the same
    definition (the bf16 call rounds what groups of 64 heads round)."""
    rng = np.random.default_rng(K + H + T + form[0] + 1)
    q, k, ks, idx, sm, kw = peaked(rng, form, T, H, 1, K, 16, 4096, True, "first", hi=16.0)
    got, out, tol = check(form, q, k, ks, idx, sm, narrow=narrow, **kw)
    n = k.shape[0] * k.shape[1]
    cu = dev(cu_from_lengths([n]))
    kv = ops.kv8_read(dev(k), dev(ks), cu, n).view(n, form[0])
    v = ops.kv8_read(dev(kw["v8"]), dev(kw["v_scale"]), cu, n).view(n, form[1]) if kw else None
    other = ops.sparse_attn_fwd(dev_bf16(q), kv, dev(idx), sm, v=v)
    o = other["out"].float().cpu().numpy().astype(np.float64)
    assert not (np.abs(o - out) > tol).any()
    assert float((got["lse"] - other["lse"]).abs().max()) <= 2e-3
