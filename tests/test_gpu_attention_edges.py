"""Rows of sparse attention that meet NaN, that have no slot, or whose cache rows have large scales, in every
form of the calls."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as R
import test_gpu_kv8 as kv8
from gpu_util import DEV, dev, dev_bf16, rand_bf16_bits
from sparse_attention_gemm_gb300 import ops
from test_gpu_kv4 import FORMS, attention_case, cache_of, check_attention

pytestmark = pytest.mark.gpu

STATISTICS = ("lse", "lse_kv", "max_logits")
# 16 heads whole and in splits; 64 heads whole and in splits; a cache that is widened once
SHAPES = [(4, 16, 70, None), (4, 16, 1500, None), (130, 64, 70, None), (12, 64, 1500, None), (700, 64, 700, 900)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    ops.device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0, "a kernel raised a device status flag"


def kv4_call(q, k, ks, idx, sm, kw, **more):
    d = {n: dev(kw[n]) for n in ("v4", "v_scale", "sink") if n in kw}
    if "length" in kw:
        d["topk_length"] = dev(kw["length"])
    return ops.sparse_attn_fwd_kv4(q, dev(k), dev(ks), dev(idx), sm, want_lse_kv=True, want_max_logits=True, **d, **more)


def assert_widened(T, H, dqk, dv, K, k, n):
    if n:
        need = ops.sparse_attn_fwd_kv4_workspace_size(T, H, 1, dqk, dv, K, k.shape[1], k.shape[0])
        assert need >= k.shape[0] * k.shape[1] * dqk * 2


def assert_nan_only(got, clean, hit, names):
    """Every result of the (row, head) pairs in `hit` is NaN, the others' bits are those of `clean`."""
    for n in names:
        assert bool(got[n][hit].isnan().all()), f"{n}: not NaN"
        assert torch.equal(got[n][~hit], clean[n][~hit]), n


def pairs(T, H, *hits):
    m = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    for t, h in hits:
        m[t, h] = True
    return m


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K,n", SHAPES)
def test_nan_reaches_every_result_of_its_rows(dqk, dv, T, H, K, n):
    rng = np.random.default_rng(dqk + T + K)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, 1, False, n=n, holes=False)
    assert_widened(T, H, dqk, dv, K, k, n)
    kw["sink"] = rng.standard_normal(H).astype(np.float32)
    hit = idx[0, 5]
    idx[1:][idx[1:] == hit] = (hit + 1) % k.shape[0]
    names = ("out", *STATISTICS)
    clean = kv4_call(dev_bf16(q), k, ks, idx, sm, kw)
    bad = ks.copy()
    bad[hit, 0, 0, 2] = 255
    assert_nan_only(kv4_call(dev_bf16(q), k, bad, idx, sm, kw), clean, pairs(T, H, (0, slice(None))), names)
    q2 = dev_bf16(q)
    q2[2, 7, 3], q2[3, 9, 200] = float("nan"), float("inf")
    assert_nan_only(kv4_call(q2, k, ks, idx, sm, kw), clean, pairs(T, H, (2, 7), (3, 9)), names)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H", [(5, 64), (200, 20)])
def test_nan_over_bf16_rows(dqk, dv, T, H):
    """The call over bf16 rows, with the statistic of the first slots: NaN from a key and from a query's head."""
    rng = np.random.default_rng(dqk + T)
    K, n = 200, 900
    q, kv = dev_bf16(rand_bf16_bits(rng, (T, H, dqk))), dev_bf16(rand_bf16_bits(rng, (n, dqk)))
    idx = rng.integers(0, n, (T, K)).astype(np.int32)
    hit, late = idx[0, 5], idx[1, 150]
    idx[1:][idx[1:] == hit] = (hit + 1) % n
    idx[idx == late] = (late + 1) % n
    idx[0, 5], idx[1, 150] = hit, late
    args = dict(sink=dev(rng.standard_normal(H).astype(np.float32)), want_lse_kv=True, want_max_logits=True, indexer_topk=64,
                v=dev_bf16(rand_bf16_bits(rng, (n, dv))) if dqk == 256 else None)
    clean = ops.sparse_attn_fwd(q, kv, dev(idx), 0.05, **args)
    bad = kv.clone()
    bad[int(hit), 40] = float("nan")
    names = ("out", "lse_indexer", *STATISTICS)
    assert_nan_only(ops.sparse_attn_fwd(q, bad, dev(idx), 0.05, **args), clean, pairs(T, H, (0, slice(None))), names)
    bad = kv.clone()
    bad[int(late), 40] = float("nan")  # behind the first slots: their statistic stays
    got = ops.sparse_attn_fwd(q, bad, dev(idx), 0.05, **args)
    assert_nan_only(got, clean, pairs(T, H, (1, slice(None))), ("out", *STATISTICS))
    assert torch.equal(got["lse_indexer"], clean["lse_indexer"])
    q2 = q.clone()
    q2[2, 7, 3], q2[3, 9, 200] = float("nan"), float("inf")
    assert_nan_only(ops.sparse_attn_fwd(q2, kv, dev(idx), 0.05, **args), clean, pairs(T, H, (2, 7), (3, 9)), names)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K", [(4, 16, 70), (4, 64, 1500), (200, 64, 70), (100, 128, 700)])
def test_nan_over_the_8_bit_cache(dqk, dv, T, H, K):
    rng = np.random.default_rng(dqk + T + K)
    q, k, ks, idx, sm, kw = kv8.attention_case(rng, dqk, dv, T, H, 1, K, 1, False, holes=False)
    args = dict(sink=dev(rng.standard_normal(H).astype(np.float32)), want_lse_kv=True, want_max_logits=True,
                **{n: dev(kw[n]) for n in ("v8", "v_scale") if n in kw})
    hit = idx[0, 5]
    idx[1:][idx[1:] == hit] = (hit + 1) % k.shape[0]
    clean = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, **args)
    bad = k.copy()
    bad[hit, 0, 0, 40] = 127
    got = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(bad), dev(ks), dev(idx), sm, **args)
    assert_nan_only(got, clean, pairs(T, H, (0, slice(None))), ("out", *STATISTICS))


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K,n", SHAPES)
@pytest.mark.parametrize("sink", [True, False])
def test_rows_without_slots_give_the_sink_itself(dqk, dv, T, H, K, n, sink):
    """Rows whose slots are all unmapped: lse is the sink's own bits (-inf without one), not the sink taken to powers of
    two and back."""
    rng = np.random.default_rng(dqk + T + K + 1)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, 1, False, n=n, holes=False)
    assert_widened(T, H, dqk, dv, K, k, n)
    idx[0], idx[2], idx[3, ::2], idx[3, 1::2] = -1, 1 << 30, -7, k.shape[0]
    kw["length"] = np.full(T, K, np.int32)
    kw["length"][1] = 0
    want = torch.full((4, H), -math.inf, device=DEV)
    if sink:
        kw["sink"] = (3 * rng.standard_normal(H)).astype(np.float32)
        want = dev(kw["sink"]).expand(4, H)
    got = kv4_call(dev_bf16(q), k, ks, idx, sm, kw)
    assert bool((got["out"][:4] == 0).all()) and torch.equal(got["lse"][:4], want)
    assert bool((got["lse_kv"][:4] == math.inf).all()) and bool((got["max_logits"][:4] == -math.inf).all())


@pytest.mark.parametrize("T,H", [(5, 64), (200, 20)])
def test_bf16_rows_without_slots_give_the_sink_itself(T, H):
    rng = np.random.default_rng(T)
    q, kv = dev_bf16(rand_bf16_bits(rng, (T, H, 576))), dev_bf16(rand_bf16_bits(rng, (300, 576)))
    idx = torch.full((T, 130), -1, dtype=torch.int32, device=DEV)
    idx[1:] = 300
    sink = dev((3 * rng.standard_normal(H)).astype(np.float32))
    got = ops.sparse_attn_fwd(q, kv, idx, 0.05, sink=sink, want_lse_kv=True, want_max_logits=True, indexer_topk=64)
    assert bool((got["out"] == 0).all()) and torch.equal(got["lse"], sink.expand(T, H))
    assert bool((got["lse_kv"] == math.inf).all()) and bool((got["max_logits"] == -math.inf).all())
    assert bool((got["lse_indexer"] == math.inf).all())


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K,n", SHAPES + [(32, 128, 2048, None)])
@pytest.mark.parametrize("cache", ["4 bits", "8 bits"])
def test_statistics_under_a_sink_far_above_the_scores(dqk, dv, T, H, K, n, cache):
    """lse_kv and max_logits know nothing of the sink; lse is the sink's, out next to nothing."""
    rng = np.random.default_rng(dqk + T + K + 2)
    if cache == "4 bits":
        q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, 1, False, n=n, holes=False)

        def call(sink):
            return kv4_call(dev_bf16(q), k, ks, idx, sm, dict(kw, sink=sink))
    else:
        q, k, ks, idx, sm, kw = kv8.attention_case(rng, dqk, dv, T, H, 1, K, 1, False, n=n, holes=False)
        args = {m: dev(kw[m]) for m in ("v8", "v_scale") if m in kw}

        def call(sink):
            return ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, sink=dev(sink), want_lse_kv=True,
                                           want_max_logits=True, **args)
    low = call(np.full(H, -100.0, np.float32))
    sink = (90 + 60 * rng.random(H)).astype(np.float32)
    high = call(sink)
    # (a product with ln 2 and, of both, a sum and a logarithm: a few roundings of numbers below 2^8)
    tol = 8 * 2.0 ** -24 * 256
    assert bool(((high["lse_kv"] - low["lse_kv"]).abs() <= tol).all()), "lse_kv"
    assert torch.equal(high["max_logits"], low["max_logits"])
    assert bool(((high["lse"] - dev(sink)).abs() <= tol).all()) and bool((high["out"].abs() <= 1e-20).all())


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,heads,K,block", [(6, 12, 1, 130, 1), (4, 16, 1, 1500, 16), (3, 24, 2, 65, 4), (2, 64, 1, 700, 64)])
@pytest.mark.parametrize("hi", [129, 134])
def test_large_scales_in_groups_of_16_heads(dqk, dv, T, H, heads, K, block, hi):
    """Bytes above 128, whose factor takes two products: alone in a tile and among small ones, in rows whose scales begin
    at either half of a word, in the first and the last of a row's blocks, in keys and values; whole and in splits."""
    rng = np.random.default_rng(dqk + T + K + hi)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, heads, K, block, False)
    assert ops.sparse_attn_fwd_kv4_workspace_size(T, H, heads, dqk, dv, K, block, k.shape[0]) == 0
    flat = ks.reshape(-1, heads, dqk // 32)
    many = rng.choice(flat.shape[0], flat.shape[0] // 3, replace=False)
    flat[many, 0, rng.integers(0, dqk // 32, many.size)] = rng.integers(129, hi + 1, many.size)
    flat[many[::2], heads - 1, 0], flat[many[1::2], heads - 1, dqk // 32 - 1] = hi, hi
    if dqk == 256:
        vs = kw["v_scale"].reshape(-1, heads, dv // 32)
        vs[many, 0, rng.integers(0, dv // 32, many.size)] = rng.integers(129, hi + 1, many.size)
    check_attention(q, k, ks, idx, sm * 2.0 ** (127 - hi), sink=rng.standard_normal(H).astype(np.float32), **kw)


def many_sequences(rng, T, n_seqs, pad, block, n_blocks, width):
    """cu (empty sequences among them, `pad` rows behind the last), and a table with unmapped and foreign pages."""
    cuts = np.sort(rng.integers(0, T - pad + 1, n_seqs - 1))
    cu = np.concatenate([[0], cuts, [T - pad]]).astype(np.int32)
    table = rng.integers(0, n_blocks, (n_seqs, width)).astype(np.int32)
    table[rng.random(table.shape) < 0.1] = -1
    table[rng.random(table.shape) < 0.05] = n_blocks + 3
    return cu, table


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K,n_seqs,pad", [(60, 16, 70, 50, 7), (5, 16, 1500, 40, 2), (3, 64, 2000, 2, 2), (150, 64, 70, 1100, 20),
                                              (14, 64, 1500, 33, 3), (40, 12, 130, 3, 40)])
def test_batches_of_many_sequences(dqk, dv, T, H, K, n_seqs, pad):
    """More sequences than a warp looks up at once, empty ones, padding behind them (or nothing else), rows in splits."""
    rng = np.random.default_rng(dqk + T + K + 3)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, 16, False, n=600)
    kw["cu"], kw["table"] = many_sequences(rng, T, n_seqs, pad, 16, k.shape[0], 20)
    idx %= 20 * 16 + 40  # positions behind the table among them
    check_attention(q, k, ks, idx, sm, sink=rng.standard_normal(H).astype(np.float32), **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K,n_seqs,pad", [(700, 64, 700, 300, 45), (14000, 17, 33, 40, 700), (600, 100, 900, 1, 0), (330000, 20, 1, 9, 11)])
def test_a_widened_cache_gives_the_bits_of_the_bf16_call(dqk, dv, T, H, K, n_seqs, pad):
    rng = np.random.default_rng(dqk + T + K + 4)
    block = 16
    n = 600
    n_blocks = n // block + 2
    k, ks = (dev(a) for a in cache_of(rng, n_blocks, block, 1, dqk))
    v, vs = (dev(a) for a in cache_of(rng, n_blocks, block, 1, dv)) if dqk == 256 else (None, None)
    cu, table = many_sequences(rng, T, n_seqs, pad, block, n_blocks, 20)
    q = torch.randn(T, H, dqk, device=DEV, generator=torch.Generator(DEV).manual_seed(T)).to(torch.bfloat16)
    idx = rng.integers(-30, 20 * block + 40, (T, K)).astype(np.int32)
    length = rng.integers(-3, K + 9, T).astype(np.int32)
    sink = dev(rng.standard_normal(H).astype(np.float32))
    need = ops.sparse_attn_fwd_kv4_workspace_size(T, H, 1, dqk, dv, K, block, n_blocks, True)
    assert need >= n_blocks * block * dqk * 2 + T * K * 4
    out, lse = torch.full((T, H, dv), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, H), 7.0, device=DEV)
    got = ops.sparse_attn_fwd_kv4(q, k, ks, dev(idx), 0.05, topk_length=dev(length), sink=sink, v4=v, v_scale=vs, cu_seqlens=dev(cu),
                                  block_table=dev(table), want_lse_kv=True, want_max_logits=True, out=out, lse=lse)
    done = T - pad
    assert bool((out[done:] == 7.0).all()) and bool((lse[done:] == 7.0).all())
    seq = np.searchsorted(cu, np.arange(done), side="right") - 1
    page = idx[:done] // block
    there = (idx[:done] >= 0) & (page < table.shape[1])
    blk = table[seq[:, None], np.where(there, page, 0)]
    row = np.where(there & (blk >= 0) & (blk < n_blocks), blk * block + idx[:done] % block, -1).astype(np.int32)
    every = dev(np.array([0, n_blocks * block], np.int32))
    wide = [None if c is None else ops.kv4_read(c, s, every, n_blocks * block)[:, 0] for c, s in ((k, ks), (v, vs))]
    want = ops.sparse_attn_fwd(q[:done], wide[0], dev(row), 0.05, topk_length=dev(length[:done]), sink=sink, v=wide[1], want_lse_kv=True,
                               want_max_logits=True)
    for name in ("out", *STATISTICS):
        assert torch.equal(got[name][:done], want[name]), name
