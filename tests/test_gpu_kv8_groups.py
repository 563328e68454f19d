"""Attention over the 8-bit block cache in both of its forms, groups of 64 and
of 16 query heads: sizes that take the wide form (more than 16 heads per KV
head and more work than a few rows), against the 64-bit definition; rows that
are the same in both; aborts, other streams and captured calls of either."""
import math

import numpy as np
import pytest
import torch

from gpu_util import DEV, cu_from_lengths, dev, dev_bf16, f64, rand_bf16_bits
import kv8_ref as R
from sparse_attention_gemm_gb300 import ops
from test_gpu_kv8 import FORMS, attention_case, cache_of, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    ops.set_wait_limit_ns(0)
    ops.device_status(clear=True)
    yield
    ops.set_wait_limit_ns(0)
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0, "a kernel raised a device status flag"


def call(q, k, ks, idx, sm, **kw):
    d = {n: None if kw.get(n) is None else dev(kw[n]) for n in ("length", "sink", "v8", "v_scale", "cu", "table")}
    args = [dev_bf16(q), dev(k), dev(ks), dev(idx), sm]
    return lambda: ops.sparse_attn_fwd_kv8(*args, topk_length=d["length"], sink=d["sink"], v8=d["v8"], v_scale=d["v_scale"],
                                           cu_seqlens=d["cu"], block_table=d["table"], want_lse_kv=True)


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in ("out", "lse", "lse_kv"))


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,heads,K,block,table,sink", [
    (100, 64, 1, 260, 16, True, True),      # odd lengths, the last tile half empty
    (60, 128, 1, 290, 64, False, False),    # two full groups
    (40, 200, 2, 193, 32, True, True),      # groups of 64 and 36 heads, two KV heads
    (50, 64, 1, 700, 64, True, False),      # three splits of a row
    (20, 64, 1, 2048, 64, False, True),     # slots split between CTAs, joined by the second kernel
    (400, 64, 1, 130, 4, True, False),      # several items a CTA, some empty
    (170, 33, 1, 300, 1, False, True),      # one head in the upper half of a group
    (330, 20, 1, 380, 16, True, False),     # half a group
])
def test_wide_groups(dqk, dv, T, H, heads, K, block, table, sink):
    rng = np.random.default_rng(T * 1000 + H + K + dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, heads, K, block, table)
    if sink:
        kw["sink"] = rng.standard_normal(H).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_narrow_groups_of_many_heads(dqk, dv):
    """Few rows of 128 heads: eight groups of 16, undivided, in two and in eight splits."""
    for T, K in ((3, 60), (9, 500), (1, 2048)):
        rng = np.random.default_rng(dqk + T)
        q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, 128, 1, K, 64, False, n=3000)
        check_attention(q, k, ks, idx, sm, sink=rng.standard_normal(128).astype(np.float32), **kw)


def test_many_sequences():
    """The row's sequence among more than 32 and more than 1024, some of them empty, in both forms."""
    for n_seqs, T, H in ((50, 210, 64), (1500, 700, 16), (33, 33, 16)):
        rng = np.random.default_rng(n_seqs)
        K, block, per = 70, 8, 3
        n_blocks = 60
        k, ks = cache_of(rng, n_blocks, block, 1, 576)
        new = rng.multinomial(T - 3, np.ones(n_seqs) / n_seqs)  # and three rows of padding
        table = rng.integers(0, n_blocks, (n_seqs, per)).astype(np.int32)
        table[rng.random(table.shape) < 0.1] = -1
        idx = rng.integers(-2, per * block + 5, (T, K)).astype(np.int32)
        q = rand_bf16_bits(rng, (T, H, 576))
        check_attention(q, k, ks, idx, 1 / 24, cu=cu_from_lengths([int(x) for x in new]), table=table)


def test_wide_leaves_padding_rows():
    rng = np.random.default_rng(78)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 200, 64, 1, 90, 16, True)
    kw["cu"] = cu_from_lengths([50, 100])
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("lo,hi", [(-120, -100), (60, 90), (-126, 90)])
def test_wide_scales_of_every_size(lo, hi):
    rng = np.random.default_rng(300 + hi)
    q, k, ks, idx, sm, kw = attention_case(rng, 256, 256, 150, 40, 1, 200, 4, False, holes=False)
    kw["v_scale"] = np.exp2(rng.integers(lo, hi + 1, kw["v_scale"].shape)).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_wide_rising_and_falling_scores(dqk, dv):
    """The running maximum moves in many tiles, for rows that share a CTA."""
    rng = np.random.default_rng(dqk + 1)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, 60, 64, 1, 512, 1, False, holes=False)
    ks[:] = 2.0 ** -4
    s = f64(q)[:, 0] @ (R.VALUES[k[:, 0, 0]]).T
    for t in range(60):
        order = np.argsort(s[t])[:: 1 if t % 2 else -1]
        idx[t] = order[np.linspace(0, order.size - 1, idx.shape[1]).astype(int)]
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_wide_never_uses_unselected_rows(dqk, dv):
    """NaN codes and scales in blocks that no slot names."""
    rng = np.random.default_rng(dqk + 4)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, 200, 64, 1, 90, 8, False)
    rows = k.shape[0] * 8
    cut = rng.permutation(k.shape[0])[:5]
    idx[(idx >= 0) & (idx < rows) & np.isin(np.clip(idx, 0, rows - 1) // 8, cut)] = -1
    spoilt = dict(kw)
    k2, ks2 = k.copy(), ks.copy()
    k2[cut], ks2[cut] = 127, np.nan
    if dqk == 256:
        spoilt["v8"], spoilt["v_scale"] = kw["v8"].copy(), kw["v_scale"].copy()
        spoilt["v8"][cut], spoilt["v_scale"][cut] = 255, np.inf
    assert same(call(q, k, ks, idx, sm, **kw)(), call(q, k2, ks2, idx, sm, **spoilt)())


def test_wide_nan_reaches_only_its_rows():
    rng = np.random.default_rng(22)
    q, k, ks, idx, sm, _ = attention_case(rng, 576, 512, 200, 64, 1, 70, 1, False, holes=False)
    hit = idx[0, 5]
    idx[1:][idx[1:] == hit] = (hit + 1) % k.shape[0]
    clean = call(q, k, ks, idx, sm)()["out"]
    bad = k.copy()
    bad[hit, 0, 0, 570] = 127
    got = call(q, bad, ks, idx, sm)()["out"]
    assert bool(got[0].isnan().all()) and torch.equal(got[1:], clean[1:])
    q2 = dev_bf16(q)
    q2[2, 7, 3], q2[199, 63, 500] = float("nan"), float("inf")
    got = ops.sparse_attn_fwd_kv8(q2, dev(k), dev(ks), dev(idx), sm)["out"]
    hit = torch.zeros(200, 64, dtype=torch.bool, device=DEV)
    hit[2, 7] = hit[199, 63] = True
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], clean[~hit])


def test_wide_offsets_beyond_32_bits():
    rng = np.random.default_rng(33)
    block, n_blocks = 64, 120000
    cache = torch.zeros((n_blocks, block, 1, 576), dtype=torch.uint8, device=DEV)
    scale = torch.ones((n_blocks, 1), device=DEV)
    k, ks = cache_of(rng, 4, block, 1, 576)
    at = [0, 1, n_blocks - 2, n_blocks - 1]
    for i, b in enumerate(at):
        cache[b], scale[b] = dev(k[i]), dev(ks[i])
    idx = rng.integers(0, 4 * block, (200, 150)).astype(np.int32)
    far = (np.array(at)[idx // block] * block + idx % block).astype(np.int32)
    q = dev_bf16(rand_bf16_bits(rng, (200, 64, 576)))
    a = ops.sparse_attn_fwd_kv8(q, cache, scale, dev(far), 0.04)
    b = ops.sparse_attn_fwd_kv8(q, dev(k), dev(ks), dev(idx), 0.04)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


# (form, T, H, K): narrow undivided and in a cluster, wide undivided and in splits
CALLS = [((576, 512), 300, 16, 256), ((512, 512), 2, 64, 1024), ((256, 256), 90, 12, 700), ((576, 512), 400, 64, 300),
         ((512, 512), 300, 64, 300), ((256, 256), 300, 64, 300), ((576, 512), 20, 64, 2048),
         ((512, 512), 50, 64, 700), ((256, 256), 30, 64, 1200)]


def made(form, T, H, K, seed=50):
    rng = np.random.default_rng(seed + T + H + K)
    q, k, ks, idx, sm, kw = attention_case(rng, *form, T, H, 1, K, 16, True)
    kw["sink"] = rng.standard_normal(H).astype(np.float32)
    return call(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("form,T,H,K", CALLS)
def test_forced_wait_timeout_aborts_cleanly(form, T, H, K):
    """Every wait that is not satisfied at once gives up: the call returns, the status says so, nothing is left in
    flight, and the next call gives the bits of the one before."""
    f = made(form, T, H, K)
    before = {n: x.clone() for n, x in f().items()}
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0
    ops.set_wait_limit_ns(1)
    try:
        f()
        torch.cuda.synchronize()
        st = ops.device_status(clear=True)
        assert st & ops.DSA_STATUS_WAIT_TIMEOUT and not st & ops.DSA_STATUS_DRAIN_TIMEOUT, hex(st)
    finally:
        ops.set_wait_limit_ns(0)
    ops.device_status(clear=True)
    assert same(f(), before)
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0


def test_calls_on_two_streams():
    """Calls of both forms at once on two streams give the bits they give alone; each allocates its own workspace."""
    fs = [made(*c) for c in CALLS]
    alone = [f() for f in fs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for i, f in enumerate(fs):
            with torch.cuda.stream(streams[i % 2]):
                got.append((i, f()))
    torch.cuda.synchronize()
    assert all(same(r, alone[i]) for i, r in got)


@pytest.mark.parametrize("form,T,H,K", CALLS)
def test_captured_and_repeated(form, T, H, K):
    f = made(form, T, H, K, seed=60)
    first = f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = f()
    for _ in range(5):
        for x in r.values():
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(r, first) and same(f(), first)


def test_row_does_not_depend_on_its_batch():
    """A row of a batch in the wide form, alone in the narrow one: both within the definition's bounds, so within
    twice those of each other; equal bits within a form (a batch cut in two)."""
    rng = np.random.default_rng(70)
    q, k, ks, idx, sm, _ = attention_case(rng, 576, 512, 320, 64, 1, 140, 16, False, holes=False)
    ref = R.attention(f64(q)[:4], k, ks, idx[:4], sm)
    whole = call(q, k, ks, idx, sm)()
    assert torch.equal(whole["out"][:180], call(q[:180], k, ks, idx[:180], sm)()["out"])
    alone = call(q[:4], k, ks, idx[:4], sm)()
    d = (whole["out"][:4].float() - alone["out"].float()).abs().cpu().numpy()
    assert not (d > 2 * ref["out_tol"]).any()
    assert math.isclose(float(whole["lse"][0, 0]), float(alone["lse"][0, 0]), rel_tol=1e-5, abs_tol=1e-4)


@pytest.mark.parametrize("H,K", [(64, 64), (64, 200), (16, 64)])
def test_thousands_of_short_rows(H, K):
    """200 rows (a third of them empty) thirty times over: CTAs go from item to item; the copies have the same bits, and
    they are those of the definition within its bounds (200 rows alone may take the other form: other bits)."""
    rng = np.random.default_rng(80 + K + H)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 200, H, 1, K, 16, False)
    kw["length"] = np.where(np.arange(200) % 3 == 0, 0, kw["length"]).astype(np.int32)
    ref = R.attention(f64(q), k, ks, idx, sm, length=kw["length"])
    many = call(np.tile(q, (30, 1, 1)), k, ks, np.tile(idx, (30, 1)), sm, length=np.tile(kw["length"], 30))()
    for n in ("out", "lse", "lse_kv"):
        copies = many[n].view(30, 200, *many[n].shape[1:])
        assert bool((copies == copies[0]).all()), n
    o = many["out"][:200].float().cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all() and not (np.abs(o - ref["out"]) > ref["out_tol"]).any()
    g, r = many["lse"][:200].cpu().numpy().astype(np.float64), ref["lse"]
    fin = np.isfinite(r)
    assert np.array_equal(g[~fin], r[~fin]) and not (np.abs(g[fin] - r[fin]) > ref["lse_tol"][fin]).any()
