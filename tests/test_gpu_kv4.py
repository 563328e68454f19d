"""The 4-bit block cache on the GPU against its 64-bit definitions: writing (bit for
bit, untouched bytes included), reading back (bit for bit) and sparse attention over
it (within bounds that kv4_ref derives per element)."""
import math
import threading

import numpy as np
import pytest
import torch

import kv4_ref as R
import rows_ref
from gpu_util import DEV, cu_from_lengths, dev, dev_bf16, f64, rand_bf16_bits
from sparse_attention_gemm_gb300 import ops
from sparse_attention_gemm_gb300 import workloads as W
from test_gpu_kv8 import Pages, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    ops.device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert ops.device_status(clear=True) == 0, "a kernel raised a device status flag"


def cache_of(rng, n_blocks, block, heads, dim, lo=-4, hi=-1):
    codes = rng.integers(0, 256, (n_blocks, block, heads, dim // 2)).astype(np.uint8)
    return codes, (rng.integers(lo, hi + 1, (n_blocks, block, heads, dim // 32)) + 127).astype(np.uint8)


def check_write(g, src, codes, scale):
    c, s = dev(codes), dev(scale)
    ops.kv4_write(dev_bf16(src), c, s, dev(g.cu), **g.args())
    rc, rs = R.write(f64(src), codes, scale, g.cu, g.pos, g.table)
    assert np.array_equal(s.cpu().numpy(), rs), "scales"
    assert np.array_equal(c.cpu().numpy(), rc), "codes"


GEOMETRIES = [
    (1, 576, 64, [1], [0], True, 0),
    (1, 576, 64, [1, 1, 1, 1], [0, 63, 64, 100], True, 3),
    (1, 576, 64, [20, 1, 65, 0, 64], [5, 70, 0, 9, 64], True, 2),
    (1, 512, 128, [90, 17], [127, 1], True, 0),
    (2, 256, 16, [33, 16, 1, 15, 2], [3, 0, 15, 1, 14], True, 5),
    (3, 32, 4, [9, 2, 30], [2, 5, 0], False, 0),
    (1, 96, 256, [300], [77], False, 1),
    (1, 1024, 8, [21, 8], [4, 8], True, 0),
    (1, 128, 1, [1], [0], False, 0),
    (1024, 32, 2, [3], [1], True, 0),
    (2, 64, 32, [1] * 300, list(range(300)), True, 7),
]


@pytest.mark.parametrize("heads,dim,block,new,ctx,table,pad", GEOMETRIES)
def test_write(heads, dim, block, new, ctx, table, pad):
    rng = np.random.default_rng(sum(new) + dim)
    g = Pages(rng, new, ctx, block, table, pad)
    check_write(g, rows(rng, g.T, heads, dim, 3.0), *cache_of(rng, g.n_blocks, block, heads, dim))


def test_write_borders_and_special_values():
    """Borders between codes, infinities, NaN, zeros of both signs, the smallest and the largest bf16."""
    rng = np.random.default_rng(4)
    g = Pages(rng, [4, 5, 3, 6, 8], [0, 3, 2, 0, 5], 8)
    v = W.bf16_bits_to_f32(rows(rng, g.T, 2, 64)).copy()
    mid = (R.MAGNITUDES[1:] + R.MAGNITUDES[:-1]) / 2
    for i in range(4):
        v[i, 0, :32] = np.resize(np.concatenate([mid, -mid, R.MAGNITUDES, [6.0]]), 32) * 2.0 ** (3 * i - 5)
    v[4, 0, 3], v[5, 0, 5], v[5, 0, 40], v[6, 1, 0] = np.inf, -np.inf, np.nan, np.nan
    v[7, 0], v[7, 1] = 0.0, -0.0
    v[8, 0, :32] = np.inf
    v[9, 1] = np.nan
    v[10, 0, :4] = [1e-40, -3e-39, 9.2e-41, 0]
    v[10, 0, 4:] = 0
    v[11, 0], v[12, 0, 1] = 3.3895314e38, -3.3895314e38
    v[13, 0, :32] = 6 * 2.0 ** 125
    check_write(g, W.f32_to_bf16_bits(v), *cache_of(rng, g.n_blocks, 8, 2, 64))


def test_write_skips_unmapped_positions():
    rng = np.random.default_rng(5)
    g = Pages(rng, [40, 12, 9], [0, 30, 6], 8)
    g.table[0, 2], g.table[0, 3], g.table[1, 4] = -1, g.n_blocks, 1 << 30
    g.pos[2] = -5                                   # four tokens land at positions 0..3
    g.table = np.ascontiguousarray(g.table[:, :5])  # position 40 and later are beyond the table
    check_write(g, rows(rng, g.T, 1, 64), *cache_of(rng, g.n_blocks, 8, 1, 64))


def test_write_rows_of_one_block_in_two_calls():
    """Rows depend on themselves alone: two calls into one block, in any order, give what one gives."""
    rng = np.random.default_rng(6)
    x = dev_bf16(rows(rng, 40, 1, 576))
    made = []
    for parts in ([(0, 40)], [(13, 40), (0, 13)], [(0, 1), (1, 39), (39, 40)]):
        c, s = torch.zeros(1, 64, 1, 288, dtype=torch.uint8, device=DEV), torch.zeros(1, 64, 1, 18, dtype=torch.uint8, device=DEV)
        for a, b in parts:
            ops.kv4_write(x[a:b].contiguous(), c, s, dev(cu_from_lengths([b - a])), pos=dev(np.array([a], np.int32)))
        made.append((c, s))
    assert all(torch.equal(c, made[0][0]) and torch.equal(s, made[0][1]) for c, s in made[1:])
    # values read back are written as they are
    back = ops.kv4_read(*made[0], dev(cu_from_lengths([40])), 40)
    c, s = (torch.zeros_like(t) for t in made[0])
    ops.kv4_write(back, c, s, dev(cu_from_lengths([40])))
    assert torch.equal(ops.kv4_read(c, s, dev(cu_from_lengths([40])), 40), back)


@pytest.mark.parametrize("heads,dim,block,new,ctx,table,pad", GEOMETRIES + [(1, 576, 64, [5000, 2001], [100, 3], True, 0)])
def test_read(heads, dim, block, new, ctx, table, pad):
    rng = np.random.default_rng(sum(new) + dim + 1)
    g = Pages(rng, new, ctx, block, table, pad)
    codes, scale = cache_of(rng, g.n_blocks, block, heads, dim)
    at = rng.integers(0, scale.size, scale.size // 3)
    scale.reshape(-1)[at] = rng.integers(0, 256, at.size)  # every byte: the smallest, those beyond the range, NaN
    if table and g.table.shape[1] > 2:
        g.table[0, 1] = -1
        g.table[0, 2] = g.n_blocks + 5
    want = R.read(codes, scale, g.cu, g.pos, g.table, np.full((g.T, heads, dim), 7.0))
    out = torch.full((g.T, heads, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    got = ops.kv4_read(dev(codes), dev(scale), dev(g.cu), g.T, out=out, **g.args())
    assert got.data_ptr() == out.data_ptr()
    a = got.double().cpu().numpy()
    # (the fourth lowest magnitudes of byte 0, 2^-128, are bf16 too: nothing is rounded)
    assert np.array_equal(np.isnan(a), np.isnan(want)) and np.array_equal(a[~np.isnan(a)], want[~np.isnan(a)])


def test_read_shared_prefix():
    rng = np.random.default_rng(8)
    codes, scale = cache_of(rng, 6, 16, 1, 64)
    table = dev(np.array([[3, 1, 5], [3, 1, 0]], np.int32))
    out = ops.kv4_read(dev(codes), dev(scale), dev(cu_from_lengths([40, 35])), 75, block_table=table)
    assert torch.equal(out[:32], out[40:72]) and not torch.equal(out[32:35], out[72:75])


# ------------------------------------------------------------------- attention
def check_attention(q, k, ks, idx, sm, **kw):
    host = {n: kw.get(n) for n in ("length", "sink", "v4", "v_scale", "cu", "table")}
    ref = R.attention(f64(q), k, ks, idx, sm, **host)
    d = {n: (None if a is None else dev(a)) for n, a in host.items()}
    T, H = q.shape[:2]
    done = ref["done"]
    args = dict(topk_length=d["length"], sink=d["sink"], v4=d["v4"], v_scale=d["v_scale"], cu_seqlens=d["cu"],
                block_table=d["table"])
    out = torch.full((T, H, ref["out"].shape[2]), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    got = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, want_lse_kv=True, want_max_logits=True,
                                  out=out, lse=lse, **args)
    assert bool((out[dev(~done)] == 7.0).all()) and bool((lse[dev(~done)] == 7.0).all())
    bare = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, **args)
    assert set(bare) == {"out", "lse"}
    for r in (got, bare):
        o = r["out"].double().cpu().numpy()[done]
        over = np.abs(o - ref["out"][done]) - ref["out_tol"][done]
        assert np.isfinite(o).all() and not (over > 0).any(), f"{(over > 0).sum()} of {over.size} outputs out of tolerance"
        for n in r:
            if n == "out":
                continue
            g, want = r[n].double().cpu().numpy()[done], ref[n][done]
            fin = np.isfinite(want)
            assert np.array_equal(g[~fin], want[~fin]), n
            far = np.abs(g[fin] - want[fin]) - ref["lse_tol"][done][fin]
            assert not (far > 0).any(), f"{n}: {far.max():.3g} over its bound"
    return got


FORMS = [(576, 512), (512, 512), (256, 256)]


def attention_case(rng, dqk, dv, T, H, heads, K, block, table, n=None, holes=True):
    n = n or max(2 * K, 80)
    n_blocks = (n + block - 1) // block + 2
    k, ks = cache_of(rng, n_blocks, block, heads, dqk)
    kw = {}
    if dqk == 256:
        kw["v4"], kw["v_scale"] = cache_of(rng, n_blocks, block, heads, dv, -9, 3)
    q = rand_bf16_bits(rng, (T, H, dqk), 1.0)
    hi = n
    if table:
        per = n_blocks // 2 or 1
        kw["table"] = rng.permutation(n_blocks)[:2 * per].reshape(2, -1).astype(np.int32)
        kw["cu"] = cu_from_lengths([T // 3, T - T // 3])
        hi = kw["table"].shape[1] * block
    idx = rng.integers(0, hi, (T, K)).astype(np.int32)
    if holes:
        idx[rng.random((T, K)) < 0.1] = -1
        idx[rng.random((T, K)) < 0.02] = 1 << 30
        kw["length"] = rng.integers(-3, K + 9, T).astype(np.int32)
        if T > 2:
            idx[T // 2] = -1  # a row of nothing but holes
            kw["length"][T // 2], kw["length"][1] = K, 0
    return q, k, ks, idx, 1.0 / math.sqrt(dqk), kw


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,heads,K,block,table,sink", [
    (1, 1, 1, 1, 1, False, False),
    (1, 64, 1, 300, 64, True, True),
    (5, 64, 1, 64, 16, False, True),
    (7, 12, 1, 65, 32, True, False),
    (6, 24, 2, 130, 16, True, True),
    (9, 100, 1, 63, 4, False, True),
    (4, 128, 1, 257, 128, True, False),
    (3, 260, 4, 40, 256, False, True),
    (40, 16, 1, 33, 64, True, True),
    (3, 66, 2, 129, 1, False, False),
])
def test_attention(dqk, dv, T, H, heads, K, block, table, sink):
    rng = np.random.default_rng(T * 1000 + H + K + dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, heads, K, block, table)
    if sink:
        kw["sink"] = rng.standard_normal(H).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


def test_attention_leaves_padding_rows():
    rng = np.random.default_rng(77)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 9, 64, 1, 90, 16, True)
    kw["cu"] = cu_from_lengths([2, 4])
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H", [(1, 64), (2, 16), (3, 128)])
def test_attention_long_rows_of_few_queries(dqk, dv, T, H):
    """A few queries over 2048 slots: the slots are split between CTAs and joined."""
    rng = np.random.default_rng(dqk + T)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, 2048, 64, False, n=5000, holes=T > 1)
    check_attention(q, k, ks, idx, sm, sink=rng.standard_normal(H).astype(np.float32), **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("H", [6, 40])
def test_attention_many_rows(dqk, dv, H):
    """More rows than CTAs, lengths from none to three tiles."""
    rng = np.random.default_rng(dqk + 9)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, 500, H, 1, 170, 16, True)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K,table", [(1, 16, 8192, True), (2, 5, 6200, False), (80, 12, 1100, True), (9, 40, 1500, False)])
def test_attention_long_rows_of_few_heads(dqk, dv, T, H, K, table):
    """Few heads and rows too long for a cluster, and more rows of few heads than clusters: groups of 64 heads, and of 16."""
    rng = np.random.default_rng(K + dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, 32, table, n=3000, holes=T > 2)
    check_attention(q, k, ks, idx, sm, sink=rng.standard_normal(H).astype(np.float32), **kw)


# (110 rows of more than 16 heads: groups of 64 heads, whole; a dozen of many slots: the same in splits)
@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,heads,K,block,table,sink", [
    (110, 100, 1, 150, 16, True, True),
    (90, 48, 1, 350, 64, False, True),
    (60, 130, 2, 200, 4, True, False),
    (160, 64, 1, 64, 32, True, True),
    (40, 64, 1, 350, 16, True, False),
    (12, 128, 1, 1500, 64, True, True),
    (9, 40, 1, 2000, 1, False, False),
    (50, 17, 1, 65, 1, False, True),
    (170, 17, 1, 1, 1, False, True),
])
def test_attention_in_groups_of_64(dqk, dv, T, H, heads, K, block, table, sink):
    rng = np.random.default_rng(T * 1000 + H + K + dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, heads, K, block, table)
    if sink:
        kw["sink"] = rng.standard_normal(H).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("T,H", [(6, 12), (110, 64), (10, 128)])
@pytest.mark.parametrize("lo,hi", [(-60, -50), (-30, 4), (40, 60), (-100, 60), (-126, -90)])
def test_attention_values_of_every_size(lo, hi, T, H):
    """Value scales that differ by many powers of two (keys of one size, so that scores stay finite)."""
    rng = np.random.default_rng(200 + hi)
    q, k, ks, idx, sm, kw = attention_case(rng, 256, 256, T, H, 1, 1500 if T == 10 else 200, 4, False, holes=False)
    kw["v_scale"] = (rng.integers(lo, hi + 1, kw["v_scale"].shape) + 127).astype(np.uint8)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H,K", [(4, 12, 512), (4, 64, 512), (100, 64, 512), (12, 64, 1500)])
def test_attention_rising_and_falling_scores(dqk, dv, T, H, K):
    """The running maximum moves in many tiles: keys in order of their scores, up and down."""
    rng = np.random.default_rng(dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, 1, False, holes=False)
    s = f64(q)[:, 0] @ R.values(k[:, 0, 0], ks[:, 0, 0]).T
    for t in range(T):
        order = np.argsort(s[t])[:: 1 if t % 2 else -1]
        idx[t] = order[np.linspace(0, order.size - 1, idx.shape[1]).astype(int)]
    check_attention(q, k, ks, idx, 4 * sm, **kw)


def test_attention_peaked_row():
    """One key far above the rest whose value is tiny, the others' large: nothing of the small weights is lost."""
    rng = np.random.default_rng(90)
    for T, H in ((3, 12), (3, 64), (130, 64)):
        q, k, ks, idx, sm, kw = attention_case(rng, 256, 256, T, H, 1, 150, 1, False, holes=False)
        q[:] = W.f32_to_bf16_bits(np.ones(q.shape, np.float32))
        k[:], ks[:] = 0, 127
        k[5] = 0x22                    # the value 1 in every element: a score of 256 sm = 16
        kw["v_scale"][:] = 127 + 10
        kw["v_scale"][5] = 127 - 20
        idx[idx == 5] = 6
        idx[:, 70] = 5
        check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("T,H", [(6, 20), (6, 60), (120, 60)])
def test_attention_never_uses_unselected_rows(dqk, dv, T, H):
    """NaN scales in rows that no valid slot names, the slots behind topk_length among them."""
    rng = np.random.default_rng(dqk + 3)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, 90, 1, False, n=400 if T == 6 else 12000)
    used = np.zeros(k.shape[0], bool)
    for t in range(T):
        i = idx[t, :max(0, min(int(kw["length"][t]), 90))]
        used[i[(i >= 0) & (i < k.shape[0])]] = True
    assert not used.all()
    spoilt = dict(kw)
    ks2 = ks.copy()
    ks2[~used] = 255
    if dqk == 256:
        spoilt["v_scale"] = kw["v_scale"].copy()
        spoilt["v_scale"][~used] = 255
    a = check_attention(q, k, ks, idx, sm, **kw)
    b = check_attention(q, k, ks2, idx, sm, **spoilt)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("T,H", [(4, 16), (4, 64), (130, 64)])
def test_attention_nan_reaches_only_its_rows(T, H):
    """A NaN scale in a selected row, and a query head with NaN or infinity, give NaN there and nowhere else."""
    rng = np.random.default_rng(21)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, T, H, 1, 70, 1, False, holes=False)
    hit = idx[0, 5]
    idx[1:][idx[1:] == hit] = (hit + 1) % k.shape[0]
    clean = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(ks), dev(idx), sm)["out"]
    bad = ks.copy()
    bad[hit, 0, 0, 17] = 255  # key-only dims: every score of that slot
    got = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(bad), dev(idx), sm)
    assert bool(got["out"][0].isnan().all()) and bool(got["lse"][0].isnan().all()) and torch.equal(got["out"][1:], clean[1:])
    q2 = dev_bf16(q)
    q2[2, 7, 3], q2[3, 9, 500] = float("nan"), float("inf")
    got = ops.sparse_attn_fwd_kv4(q2, dev(k), dev(ks), dev(idx), sm)["out"]
    hit = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    hit[2, 7] = hit[3, 9] = True
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("T,H", [(30, 16), (30, 64), (130, 64)])
def test_attention_is_that_of_the_bf16_call_on_values_read_back(T, H):
    """The cache's values are bf16 ones: both calls round weights (2^-8) and out (2^-8), nothing else."""
    rng = np.random.default_rng(30)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, T, H, 1, 200, 16, False)
    n = k.shape[0] * 16
    kv = ops.kv4_read(dev(k), dev(ks), dev(cu_from_lengths([n])), n).view(n, 576)
    a = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, topk_length=dev(kw["length"]))
    b = ops.sparse_attn_fwd(dev_bf16(q), kv, dev(idx), sm, topk_length=dev(kw["length"]))
    d = (a["out"].float() - b["out"].float()).norm() / b["out"].float().norm()
    assert float(d) <= 4 * 2.0 ** -8
    fin = torch.isfinite(b["lse"])
    assert torch.equal(fin, torch.isfinite(a["lse"])) and float((a["lse"] - b["lse"])[fin].abs().max()) <= 1e-3


def test_attention_offsets_beyond_32_bits():
    """Rows behind the cache's first 4 GiB."""
    rng = np.random.default_rng(31)
    block, n_blocks = 64, 240000
    cache = torch.zeros((n_blocks, block, 1, 288), dtype=torch.uint8, device=DEV)
    scale = torch.full((n_blocks, block, 1, 18), 127, dtype=torch.uint8, device=DEV)
    k, ks = cache_of(rng, 4, block, 1, 576)
    at = [0, 1, n_blocks - 2, n_blocks - 1]
    for i, b in enumerate(at):
        cache[b], scale[b] = dev(k[i]), dev(ks[i])
    idx = rng.integers(0, 4 * block, (130, 150)).astype(np.int32)
    far = (np.array(at)[idx // block] * block + idx % block).astype(np.int32)
    for T, H in ((3, 16), (3, 64), (130, 64)):  # (groups of 16 heads, and of 64)
        q = dev_bf16(rand_bf16_bits(rng, (T, H, 576)))
        a = ops.sparse_attn_fwd_kv4(q, cache, scale, dev(far[:T]), 0.04)
        b = ops.sparse_attn_fwd_kv4(q, dev(k), dev(ks), dev(idx[:T]), 0.04)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    table, pos = dev(np.array([at], np.int32)), dev(np.array([40], np.int32))
    cu = dev(cu_from_lengths([200]))
    back = ops.kv4_read(cache, scale, cu, 200, pos=pos, block_table=table)
    want = ops.kv4_read(dev(k), dev(ks), cu, 200, pos=pos)
    assert torch.equal(back, want)
    ops.kv4_write(back, cache, scale, cu, pos=pos, block_table=table)
    assert torch.equal(ops.kv4_read(cache, scale, cu, 200, pos=pos, block_table=table), want)


@pytest.mark.parametrize("T,H", [(33, 16), (33, 128), (150, 128)])
def test_repeated_calls_give_the_same_bits(T, H):
    rng = np.random.default_rng(32)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, T, H, 1, 300, 16, False)
    a = [dev_bf16(q), dev(k), dev(ks), dev(idx), sm]
    first = ops.sparse_attn_fwd_kv4(*a, topk_length=dev(kw["length"]))
    for _ in range(20):
        again = ops.sparse_attn_fwd_kv4(*a, topk_length=dev(kw["length"]))
        assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


@pytest.mark.parametrize("dqk,dv", FORMS)
@pytest.mark.parametrize("H,table", [(40, True), (64, False), (128, True)])
def test_attention_over_a_cache_widened_once(dqk, dv, H, table):
    """Many slots of a small cache: its values go through bf16 rows.  Lengths, holes, a padded batch; a few rows against
    their definition, every row against the tiles' own conversion (the same call on a part of the rows)."""
    rng = np.random.default_rng(dqk + H)
    T, K, block = 700, 700, 16
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, 1, K, block, table, n=900)
    ks.reshape(-1)[rng.integers(0, ks.size, 5)] = 131  # a few blocks of large values
    assert ops.sparse_attn_fwd_kv4_workspace_size(T, H, 1, dqk, dv, K, block, k.shape[0], table) >= k.shape[0] * block * dqk * 2
    if table:
        kw["cu"] = cu_from_lengths([300, 350])  # 50 padding rows
    kw["sink"] = rng.standard_normal(H).astype(np.float32)
    d = {n: (dev(kw[n]) if n in kw else None) for n in ("v4", "v_scale", "cu", "table", "sink")}
    out = torch.full((T, H, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    args = dict(v4=d["v4"], v_scale=d["v_scale"], sink=d["sink"], block_table=d["table"])
    got = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, topk_length=dev(kw["length"]), cu_seqlens=d["cu"],
                                  want_lse_kv=True, want_max_logits=True, out=out, lse=lse, **args)
    done = int(kw["cu"][-1]) if table else T
    assert bool((out[done:] == 7.0).all()) and bool((lse[done:] == 7.0).all())
    rows = np.array([0, 1, 5, 299, 300, T // 2, 600, 649])
    seq = np.searchsorted(kw["cu"], rows, side="right") - 1 if table else None
    for i, t in enumerate(rows):
        part = {n: kw[n] for n in ("sink", "v4", "v_scale") if n in kw}
        if table:
            part.update(table=kw["table"][seq[i]:seq[i] + 1], cu=np.array([0, 1], np.int32))
        ref = R.attention(f64(q[t:t + 1]), k, ks, idx[t:t + 1], sm, length=kw["length"][t:t + 1], **part)
        assert not (np.abs(got["out"][t].double().cpu().numpy() - ref["out"][0]) > ref["out_tol"][0]).any(), t
        for n in ("lse", "lse_kv", "max_logits"):
            g, want = got[n][t].double().cpu().numpy(), ref[n][0]
            fin = np.isfinite(want)
            # (an empty row's lse is the sink, which this form takes to powers of two and back: two products and two
            # rounded constants, 4 * 2^-24 of it)
            tol = np.maximum(ref["lse_tol"][0], 2.0 ** -22 * np.abs(kw["sink"]))
            assert np.array_equal(g[~fin], want[~fin]) and not (np.abs(g[fin] - want[fin]) > tol[fin]).any(), (n, t)
    # rows 100..139 alone: too few slots to widen the cache for
    part = slice(100, 140)
    few = ops.sparse_attn_fwd_kv4(dev_bf16(q[part]), dev(k), dev(ks), dev(idx[part]), sm, topk_length=dev(kw["length"][part]),
                                  cu_seqlens=dev(cu_from_lengths([40, 0])) if table else None, **args)
    a, b = got["out"][part].float(), few["out"].float()
    assert float((a - b).norm() / b.norm()) <= 4 * 2.0 ** -8  # each rounds weights and out (2^-8)
    fin = torch.isfinite(few["lse"])
    assert torch.equal(fin, torch.isfinite(got["lse"][part])) and float((few["lse"] - got["lse"][part])[fin].abs().max()) <= 1e-3
    again = ops.sparse_attn_fwd_kv4(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, topk_length=dev(kw["length"]), cu_seqlens=d["cu"], **args)
    assert torch.equal(again["out"][:done], got["out"][:done]) and torch.equal(again["lse"][:done], got["lse"][:done])


def test_widened_cache_never_uses_unselected_rows():
    rng = np.random.default_rng(70)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 650, 64, 1, 640, 1, False, n=1300)
    idx[(idx >= 0) & (idx % 7 == 3)] = 4
    spoilt = ks.copy()
    spoilt[np.arange(k.shape[0]) % 7 == 3] = 255
    a = [dev_bf16(q), dev(k)]
    assert ops.sparse_attn_fwd_kv4_workspace_size(650, 64, 1, 576, 512, 640, 1, k.shape[0]) > 0
    x = ops.sparse_attn_fwd_kv4(*a, dev(ks), dev(idx), sm, topk_length=dev(kw["length"]))
    y = ops.sparse_attn_fwd_kv4(*a, dev(spoilt), dev(idx), sm, topk_length=dev(kw["length"]))
    assert torch.equal(x["out"], y["out"]) and torch.equal(x["lse"], y["lse"]) and bool(torch.isfinite(y["out"]).all())


def test_empty_calls():
    k, ks = cache_of(np.random.default_rng(1), 2, 4, 1, 576)
    c, s = dev(k), dev(ks)
    cu = dev(cu_from_lengths([0]))
    ops.kv4_write(torch.empty((0, 1, 576), dtype=torch.bfloat16, device=DEV), c, s, cu)
    assert ops.kv4_read(c, s, cu, 0).shape == (0, 1, 576)
    q = torch.ones((3, 5, 576), dtype=torch.bfloat16, device=DEV)
    r = ops.sparse_attn_fwd_kv4(q, c, s, torch.empty((3, 0), dtype=torch.int32, device=DEV), 0.1)
    assert bool((r["out"] == 0).all()) and bool((r["lse"] == -math.inf).all())
    r = ops.sparse_attn_fwd_kv4(q[:0], c, s, torch.empty((0, 4), dtype=torch.int32, device=DEV), 0.1)
    assert r["out"].shape == (0, 5, 512)
    assert np.array_equal(c.cpu().numpy(), k)


def test_forced_wait_timeout_aborts_cleanly():
    """Groups of 64 heads: every wait that is not already satisfied gives up, the call returns, says so, and the next
    ones are exact.  Smaller groups wait for nothing: their results are the same under any limit."""
    rng = np.random.default_rng(50)
    for T, H, K, waits in ((300, 64, 300, True), (20, 64, 2048, True), (300, 12, 300, False), (1, 64, 2048, False)):
        q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, T, H, 1, K, 16, False, holes=False)
        a = [dev_bf16(q), dev(k), dev(ks), dev(idx), sm]
        want = ops.sparse_attn_fwd_kv4(*a)
        torch.cuda.synchronize()
        assert ops.device_status(clear=True) == 0
        ops.set_wait_limit_ns(1)
        try:
            got = ops.sparse_attn_fwd_kv4(*a)
            torch.cuda.synchronize()
            st = ops.device_status(clear=True)
            if waits:
                assert st & ops.DSA_STATUS_WAIT_TIMEOUT and not st & ops.DSA_STATUS_DRAIN_TIMEOUT, f"{st:#x}"
            else:
                assert st == 0 and torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
        finally:
            ops.set_wait_limit_ns(0)
        ops.device_status(clear=True)
        again = ops.sparse_attn_fwd_kv4(*a)
        assert torch.equal(again["out"], want["out"]) and torch.equal(again["lse"], want["lse"])
        assert ops.device_status(clear=True) == 0


def test_captured_steps_with_their_own_workspaces():
    rng = np.random.default_rng(41)
    made = []
    for T, H, K in ((2, 64, 700), (5, 64, 300), (40, 12, 100)):
        q, k, ks, idx, sm, _ = attention_case(rng, 576, 512, T, H, 1, K, 32, False, holes=False)
        st = {"q": dev_bf16(q), "k": dev(k), "s": dev(ks), "idx": dev(idx), "cu": dev(cu_from_lengths([T])),
              "pos": dev(np.array([37], np.int32)), "src": dev_bf16(rows(rng, T, 1, 576))}
        n = ops.sparse_attn_fwd_kv4_workspace_size(T, H, 1, 576, 512, K, 32, k.shape[0])
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)

        def step(st=st, sm=sm):
            ops.kv4_write(st["src"], st["k"], st["s"], st["cu"], pos=st["pos"])
            return ops.sparse_attn_fwd_kv4(st["q"], st["k"], st["s"], st["idx"], sm, workspace=st["ws"])

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st["res"] = step()
        made.append((graph, st, step))
    side = torch.cuda.Stream()
    for r in range(3):
        for graph, st, step in made:
            st["q"].copy_(torch.randn_like(st["q"].float()).to(torch.bfloat16))
            st["src"].copy_(torch.randn_like(st["src"].float()).to(torch.bfloat16))
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side if r == 1 else torch.cuda.current_stream()):
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
            out, lse = st["res"]["out"].clone(), st["res"]["lse"].clone()
            eager = step()
            assert torch.equal(out, eager["out"]) and torch.equal(lse, eager["lse"])


def test_threads_with_streams_of_their_own():
    """Calls of several host threads at once, each on a stream of its own: the results of one after another."""
    rng = np.random.default_rng(43)
    f, _ = ops.rotary_inv_freq(64)
    calls = []
    for T, H, heads, K, d, v in ((3, 128, 1, 900, 576, 512), (1, 16, 1, 2048, 512, 512), (30, 12, 1, 300, 256, 256),
                                 (400, 64, 1, 1024, 576, 512), (2, 64, 1, 7000, 576, 512)):
        q, k, ks, idx, sm, kw = attention_case(rng, d, v, T, H, heads, K, 32, T == 400, n=2000, holes=False)
        args = (dev_bf16(q), dev(k), dev(ks), dev(idx), sm)
        kw = {("cu_seqlens" if n == "cu" else "block_table" if n == "table" else n): dev(a) for n, a in kw.items()}
        x, g = dev_bf16(rows(rng, 500, 1, 264))[:, 0], dev_bf16(rows(rng, 500, 1, 264))[:, 0]
        w, cu = torch.ones(264, device=DEV), dev(cu_from_lengths([100, 400]))
        turned = dev_bf16(rows(rng, 500, 9, 64))

        def call(args=args, kw=kw, x=x, g=g, w=w, cu=cu, turned=turned):
            a = ops.sparse_attn_fwd_kv4(*args, **kw)
            n = ops.rms_norm_fwd(x, w, 1e-6, residual=g, want_rstd=True)
            b = ops.rms_norm_bwd(g, n["sum"], w, n["rstd"])
            r = ops.rotary(turned, f, cu, x2=turned[:, :1])
            c, s = torch.zeros(8, 64, 9, 32, dtype=torch.uint8, device=DEV), torch.zeros(8, 64, 9, 2, dtype=torch.uint8, device=DEV)
            ops.kv4_write(r[0], c, s, cu)
            return [a["out"], a["lse"], n["out"], b["dx"], b["dweight"], r[0], r[1], c, s, ops.kv4_read(c, s, cu, 500)]
        calls.append(call)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for r in range(12):
                    j = (i + r) % len(calls)
                    got = calls[j]()
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[j])):
                        failed.append((i, r, j))
        except Exception as e:  # (reported by the test's own thread)
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_a_layers_step_together():
    """Prompt and decode steps: latent rows normed, their last 64 rotated with the queries', written into the 4-bit
    cache, normed indexer rows in 8 bits to the indexer's top-k, attention over the selected positions; and the
    gradient's way back through rotary and norm."""
    rng = np.random.default_rng(40)
    n_seqs, slot, block, Hi, H, K = 3, 256, 64, 32, 64, 48
    per = slot // block
    table = rng.permutation(n_seqs * per + 2)[:n_seqs * per].reshape(n_seqs, per).astype(np.int32)
    kv = torch.full((n_seqs * per + 2, block, 1, 288), 17, dtype=torch.uint8, device=DEV)
    kvs = torch.full((n_seqs * per + 2, block, 1, 18), 255, dtype=torch.uint8, device=DEV)
    ki8 = torch.zeros((n_seqs * slot, 128), dtype=torch.uint8, device=DEV)
    kis = torch.ones(n_seqs * slot, device=DEV)
    cu_k, dt = dev((np.arange(n_seqs + 1) * slot).astype(np.int32)), dev(table)
    f, mul = ops.rotary_inv_freq(64, scaling="yarn", factor=40.0)
    w_kv, w_i = (torch.from_numpy((1 + 0.1 * rng.standard_normal(n)).astype(np.float32)).to(DEV) for n in (512, 128))
    have = np.zeros(n_seqs, np.int32)
    for new in ([100, 37, 64], [1, 1, 1], [1, 1, 1], [30, 1, 0]):
        T, cu = sum(new), cu_from_lengths(new)
        dcu, pos = dev(cu), dev(have)
        proj = dev_bf16(rows(rng, T, 1, 576))[:, 0]
        q = dev_bf16(rand_bf16_bits(rng, (T, H, 576)))
        at = positions = [int(have[b]) + t - int(cu[b]) for b in range(n_seqs) for t in range(cu[b], cu[b + 1])]
        row = torch.empty(T, 576, dtype=torch.bfloat16, device=DEV)
        n = ops.rms_norm_fwd(proj[:, :512], w_kv, 1e-6, out=row[:, :512], want_rstd=True)
        q0 = q.clone()
        ops.rotary(q[..., 512:], f, dcu, pos=pos, x2=proj[:, None, 512:], mul=mul, out=q[..., 512:], out2=row[:, None, 512:])
        h, rstd, y = rows_ref.norm(proj[:, :512].double().cpu().numpy(), w_kv.double().cpu().numpy(), 1e-6)
        assert (np.abs(row[:, :512].double().cpu().numpy() - y) <= rows_ref.norm_bounds(h, rstd, y)[2]).all()
        want, tol = rows_ref.rotary(q0[..., 512:].double().cpu().numpy(), f.cpu().numpy(), at, True, False, mul)
        assert (np.abs(q[..., 512:].double().cpu().numpy() - want) <= tol).all() and torch.equal(q[..., :512], q0[..., :512])
        before_c, before_s = kv.cpu().numpy(), kvs.cpu().numpy()
        ops.kv4_write(row.view(T, 1, 576), kv, kvs, dcu, pos=pos, block_table=dt)
        rc, rs = R.write(row.double().cpu().numpy()[:, None], before_c, before_s, cu, have, table)
        assert np.array_equal(kv.cpu().numpy(), rc) and np.array_equal(kvs.cpu().numpy(), rs)
        # indexer: keys and queries as 8-bit rows with a scale each
        ki = ops.rms_norm_fwd(dev_bf16(rows(rng, T, 1, 128))[:, 0], w_i, 1e-6, fmt="e4m3")
        slots = torch.from_numpy(np.array([b * slot + p for b in range(n_seqs) for p in positions[cu[b]:cu[b + 1]]], np.int64)).to(DEV)
        ki8[slots], kis[slots] = ki["out"], ki["scale"][:, 0]
        qi = ops.rms_norm_fwd(dev_bf16(rows(rng, T * Hi, 1, 128))[:, 0], w_i, 1e-6, fmt="e4m3")
        w = torch.from_numpy((rng.random((T, Hi)) / 8).astype(np.float32)).to(DEV)
        top = ops.indexer_topk_fp8(qi["out"].view(T, Hi, 128), ki8, qi["scale"].view(T, Hi), kis, w, dcu, cu_k, pos, 1, K, slot)
        start = torch.repeat_interleave(torch.arange(n_seqs, device=DEV, dtype=torch.int32) * slot, dev(np.array(new)))
        local = torch.where(top["idx"] >= 0, top["idx"] - start[:, None], -1).contiguous()
        length = top["topk_length"].cpu().numpy()
        assert np.array_equal(length, np.minimum(np.array(at) + 1, K))
        got = ops.sparse_attn_fwd_kv4(q, kv, kvs, local, 1 / 24, topk_length=top["topk_length"], cu_seqlens=dcu, block_table=dt)
        ref = R.attention(q.double().cpu().numpy(), rc, rs, local.cpu().numpy(), 1 / 24, length=length, cu=cu, table=table)
        assert not (np.abs(got["out"].double().cpu().numpy() - ref["out"]) > ref["out_tol"]).any()
        assert not (np.abs(got["lse"].double().cpu().numpy() - ref["lse"]) > ref["lse_tol"]).any()
        # back: the row's gradient through rotary and norm into that of the projection
        g = dev_bf16(rows(rng, T, 1, 576))[:, 0]
        d_proj = torch.empty_like(g)
        back = ops.rms_norm_bwd(g[:, :512], proj[:, :512], w_kv, n["rstd"], dx=d_proj[:, :512])
        ops.rotary(g[:, None, 512:], f, dcu, pos=pos, mul=mul, inverse=True, out=d_proj[:, None, 512:])
        dx, dw, tx, tw = rows_ref.norm_back(*(t.double().cpu().numpy() for t in (g[:, :512], proj[:, :512], w_kv, n["rstd"])))
        turned, tt = rows_ref.rotary(g[:, None, 512:].double().cpu().numpy(), f.cpu().numpy(), at, True, True, mul)
        d = d_proj.double().cpu().numpy()
        assert (np.abs(d[:, :512] - dx) <= tx).all() and (np.abs(d[:, None, 512:] - turned) <= tt).all()
        assert (np.abs(back["dweight"].double().cpu().numpy() - dw) <= tw).all()
        have = (have + np.array(new)).astype(np.int32)


def test_binding_refuses():
    k, ks = cache_of(np.random.default_rng(1), 4, 8, 1, 576)
    c, s, cu = dev(k), dev(ks), dev(cu_from_lengths([3]))
    x = torch.zeros((3, 1, 576), dtype=torch.bfloat16, device=DEV)
    q, idx = torch.zeros((2, 4, 576), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 8), dtype=torch.int32, device=DEV)
    for bad in (lambda: ops.kv4_write(x[:, :, :512], c, s, cu), lambda: ops.kv4_write(x, c, s[:3].contiguous(), cu),
                lambda: ops.kv4_write(x, c.transpose(0, 1), s, cu), lambda: ops.kv4_write(x, c, s, cu, pos=cu),
                lambda: ops.kv4_write(x, c, s[..., :17].contiguous(), cu),
                lambda: ops.kv4_write(x, c, s, cu, block_table=dev(np.zeros((2, 2), np.int32))),
                lambda: ops.kv4_read(c, s, cu, 3, out=x[:2]), lambda: ops.kv4_read(c, s, cu, 2, out=x),
                lambda: ops.sparse_attn_fwd_kv4(q, c, s, idx[:1], 0.1),
                lambda: ops.sparse_attn_fwd_kv4(q, c, s, idx, 0.1, v4=c),
                lambda: ops.sparse_attn_fwd_kv4(q, c, s, idx, 0.1, sink=torch.zeros(3, device=DEV)),
                lambda: ops.sparse_attn_fwd_kv4(q, c, s, idx, 0.1, block_table=dev(np.zeros((1, 2), np.int32))),
                lambda: ops.sparse_attn_fwd_kv4(q[:, :, :512].contiguous(), c, s, idx, 0.1),
                lambda: ops.sparse_attn_fwd_kv4(q, c, s, idx, -1.0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.kv4_write(x.float(), c, s, cu), lambda: ops.kv4_write(x, c.to(torch.int8), s, cu),
                lambda: ops.kv4_write(x, c, s.float(), cu), lambda: ops.kv4_read(c, s, cu.long(), 3),
                lambda: ops.sparse_attn_fwd_kv4(q, c, s, idx.long(), 0.1)):
        with pytest.raises(TypeError):
            bad()
