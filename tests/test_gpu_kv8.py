"""The 8-bit block cache on the GPU against its 64-bit definitions: writing
(bit for bit, untouched bytes included), reading back (bit for bit) and sparse
attention over it (within bounds that kv8_ref derives per element)."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as R
import oracle
from gpu_util import DEV, cu_from_lengths, dev, dev_bf16, f64, rand_bf16_bits
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


def same_codes(a, b):
    """Equal codes; all NaN codes are one."""
    a, b = np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b)
    return np.array_equal(a, b)


class Pages:
    """A drawn geometry: sequences with earlier positions, a shuffled block table or flat slots."""

    def __init__(self, rng, new, ctx, block, table=True, pad=0, spare=3):
        self.new, self.block, self.T = np.asarray(new), block, int(sum(new)) + pad
        self.cu = cu_from_lengths(new)
        need = [(c + n + block - 1) // block for c, n in zip(ctx, new)]
        self.n_blocks = sum(need) + spare
        self.pos = np.asarray(ctx, np.int32)
        self.table = None
        if table:
            order = rng.permutation(self.n_blocks).astype(np.int32)
            self.table = np.full((len(new), max(max(need), 1)), -1, np.int32)
            at = 0
            for i, k in enumerate(need):
                self.table[i, :k] = order[at:at + k]
                at += k
        else:
            first = np.concatenate([[0], np.cumsum(need)[:-1]]) * block
            self.pos = (self.pos + first).astype(np.int32)

    def args(self):
        return dict(pos=dev(self.pos), block_table=None if self.table is None else dev(self.table))


def rows(rng, n, heads, dim, spread=1.0):
    x = rng.standard_normal((n, heads, dim)) * np.exp2(rng.uniform(-spread, spread, (n, 1, 1)))
    return W.f32_to_bf16_bits(x.astype(np.float32))


def cache_of(rng, n_blocks, block, heads, dim, lo=-9, hi=-5):
    codes = rng.integers(0, 256, (n_blocks, block, heads, dim)).astype(np.uint8)
    codes = np.where((codes & 127) == 127, codes & 0x80, codes).astype(np.uint8)
    scale = np.exp2(rng.integers(lo, hi + 1, (n_blocks, heads))).astype(np.float32)
    return codes, scale


def check_write(g, src, codes, scale, heads, dim):
    c, s = dev(codes), dev(scale)
    ops.kv8_write(dev_bf16(src), c, s, dev(g.cu), **g.args())
    rc, rs = R.write(f64(src), codes, scale, g.cu, g.pos, g.table)
    assert np.array_equal(s.cpu().numpy(), rs), "scales"
    assert same_codes(c.cpu().numpy(), rc), "codes"


# ----------------------------------------------------------------------- write
@pytest.mark.parametrize("heads,dim,block,new,ctx,table,pad", [
    (1, 576, 64, [1], [0], True, 0),
    (1, 576, 64, [1, 1, 1, 1], [0, 63, 64, 100], True, 3),
    (1, 576, 64, [200, 1, 65, 0, 64], [5, 70, 0, 9, 64], True, 2),
    (1, 512, 128, [300, 17], [127, 1], True, 0),
    (2, 256, 16, [33, 16, 1, 15, 2], [3, 0, 15, 1, 14], True, 5),
    (3, 32, 4, [9, 2, 30], [2, 5, 0], False, 0),
    (1, 16, 256, [600], [77], False, 1),
    (1, 1024, 8, [21, 8], [4, 8], True, 0),
    (64, 128, 1, [37, 5], [0, 11], True, 0),
    (1, 128, 1, [1], [0], False, 0),
    (1024, 16, 2, [3], [1], True, 0),
    (2, 48, 32, [1] * 300, list(range(300)), True, 7),
])
def test_write(heads, dim, block, new, ctx, table, pad):
    rng = np.random.default_rng(sum(new) + dim)
    g = Pages(rng, new, ctx, block, table, pad)
    codes, scale = cache_of(rng, g.n_blocks, block, heads, dim, -14, -4)  # some scales grow, some do not
    check_write(g, rows(rng, g.T, heads, dim, 3.0), codes, scale, heads, dim)


def test_write_rows_only():
    """block 1, no table, no positions: row t of the batch is row t of the cache."""
    rng = np.random.default_rng(3)
    T, Hi, d = 50, 32, 128
    x = rows(rng, T, Hi, d, 8.0)
    x[7, 3] = 0
    c = torch.full((T, 1, Hi, d), 7, dtype=torch.uint8, device=DEV)
    s = torch.full((T, Hi), 7.0, device=DEV)
    ops.kv8_write(dev_bf16(x), c, s, dev(cu_from_lengths([20, 0, 29])))  # the last token is padding
    v = f64(x)
    want = np.array([[R.scale_of(np.abs(v[t, h]).max()) for h in range(Hi)] for t in range(T)])
    want[49] = 7.0
    codes = np.concatenate([R.to_codes(v[:49] / want[:49, :, None]), np.full((1, Hi, d), 7, np.uint8)])
    assert np.array_equal(s.cpu().numpy(), want.astype(np.float32))
    assert np.array_equal(c.cpu().numpy()[:, 0], codes)


def test_write_special_values():
    """Infinities, NaN, zeros, the smallest and the largest bf16; a scale that is no power of two."""
    rng = np.random.default_rng(4)
    g = Pages(rng, [4, 5, 3, 6, 8], [0, 3, 2, 0, 5], 8)
    x = rows(rng, g.T, 2, 32)
    v = W.bf16_bits_to_f32(x).copy()
    v[0, 0, 3], v[1, 0, 5], v[2, 1, 0] = np.inf, -np.inf, np.nan
    v[4:9, 0] = 0.0
    v[9:12, 1] = np.nan
    v[12, 0, :4] = [1e-40, -3e-39, 9.2e-41, 0]
    v[12, 0, 4:] = 0
    v[13:18, 0] = 0
    v[18:, 0, 0] = 3.3895314e38
    v[18:, 1] = 448.0 * 2.0 ** -3
    codes, scale = cache_of(rng, g.n_blocks, 8, 2, 32)
    codes[g.table[1, 0], 1, 0, 4] = 127  # an earlier NaN code stays NaN when its block is rescaled
    scale[g.table[1, 0]] = 1e-30
    scale[g.table[4, 0]] = 0.3
    check_write(g, W.f32_to_bf16_bits(v), codes, scale, 2, 32)


def test_write_skips_unmapped_positions():
    rng = np.random.default_rng(5)
    g = Pages(rng, [40, 12, 9], [0, 30, 6], 8)
    g.table[0, 2] = -1
    g.table[0, 3] = g.n_blocks
    g.table[1, 4] = 1 << 30
    g.pos[2] = -5                                   # four tokens land at positions 0..3
    g.table = np.ascontiguousarray(g.table[:, :5])  # position 40 and later are beyond the table
    codes, scale = cache_of(rng, g.n_blocks, 8, 1, 64, -14, -4)
    check_write(g, rows(rng, g.T, 1, 64), codes, scale, 1, 64)


def test_write_then_read_is_exact_and_repeatable():
    """Writing the values read back changes nothing; a second write of the same rows neither."""
    rng = np.random.default_rng(6)
    g = Pages(rng, [100, 31, 7], [0, 0, 0], 32)
    src = dev_bf16(rows(rng, g.T, 2, 256))
    c = torch.zeros((g.n_blocks, 32, 2, 256), dtype=torch.uint8, device=DEV)
    s = torch.zeros((g.n_blocks, 2), device=DEV)
    ops.kv8_write(src, c, s, dev(g.cu), **g.args())
    back = ops.kv8_read(c, s, dev(g.cu), g.T, **g.args())
    # a value is off by half an E4M3 step at most: 2^-4 of it, or of the smallest normal
    x = src.float()
    unit = torch.zeros(g.T, 2, 1, device=DEV)
    for b, t, p in R.positions(g.cu, g.pos, g.table):
        unit[t, :, 0] = s[int(g.table[b, p // 32])]
    assert bool(((back.float() - x).abs() <= 2.0 ** -4 * torch.maximum(x.abs(), 2.0 ** -6 * unit)).all())
    c2, s2 = torch.zeros_like(c), torch.zeros_like(s)
    ops.kv8_write(back, c2, s2, dev(g.cu), **g.args())
    assert torch.equal(ops.kv8_read(c2, s2, dev(g.cu), g.T, **g.args()), back)
    c3, s3 = c.clone(), s.clone()
    ops.kv8_write(src, c, s, dev(g.cu), **g.args())
    assert torch.equal(c, c3) and torch.equal(s, s3)


# ------------------------------------------------------------------------ read
@pytest.mark.parametrize("heads,dim,block,new,ctx,table,pad", [
    (1, 576, 64, [1], [0], True, 0),
    (1, 576, 64, [200, 1, 65, 0, 64], [5, 70, 0, 9, 64], True, 2),
    (2, 256, 16, [33, 16, 1, 15, 2], [3, 0, 15, 1, 14], True, 5),
    (3, 48, 4, [9, 2, 30], [2, 5, 0], False, 0),
    (1, 16, 256, [600], [77], False, 1),
    (64, 128, 1, [37, 5], [0, 11], True, 0),
    (1, 1024, 8, [21, 8], [4, 8], True, 0),
    (1, 32, 32, [1] * 300, list(range(300)), True, 70),
    (1, 576, 64, [10000, 4001], [100, 3], True, 0),
])
def test_read(heads, dim, block, new, ctx, table, pad):
    rng = np.random.default_rng(sum(new) + dim + 1)
    g = Pages(rng, new, ctx, block, table, pad)
    codes, scale = cache_of(rng, g.n_blocks, block, heads, dim)
    codes[0, 0, 0, :2] = [127, 255]
    scale[1:3] = [[0.3], [1.7e-3]]  # any positive scale is read
    if table and g.table.shape[1] > 2:
        g.table[0, 1] = -1
        g.table[0, 2] = g.n_blocks + 5
    want = R.read(codes, scale, g.cu, g.T, g.pos, g.table, np.full((g.T, heads, dim), 7.0, np.float32))
    out = torch.full((g.T, heads, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    got = ops.kv8_read(dev(codes), dev(scale), dev(g.cu), g.T, out=out, **g.args())
    assert got.data_ptr() == out.data_ptr()
    a, b = got.float().cpu().numpy(), torch.from_numpy(want).to(torch.bfloat16).float().numpy()
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


def test_read_shared_prefix():
    """Two sequences that share pages read the same rows."""
    rng = np.random.default_rng(8)
    codes, scale = cache_of(rng, 6, 16, 1, 64)
    table = dev(np.array([[3, 1, 5], [3, 1, 0]], np.int32))
    out = ops.kv8_read(dev(codes), dev(scale), dev(cu_from_lengths([40, 35])), 75, block_table=table)
    assert torch.equal(out[:32], out[40:72]) and not torch.equal(out[32:35], out[72:75])


# ------------------------------------------------------------------- attention
def check_attention(q, k, ks, idx, sm, **kw):
    host = {n: kw.get(n) for n in ("length", "sink", "v8", "v_scale", "cu", "table")}
    ref = R.attention(f64(q), k, ks, idx, sm, **host)
    d = {n: (None if a is None else dev(a)) for n, a in host.items()}
    T, H = q.shape[:2]
    out = torch.full((T, H, ref["out"].shape[2]), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    got = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, topk_length=d["length"], sink=d["sink"],
                                  v8=d["v8"], v_scale=d["v_scale"], cu_seqlens=d["cu"], block_table=d["table"],
                                  want_lse_kv=True, want_max_logits=True, out=out, lse=lse)
    done = ref["done"]
    assert bool((out[dev(~done)] == 7.0).all()) and bool((lse[dev(~done)] == 7.0).all())
    o = out.float().cpu().numpy().astype(np.float64)[done]
    bad = np.abs(o - ref["out"][done]) > ref["out_tol"][done]
    assert np.isfinite(o).all() and not bad.any(), f"{bad.sum()} of {bad.size} outputs out of tolerance"
    for n in ("lse", "lse_kv", "max_logits"):
        g, r = got[n].cpu().numpy().astype(np.float64)[done], ref[n][done]
        fin = np.isfinite(r)
        assert np.array_equal(g[~fin], r[~fin]), n
        far = np.abs(g[fin] - r[fin]) - ref["lse_tol"][done][fin]
        assert not (far > 0).any(), f"{n}: {far.max():.3g} over its bound"
    bare = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, topk_length=d["length"], sink=d["sink"],
                                   v8=d["v8"], v_scale=d["v_scale"], cu_seqlens=d["cu"], block_table=d["table"])
    o = bare["out"][dev(done)].float().cpu().numpy().astype(np.float64)
    assert set(bare) == {"out", "lse"} and not (np.abs(o - ref["out"][done]) > ref["out_tol"][done]).any()
    g, r = bare["lse"].cpu().numpy().astype(np.float64)[done], ref["lse"][done]
    fin = np.isfinite(r)
    assert np.array_equal(g[~fin], r[~fin]) and not (np.abs(g[fin] - r[fin]) > ref["lse_tol"][done][fin]).any()
    return got


FORMS = [(576, 512), (512, 512), (256, 256)]


def attention_case(rng, dqk, dv, T, H, heads, K, block, table, n=None, holes=True):
    n = n or max(2 * K, 80)
    n_blocks = (n + block - 1) // block + 2
    k, ks = cache_of(rng, n_blocks, block, heads, dqk)
    kw = {}
    if dqk == 256:
        kw["v8"], kw["v_scale"] = cache_of(rng, n_blocks, block, heads, dv, -12, -3)
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
])
def test_attention(dqk, dv, T, H, heads, K, block, table, sink):
    rng = np.random.default_rng(T * 1000 + H + K + dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, H, heads, K, block, table)
    if sink:
        kw["sink"] = rng.standard_normal(H).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


def test_attention_leaves_padding_rows():
    """With a block table, rows behind the last sequence keep what they held."""
    rng = np.random.default_rng(77)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 9, 64, 1, 90, 16, True)
    kw["cu"] = cu_from_lengths([2, 4])
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_attention_long_rows_of_few_queries(dqk, dv):
    """One and two queries over 2048 slots: the slots are split between CTAs and joined."""
    for T in (1, 2):
        rng = np.random.default_rng(dqk + T)
        q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, T, 64, 1, 2048, 64, False, n=5000, holes=T == 2)
        check_attention(q, k, ks, idx, sm, sink=rng.standard_normal(64).astype(np.float32), **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_attention_many_rows(dqk, dv):
    """More rows than CTAs, lengths from none to three tiles."""
    rng = np.random.default_rng(dqk + 9)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, 700, 6, 1, 170, 16, True)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("lo,hi", [(-120, -100), (-30, 4), (60, 90), (-126, 90)])
def test_attention_scales_of_every_size(lo, hi):
    """Value scales that differ by many powers of two between blocks (keys of one size, so that scores stay finite)."""
    rng = np.random.default_rng(200 + hi)
    q, k, ks, idx, sm, kw = attention_case(rng, 256, 256, 6, 12, 1, 200, 4, False, holes=False)
    kw["v_scale"] = np.exp2(rng.integers(lo, hi + 1, kw["v_scale"].shape)).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_attention_rising_and_falling_scores(dqk, dv):
    """The running maximum moves in many tiles: keys in order of their scores, up and down."""
    rng = np.random.default_rng(dqk)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, 4, 64, 1, 512, 1, False, holes=False)
    ks[:] = 2.0 ** -4
    s = f64(q)[:, 0] @ (R.VALUES[k[:, 0, 0]]).T
    for t in range(4):
        order = np.argsort(s[t])[:: 1 if t % 2 else -1]
        idx[t] = order[np.linspace(0, order.size - 1, idx.shape[1]).astype(int)]
    check_attention(q, k, ks, idx, sm, **kw)


def test_attention_scales_need_not_be_powers_of_two():
    rng = np.random.default_rng(12)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 5, 64, 1, 100, 16, True)
    ks = (ks * rng.uniform(0.5, 2, ks.shape)).astype(np.float32)
    check_attention(q, k, ks, idx, sm, **kw)


@pytest.mark.parametrize("dqk,dv", FORMS)
def test_attention_never_uses_unselected_rows(dqk, dv):
    """NaN codes and scales in rows that no valid slot names, the slots behind topk_length among them."""
    rng = np.random.default_rng(dqk + 3)
    q, k, ks, idx, sm, kw = attention_case(rng, dqk, dv, 6, 20, 1, 90, 8, False)
    used = np.zeros(k.shape[0], bool)
    for t in range(6):
        i = idx[t, :max(0, min(int(kw["length"][t]), 90))]
        used[i[(i >= 0) & (i < k.shape[0] * 8)] // 8] = True
    used[rng.permutation(np.nonzero(used)[0])[:3]] = False  # and three blocks that are cut out of the ids
    idx[(idx >= 0) & (idx < k.shape[0] * 8) & ~used[np.clip(idx, 0, k.shape[0] * 8 - 1) // 8]] = -1
    assert not used.all()
    spoilt = dict(kw)
    k2, ks2 = k.copy(), ks.copy()
    k2[~used], ks2[~used] = 127, np.nan
    if dqk == 256:
        spoilt["v8"], spoilt["v_scale"] = kw["v8"].copy(), kw["v_scale"].copy()
        spoilt["v8"][~used], spoilt["v_scale"][~used] = 255, np.inf
    a = check_attention(q, k, ks, idx, sm, **kw)
    b = check_attention(q, k2, ks2, idx, sm, **spoilt)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_attention_nan_reaches_only_its_rows():
    """A NaN code in a selected row, and a query head with NaN or infinity, give NaN there and nowhere else."""
    rng = np.random.default_rng(21)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 4, 64, 1, 70, 1, False, holes=False)
    hit = idx[0, 5]
    idx[1:][idx[1:] == hit] = (hit + 1) % k.shape[0]
    clean = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm)["out"]
    bad = k.copy()
    bad[hit, 0, 0, 570] = 127  # a key-only dim: every score of that slot
    got = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(bad), dev(ks), dev(idx), sm)
    assert bool(got["out"][0].isnan().all()) and bool(got["lse"][0].isnan().all()) and torch.equal(got["out"][1:], clean[1:])
    q2 = dev_bf16(q)
    q2[2, 7, 3], q2[3, 9, 500] = float("nan"), float("inf")
    got = ops.sparse_attn_fwd_kv8(q2, dev(k), dev(ks), dev(idx), sm)["out"]
    hit = torch.zeros(4, 64, dtype=torch.bool, device=DEV)
    hit[2, 7] = hit[3, 9] = True
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], clean[~hit])


def test_attention_equals_the_bf16_call_on_values_read_back():
    """Power-of-two scales: the cache's values are bf16 exactly, so both calls compute the same formula."""
    rng = np.random.default_rng(30)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 30, 64, 1, 200, 16, False)
    n = k.shape[0] * 16
    kv = ops.kv8_read(dev(k), dev(ks), dev(cu_from_lengths([n])), n).view(n, 576)
    a = ops.sparse_attn_fwd_kv8(dev_bf16(q), dev(k), dev(ks), dev(idx), sm, topk_length=dev(kw["length"]))
    b = ops.sparse_attn_fwd(dev_bf16(q), kv, dev(idx), sm, topk_length=dev(kw["length"]))
    # each side rounds weights (2^-8) and out (2^-8): normwise well within four such steps
    d = (a["out"].float() - b["out"].float()).norm() / b["out"].float().norm()
    assert float(d) <= 4 * 2.0 ** -8
    fin = torch.isfinite(b["lse"])
    assert torch.equal(fin, torch.isfinite(a["lse"])) and float((a["lse"] - b["lse"])[fin].abs().max()) <= 1e-3


def test_attention_offsets_beyond_32_bits():
    """Rows behind the cache's first 4 GiB."""
    rng = np.random.default_rng(31)
    block, n_blocks = 64, 120000
    cache = torch.zeros((n_blocks, block, 1, 576), dtype=torch.uint8, device=DEV)
    scale = torch.ones((n_blocks, 1), device=DEV)
    k, ks = cache_of(rng, 4, block, 1, 576)
    at = [0, 1, n_blocks - 2, n_blocks - 1]
    for i, b in enumerate(at):
        cache[b], scale[b] = dev(k[i]), dev(ks[i])
    idx = rng.integers(0, 4 * block, (3, 150)).astype(np.int32)
    far = (np.array(at)[idx // block] * block + idx % block).astype(np.int32)
    q = dev_bf16(rand_bf16_bits(rng, (3, 64, 576)))
    a = ops.sparse_attn_fwd_kv8(q, cache, scale, dev(far), 0.04)
    b = ops.sparse_attn_fwd_kv8(q, dev(k), dev(ks), dev(idx), 0.04)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    table = dev(np.array([at], np.int32))
    cu = dev(cu_from_lengths([200]))
    back = ops.kv8_read(cache, scale, cu, 200, pos=dev(np.array([40], np.int32)), block_table=table)
    want = ops.kv8_read(dev(k), dev(ks), cu, 200, pos=dev(np.array([40], np.int32)))
    assert torch.equal(back, want)
    ops.kv8_write(back, cache, scale, cu, pos=dev(np.array([40], np.int32)), block_table=table)
    assert torch.equal(ops.kv8_read(cache, scale, cu, 200, pos=dev(np.array([40], np.int32)), block_table=table), want)


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(32)
    q, k, ks, idx, sm, kw = attention_case(rng, 576, 512, 33, 128, 1, 300, 16, False)
    a = [dev_bf16(q), dev(k), dev(ks), dev(idx), sm]
    first = ops.sparse_attn_fwd_kv8(*a, topk_length=dev(kw["length"]))
    for _ in range(20):
        again = ops.sparse_attn_fwd_kv8(*a, topk_length=dev(kw["length"]))
        assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


def test_empty_calls():
    k, ks = cache_of(np.random.default_rng(1), 2, 4, 1, 576)
    c, s = dev(k), dev(ks)
    cu = dev(cu_from_lengths([0]))
    ops.kv8_write(torch.empty((0, 1, 576), dtype=torch.bfloat16, device=DEV), c, s, cu)
    assert ops.kv8_read(c, s, cu, 0).shape == (0, 1, 576)
    q = torch.ones((3, 5, 576), dtype=torch.bfloat16, device=DEV)
    r = ops.sparse_attn_fwd_kv8(q, c, s, torch.empty((3, 0), dtype=torch.int32, device=DEV), 0.1)
    assert bool((r["out"] == 0).all()) and bool((r["lse"] == -math.inf).all())
    r = ops.sparse_attn_fwd_kv8(q[:0], c, s, torch.empty((0, 4), dtype=torch.int32, device=DEV), 0.1)
    assert r["out"].shape == (0, 5, 512)
    assert np.array_equal(c.cpu().numpy(), k)


# -------------------------------------------------------------- used together
def test_decode_steps_together():
    """A prompt and decode steps as they are served: rows quantised into the
    caches (indexer keys as plain rows in per-sequence slots, the latent rows
    in pages), the indexer's top-k over its 8-bit keys, attention over the
    8-bit latent rows of the selected positions."""
    rng = np.random.default_rng(40)
    n_seqs, slot, block, Hi, H, K = 3, 256, 64, 32, 64, 48
    per = slot // block
    table = rng.permutation(n_seqs * per + 2)[:n_seqs * per].reshape(n_seqs, per).astype(np.int32)
    kv8 = torch.full((n_seqs * per + 2, block, 1, 576), 127, dtype=torch.uint8, device=DEV)
    kvs = torch.full((n_seqs * per + 2, 1), math.nan, device=DEV)
    ki8 = torch.zeros((n_seqs * slot, 1, 1, 128), dtype=torch.uint8, device=DEV)
    kis = torch.full((n_seqs * slot, 1), 1.0, device=DEV)
    cu_k = dev((np.arange(n_seqs + 1) * slot).astype(np.int32))
    dt = dev(table)
    have = np.zeros(n_seqs, np.int32)
    for new in ([100, 37, 64], [1, 1, 1], [1, 1, 1], [30, 1, 0]):
        T, cu = sum(new), cu_from_lengths(new)
        kv, ki = rows(rng, T, 1, 576), rows(rng, T, 1, 128)
        qi, q = rand_bf16_bits(rng, (T, Hi, 128)), rand_bf16_bits(rng, (T, H, 576))
        w = (rng.random((T, Hi), dtype=np.float32) / 8).astype(np.float32)
        before_c, before_s = kv8.cpu().numpy(), kvs.cpu().numpy()
        dcu, pos = dev(cu), dev(have)
        ops.kv8_write(dev_bf16(kv), kv8, kvs, dcu, pos=pos, block_table=dt)
        ops.kv8_write(dev_bf16(ki), ki8, kis, dcu, pos=dev((have + np.arange(n_seqs) * slot).astype(np.int32)))
        qi8 = torch.empty((T, 1, Hi, 128), dtype=torch.uint8, device=DEV)
        qis = torch.empty((T, Hi), device=DEV)
        ops.kv8_write(dev_bf16(qi), qi8, qis, dcu)
        top = ops.indexer_topk_fp8(qi8.view(T, Hi, 128), ki8.view(-1, 128), qis, kis.view(-1), dev(w), dcu, cu_k, pos, 1, K, slot)
        start = torch.repeat_interleave(torch.arange(n_seqs, device=DEV, dtype=torch.int32) * slot, dev(np.array(new)))
        local = torch.where(top["idx"] >= 0, top["idx"] - start[:, None], -1).contiguous()
        got = ops.sparse_attn_fwd_kv8(dev_bf16(q), kv8, kvs, local, 1 / 24, topk_length=top["topk_length"], cu_seqlens=dcu,
                                      block_table=dt)
        # each part against its definition, on what the part before it gave
        rc, rs = R.write(f64(kv), before_c, before_s, cu, have, table)
        written = np.isfinite(rs[:, 0])
        assert np.array_equal(kvs.cpu().numpy()[written], rs[written]) and same_codes(kv8.cpu().numpy(), rc)
        qv = R.VALUES[qi8.cpu().numpy()[:, 0]] * qis.cpu().numpy().astype(np.float64)[:, :, None]
        kvals = R.VALUES[ki8.cpu().numpy()[:, 0, 0]] * kis.cpu().numpy().astype(np.float64)
        length = np.concatenate([np.arange(n) + p + 1 for n, p in zip(new, have)]).astype(np.int32)
        st = np.repeat(np.arange(n_seqs) * slot, new).astype(np.int32)
        sc = oracle.indexer_scores(qv, kvals, w, st, length, slot)
        tl = top["topk_length"].cpu().numpy()
        assert np.array_equal(tl, np.minimum(length, K))
        for t in range(T):  # the selected scores are the largest, up to the indexer's own tolerance
            ids = local.cpu().numpy()[t, :tl[t]]
            kth = np.sort(sc[t, :length[t]])[::-1][tl[t] - 1]
            assert np.unique(ids).size == tl[t] and (sc[t, ids] >= kth - 1e-4 * max(1.0, abs(kth))).all()
        ref = R.attention(f64(q), rc, rs, local.cpu().numpy(), 1 / 24, length=tl, cu=cu, table=table)
        o = got["out"].float().cpu().numpy()
        assert not (np.abs(o - ref["out"]) > ref["out_tol"]).any()
        assert not (np.abs(got["lse"].cpu().numpy() - ref["lse"]) > ref["lse_tol"]).any()
        have = (have + np.array(new)).astype(np.int32)


def test_captured_steps_with_their_own_workspaces():
    """Write and attention in two CUDA graphs, replayed in turn and on another stream with new inputs in place."""
    rng = np.random.default_rng(41)
    block, H = 32, 64
    made = []
    for T, K in ((2, 700), (5, 300)):
        q, k, ks, idx, sm, _ = attention_case(rng, 576, 512, T, H, 1, K, block, False, holes=False)
        st = {"q": dev_bf16(q), "k": dev(k), "s": dev(ks), "idx": dev(idx), "cu": dev(cu_from_lengths([T])),
              "pos": dev(np.array([37], np.int32)), "src": dev_bf16(rows(rng, T, 1, 576))}
        n = ops.sparse_attn_fwd_kv8_workspace_size(T, H, 1, 576, 512, K)
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)

        def step(st=st, sm=sm):
            ops.kv8_write(st["src"], st["k"], st["s"], st["cu"], pos=st["pos"])
            return ops.sparse_attn_fwd_kv8(st["q"], st["k"], st["s"], st["idx"], sm, workspace=st["ws"])

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
            k0, s0 = st["k"].clone(), st["s"].clone()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side if r == 1 else torch.cuda.current_stream()):
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
            out, lse, k1 = st["res"]["out"].clone(), st["res"]["lse"].clone(), st["k"].clone()
            st["k"].copy_(k0)
            st["s"].copy_(s0)
            eager = step()
            assert torch.equal(out, eager["out"]) and torch.equal(lse, eager["lse"]) and torch.equal(k1, st["k"])


def test_binding_refuses():
    k, ks = cache_of(np.random.default_rng(1), 4, 8, 1, 576)
    c, s, cu = dev(k), dev(ks), dev(cu_from_lengths([3]))
    x = torch.zeros((3, 1, 576), dtype=torch.bfloat16, device=DEV)
    q, idx = torch.zeros((2, 4, 576), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 8), dtype=torch.int32, device=DEV)
    for bad in (lambda: ops.kv8_write(x[:, :, :512], c, s, cu), lambda: ops.kv8_write(x, c, s[:3].contiguous(), cu),
                lambda: ops.kv8_write(x, c.transpose(0, 1), s, cu), lambda: ops.kv8_write(x, c, s, cu, pos=cu),
                lambda: ops.kv8_write(x, c, s, cu, block_table=dev(np.zeros((2, 2), np.int32))),
                lambda: ops.kv8_read(c, s, cu, 3, out=x[:2]),
                lambda: ops.sparse_attn_fwd_kv8(q, c, s, idx[:1], 0.1),
                lambda: ops.sparse_attn_fwd_kv8(q, c, s, idx, 0.1, v8=c),
                lambda: ops.sparse_attn_fwd_kv8(q, c, s, idx, 0.1, sink=s.view(-1)[:3]),
                lambda: ops.sparse_attn_fwd_kv8(q, c, s, idx, 0.1, block_table=dev(np.zeros((1, 2), np.int32))),
                lambda: ops.sparse_attn_fwd_kv8(q[:, :, :512].contiguous(), c, s, idx, 0.1),
                lambda: ops.sparse_attn_fwd_kv8(q, c, s, idx, -1.0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.kv8_write(x.float(), c, s, cu), lambda: ops.kv8_write(x, c.to(torch.int8), s, cu),
                lambda: ops.kv8_read(c, s, cu.long(), 3), lambda: ops.sparse_attn_fwd_kv8(q, c, s, idx.long(), 0.1)):
        with pytest.raises(TypeError):
            bad()
