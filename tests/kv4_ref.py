"""Plain definitions of the 4-bit block cache in 64 bits (numpy): E2M1 codes with
a power of two per 32, and sparse attention over it with the bounds its tests use."""
from __future__ import annotations

import numpy as np

from kv8_ref import positions, row_of

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BF16_MOST = 2.0 ** 127 * (2 - 2.0 ** -7)


def quantise(x):
    """Codes (4 bits, one per byte) and scale bytes of x [..., D]."""
    shape = x.shape
    x = np.asarray(x, np.float64).reshape(-1, 32)
    codes, scale = np.zeros(x.shape, np.uint8), np.zeros(x.shape[0], np.uint8)
    for i, g in enumerate(x):
        if np.isnan(g).any():
            scale[i] = 255
            continue
        fin = np.abs(g[np.isfinite(g)])
        a, e = (fin.max() if fin.size else 0.0), -126
        while e < 125 and a > 6 * 2.0 ** e:
            e += 1
        v = np.minimum(np.abs(g) / 2.0 ** e, 6.0)
        d = np.abs(v[:, None] - MAGNITUDES[None, :])
        best = d.min(1)
        for j in range(32):
            near = np.nonzero(d[j] == best[j])[0]
            codes[i, j] = near[0] if len(near) == 1 else near[near % 2 == 0][0]
        codes[i] |= np.signbit(g).astype(np.uint8) << 3
        scale[i] = e + 127
    return codes.reshape(shape), scale.reshape(*shape[:-1], shape[-1] // 32)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values(packed, scale):
    """float64 values; NaN where the byte is 255, infinite beyond the bf16 range."""
    v = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]))
    both = np.concatenate([MAGNITUDES, -MAGNITUDES])
    v[..., 0::2], v[..., 1::2] = both[packed & 15], both[packed >> 4]
    s = np.repeat(np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127)), 32, axis=-1)
    with np.errstate(invalid="ignore"):
        v = v * s
        return np.where(np.abs(v) > BF16_MOST, np.sign(v) * np.inf, v)


def write(src, cache, scale, cu, pos, table):
    cache, scale = cache.copy(), scale.copy()
    n_blocks, block = cache.shape[:2]
    for b, t, p in positions(cu, pos, table):
        r = row_of(table, block, n_blocks, b, p)
        if r >= 0:
            c, s = quantise(src[t])
            cache[r // block, r % block], scale[r // block, r % block] = pack(c), s
    return cache, scale


def read(cache, scale, cu, pos, table, out):
    n_blocks, block = cache.shape[:2]
    for b, t, p in positions(cu, pos, table):
        r = row_of(table, block, n_blocks, b, p)
        out[t] = 0.0 if r < 0 else values(cache[r // block, r % block], scale[r // block, r % block])
    return out


def attention(q, kv4, kv_scale, idx, sm, length=None, sink=None, v4=None, v_scale=None, cu=None, table=None):
    """out, lse, lse_kv, max_logits in float64 and, per output, how far a result may be off.

    Bounds.  Scores: fp32 accumulation of Dqk exact products, at most Dqk * 2^-23 of the sum of
    their magnitudes, and a few fp32 roundings (2^-21 relative): d_j.  Weights: exp is a few ulp
    (2^-20) and they are rounded to bf16 (2^-8) before the value product, whose sums are fp32
    (2^-12 stands for up to 4096 terms at 2^-24).  out is rounded to bf16 (2^-8)."""
    T, H, dqk = q.shape
    n_blocks, block, heads, _ = kv4.shape
    group, K = H // heads, idx.shape[1]
    dv = 512 if v4 is None else 2 * v4.shape[3]
    out, tol = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    lse, lse_kv, mx = np.full((T, H), -np.inf), np.full((T, H), np.inf), np.full((T, H), -np.inf)
    ltol, done = np.full((T, H), 1e-30), np.ones(T, bool)
    for t in range(T):
        b = 0
        if table is not None:
            if t >= cu[-1]:
                done[t] = False
                continue
            b = int(np.searchsorted(cu, t, side="right")) - 1
        n = K if length is None else min(max(int(length[t]), 0), K)
        rows = [row_of(table, block, n_blocks, b, int(i)) for i in idx[t, :n] if i >= 0]
        rows = np.array([r for r in rows if r >= 0], np.int64)
        for g in range(heads):
            hs = slice(g * group, (g + 1) * group)
            sk = np.full(group, -np.inf) if sink is None else sink[hs].astype(np.float64)
            if rows.size == 0:
                lse[t, hs] = sk
                continue
            k = values(kv4[rows // block, rows % block, g], kv_scale[rows // block, rows % block, g])
            v = k[:, :dv] if v4 is None else values(v4[rows // block, rows % block, g],
                                                    v_scale[rows // block, rows % block, g])
            qq = q[t, hs].astype(np.float64)
            s = sm * (qq @ k.T)
            d = sm * dqk * 2.0 ** -23 * (np.abs(qq) @ np.abs(k).T) + 2.0 ** -21 * np.abs(s)
            m = s.max(1)
            e = np.exp(s - m[:, None])
            z = e.sum(1)
            zs = z + np.exp(sk - m)
            p = e / zs[:, None]
            o = p @ v
            dm = d.max(1) + 2.0 ** -19
            out[t, hs], lse_kv[t, hs], lse[t, hs], mx[t, hs] = o, m + np.log(z), m + np.log(zs), m
            ltol[t, hs] = dm + 2.0 ** -21 * (np.abs(m) + 16)
            tol[t, hs] = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12 + 2 * dm[:, None]) * (p @ np.abs(v)) + 1e-300
    return {"out": out, "lse": lse, "lse_kv": lse_kv, "max_logits": mx, "out_tol": tol, "lse_tol": ltol, "done": done}
