"""Plain definitions of the 8-bit block cache in 64 bits (numpy): E4M3 from its
bit fields, the writer's block scales and rescaling, reading back, and sparse
attention over the cache with the error bounds its tests use."""
from __future__ import annotations

import math

import numpy as np


def _values():
    v = np.empty(256, np.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 128 else x
    return v


VALUES = _values()


def to_codes(x):
    """Nearest E4M3 code of each value, ties to the even code, saturating; NaN -> 127."""
    x = np.asarray(x, np.float64)
    pos = VALUES[:127]
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.signbit(x), c | 128, c)
    return np.where(np.isnan(x), 127, c).astype(np.uint8)


def scale_of(amax):
    """2^e, e the smallest integer with amax <= 448 * 2^e, at least -126."""
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def row_of(table, block, n_blocks, b, p):
    page = p // block
    if p < 0:
        return -1
    if table is not None:
        if page >= table.shape[1]:
            return -1
        page = int(table[b, page])
    return page * block + p % block if 0 <= page < n_blocks else -1


def positions(cu, pos, table):
    for b in range(len(cu) - 1):
        p0 = int(pos[b]) if pos is not None else (0 if table is not None else int(cu[b]))
        for t in range(int(cu[b]), int(cu[b + 1])):
            yield b, t, p0 + t - int(cu[b])


def write(src, cache, scale, cu, pos, table):
    """(codes, scale) after the write; src float64, cache uint8 [n_blocks, block, Hc, D], scale float32."""
    cache, scale = cache.copy(), scale.copy()
    n_blocks, block, heads, dim = cache.shape
    got = {}
    for b, t, p in positions(cu, pos, table):
        r = row_of(table, block, n_blocks, b, p)
        if r >= 0:
            got.setdefault(r // block, []).append((r % block, t))
    for blk, rows in got.items():
        first = min(o for o, _ in rows)
        for h in range(heads):
            x = np.stack([src[t, h] for _, t in rows])
            fin = np.abs(x[np.isfinite(x)])
            s = np.float32(scale_of(fin.max() if fin.size else 0.0))
            if first > 0:
                old = scale[blk, h]
                s = max(s, old)
                if s > old:
                    with np.errstate(invalid="ignore"):
                        v = VALUES[cache[blk, :first, h]].astype(np.float32) * np.float32(old / s)
                    cache[blk, :first, h] = to_codes(v)
            for (o, _), v in zip(rows, x):
                with np.errstate(invalid="ignore"):
                    cache[blk, o, h] = to_codes(v.astype(np.float32) / s)
            scale[blk, h] = s
    return cache, scale


def read(cache, scale, cu, T, pos, table, out):
    """out (float32, updated in place) before the rounding to bf16."""
    n_blocks, block, heads, dim = cache.shape
    for b, t, p in positions(cu, pos, table):
        r = row_of(table, block, n_blocks, b, p)
        out[t] = 0.0 if r < 0 else (VALUES[cache[r // block, r % block]].astype(np.float32) *
                                    scale[r // block][:, None].astype(np.float32))
    return out


def attention(q, kv8, kv_scale, idx, sm, length=None, sink=None, v8=None, v_scale=None, cu=None, table=None):
    """out, lse, lse_kv, max_logits in float64 and, per output, how far a result may be off.

    Bounds.  Scores: fp32 accumulation of Dqk exact products, at most Dqk *
    2^-24 of the sum of their magnitudes, a query kept to 2^-21 of its largest
    element, and a few fp32 roundings (2^-21 relative): d_j.  Weights: exp is a
    few ulp (2^-20), and a weight enters the value product as two E4M3 terms of
    a half: relative 2^-8 + 2^-11, and at least 2^-10 / 14 of the largest weight times
    the largest scale (half the smaller term's step, weights being held as 14 times themselves).  out is rounded to bf16 (2^-8)."""
    T, H, dqk = q.shape
    n_blocks, block, heads, _ = kv8.shape
    group, K = H // heads, idx.shape[1]
    dv = 512 if v8 is None else v8.shape[3]
    out, tol = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    lse, lse_kv, mx = np.full((T, H), -np.inf), np.full((T, H), np.inf), np.full((T, H), -np.inf)
    ltol = np.full((T, H), 1e-30)
    done = np.ones(T, bool)
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
            k = VALUES[kv8[rows // block, rows % block, g]] * kv_scale[rows // block, g].astype(np.float64)[:, None]
            if v8 is None:
                sv, vc = kv_scale[rows // block, g].astype(np.float64), VALUES[kv8[rows // block, rows % block, g]][:, :dv]
            else:
                sv, vc = v_scale[rows // block, g].astype(np.float64), VALUES[v8[rows // block, rows % block, g]]
            v = vc * sv[:, None]
            qq = q[t, hs].astype(np.float64)
            s = sm * (qq @ k.T)
            d = sm * (dqk * 2.0 ** -24 * (np.abs(qq) @ np.abs(k).T) +
                      2.0 ** -21 * np.abs(qq).max(1)[:, None] * np.abs(k).sum(1)[None, :]) + 2.0 ** -21 * np.abs(s)
            m = s.max(1)
            e = np.exp(s - m[:, None])
            z = e.sum(1)
            zs = z + np.exp(sk - m)
            p = e / zs[:, None]
            o = p @ v
            dm = d.max(1) + 2.0 ** -19
            out[t, hs], lse_kv[t, hs], lse[t, hs], mx[t, hs] = o, m + np.log(z), m + np.log(zs), m
            ltol[t, hs] = dm + 2.0 ** -21 * (np.abs(m) + 16)
            top = 2.0 ** np.ceil(np.log2(sv.max()))
            floor = 2.0 ** -10 / 14 * top * np.abs(vc).sum(0)[None, :] / zs[:, None]
            tol[t, hs] = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -11 + 2 * dm[:, None]) * (p @ np.abs(v)) + floor
    return {"out": out, "lse": lse, "lse_kv": lse_kv, "max_logits": mx, "out_tol": tol, "lse_tol": ltol, "done": done}
