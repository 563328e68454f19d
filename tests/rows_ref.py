"""Plain definitions of the row norm and of rotary positions in 64 bits (numpy),
with bounds on how far a result may be off."""
from __future__ import annotations

import math

import numpy as np

import kv8_ref

BF16 = 2.0 ** -8  # half a step, relative
F32 = 2.0 ** -24


def norm(x, w, eps, residual=None):
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w


# A sum of squares: a thread adds 32 at most, then 5 shuffles and 16 warps: 53 roundings, and the squares' own;
# the mean, eps, root and quotient a few more, halved by the root.  With the product by h and w: 40 of 2^-24.
RSTD_REL = 40 * F32


def norm_bounds(h, rstd, y):
    """Bounds of sum, rstd and bf16 y."""
    return BF16 * np.abs(h) * (1 + 2.0 ** -15), RSTD_REL * rstd, np.abs(y) * (BF16 + 2 * RSTD_REL)


def check_codes(codes, scale, y, group):
    """8-bit output: scales are powers of two that fit the largest finite |y| of their group (either one where that is
    within the norm's own error of the border), codes within half a step of y."""
    T, D = y.shape
    g = y.reshape(T, D // group, group)
    fin = np.where(np.isfinite(g), np.abs(g), 0.0).max(2)
    lo = np.array([[kv8_ref.scale_of(a * (1 - 4 * RSTD_REL)) for a in r] for r in fin])
    hi = np.array([[kv8_ref.scale_of(a * (1 + 4 * RSTD_REL)) for a in r] for r in fin])
    assert ((scale == lo) | (scale == hi)).all(), "scales"
    v = kv8_ref.VALUES[codes].reshape(g.shape) * scale[:, :, None]
    nan = np.isnan(g)
    assert np.array_equal(np.isnan(v), nan), "NaN"
    inf = np.isinf(g)
    assert np.array_equal(v[inf], (np.sign(g) * 448 * scale[:, :, None])[inf]), "infinities"
    ok = ~nan & ~inf
    # E4M3: half a step is 2^-4 of the value, or half of 2^-9 below the normal range
    tol = np.abs(g) * (2.0 ** -4 + 4 * RSTD_REL) + 2.0 ** -10 * scale[:, :, None]
    assert (np.abs(v - g)[ok] <= tol[ok]).all(), "codes"


def norm_back(dy, x, w, rstd, d_sum=None):
    """dx, dw and bounds of both."""
    D = x.shape[1]
    xh = x * rstd[:, None]
    g = dy * w
    mean = (g * xh).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xh * mean)
    # every term of dx has a few roundings of its own, the mean those of a sum of its magnitudes (53 and a few)
    tol = 64 * F32 * rstd[:, None] * (np.abs(g) + np.abs(xh) * (np.abs(g * xh).mean(1, keepdims=True) + np.abs(mean)))
    if d_sum is not None:
        dx = dx + d_sum
        tol = tol + 4 * F32 * np.abs(d_sum)
    terms = dy * xh
    # dw: a thread adds its rows' terms one by one, then the rest in a tree: never more than T + 64 roundings in a row
    return dx, terms.sum(0), tol + BF16 * np.abs(dx), (x.shape[0] + 64) * F32 * np.abs(terms).sum(0) + 1e-300


def rotary(x, f, positions, pairs, inverse=False, mul=1.0):
    """x [T, H, R] float64; positions: integers, or None for a row that is left alone (then NaN)."""
    T, H, R = x.shape
    y, tol = np.full_like(x, np.nan), np.full_like(x, np.inf)
    first = np.arange(0, R, 2) if pairs else np.arange(R // 2)
    second = first + 1 if pairs else first + R // 2
    for t, p in enumerate(positions):
        if p is None:
            continue
        # p * f in one rounded product, modulo the 64-bit 2 pi: what that leaves out is in e below
        theta = np.array([math.fmod(float(p) * float(v), 2 * math.pi) for v in f])
        if inverse:
            theta = -theta
        c, s = mul * np.cos(theta), mul * np.sin(theta)
        a, b = x[t][:, first], x[t][:, second]
        y[t][:, first], y[t][:, second] = a * c - b * s, a * s + b * c
        # the angle: 2^-25 of half a turn, f / (2 pi) to 2^-53 and this definition's own p * f to 2^-53 of the turns so
        # far; cosine, sine, mul and products a few 2^-24 each
        e = math.pi * 2.0 ** -25 + 8 * F32 + 2.0 ** -51 * abs(float(p)) * np.abs(f)
        d = abs(mul) * e * (np.abs(a) + np.abs(b))
        tol[t][:, first] = d + BF16 * np.abs(y[t][:, first])
        tol[t][:, second] = d + BF16 * np.abs(y[t][:, second])
    return y, tol


def inv_freq(R, base, scaling="plain", factor=1.0, first=4096, fast=32.0, slow=1.0):
    """(angles per position, factor of the result), pair by pair from the definition."""
    half, out = R // 2, []
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    for i in range(half):
        f = base ** (-2.0 * i / R)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            def pair(turns):
                return R * math.log(first / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
            blend = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f / factor * blend + f * (1 - blend)
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)
