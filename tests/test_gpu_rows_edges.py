"""Norm and rotary positions of rows and positions at the ends of their ranges, against their 64-bit definitions."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import rows_ref as R
from gpu_util import DEV, cu_from_lengths, dev
from sparse_attention_gemm_gb300 import ops
from test_gpu_rows import EPS, apart, f64, near

pytestmark = pytest.mark.gpu

MOST = 3.3895313892515355e38  # the largest bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float64)).to(torch.bfloat16).to(DEV)


def check_norm(x, w, eps, residual=None):
    h, rstd, y = R.norm(f64(x), w.astype(np.float64), float(np.float32(eps)), None if residual is None else f64(residual))
    ts, tr, ty = R.norm_bounds(h, rstd, y)
    got = ops.rms_norm_fwd(x, dev(w), eps, residual=residual, want_rstd=True)
    # (below 2^-126 rstd is a multiple of 2^-149, at least 2^-128: off by 2^-22 of itself, which the bounds leave room for;
    # results below 2^-126 are multiples of 2^-133, sums of the residual are in range)
    near(got["rstd"], rstd, tr + 2.0 ** -150, "rstd")
    near(got["out"], y, ty + 2.0 ** -134, "out")
    if residual is not None:
        near(got["sum"], h, ts, "sum")
    if x.shape[1] % 128 == 0:
        for fmt, group in (("e4m3", 128), ("mxfp8", 32)):
            q = ops.rms_norm_fwd(x, dev(w), eps, residual=residual, fmt=fmt)
            s = q["scale"].cpu().numpy()
            s = s.astype(np.float64) if fmt == "e4m3" else np.exp2(s.astype(np.float64) - 127)
            R.check_codes(q["out"].cpu().numpy(), s, y, group)


@pytest.mark.parametrize("D", [8, 64, 128, 256, 512, 1024, 1032, 4096, 8200, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_rows_up_to_the_largest_values(D, residual):
    """Squares and their sums beyond fp32's range, beside ordinary rows: every finite row has its norm."""
    rng = np.random.default_rng(D)
    x = rng.standard_normal((14, D))
    size = 2.0 ** np.array([0, 40, 60, 63, 64, 70, 90, 110, 118, 122, 125])
    x[:11] *= size[:, None] / np.abs(x[:11]).max(1, keepdims=True)
    x[11] = MOST * np.sign(x[11])
    x[12] = 0
    x[12, D // 2] = -MOST
    x[13] *= 2.0 ** rng.uniform(-120, 120, D)
    x[13] = np.clip(x[13], -MOST, MOST)
    r = None
    if residual:
        r = rng.standard_normal((14, D))
        r[:11] *= size[:, None] / 16
        r[11] = -np.sign(x[11]) * MOST / 2
    check_norm(bf16(x), rng.standard_normal(D).astype(np.float32), EPS, None if r is None else bf16(r))


@pytest.mark.parametrize("D", [8, 64, 256, 512, 1032, 4096, 16384])
@pytest.mark.parametrize("eps", [1e-45, 1e-43, 1e-38, 1e-31])
def test_norm_with_an_eps_below_small_squares(D, eps):
    """Squares below fp32's range that count beside an eps of their size."""
    rng = np.random.default_rng(D)
    x = rng.standard_normal((9, D)) * 10.0 ** np.array([-22, -22.5, -21, -20, -19, -16, -23, 0, 30])[:, None]
    x[6] = 0
    check_norm(bf16(x), rng.standard_normal(D).astype(np.float32), eps)


@pytest.mark.parametrize("D", [8, 64, 512, 4096])
def test_norm_with_an_eps_near_the_largest_number(D):
    """Squares and an eps that are in fp32's range while their sum is not."""
    x = np.random.default_rng(D).standard_normal((7, D)) * 10.0 ** np.array([19.2, 19, 18.5, 18, 25, 0, 37])[:, None]
    check_norm(bf16(x), np.ones(D, np.float32), 3e38)


def test_sizes_beyond_32_bits_are_refused():
    """The library's sizes are 32-bit: a larger one does not come in modulo 2^32."""
    far = 1 << 32
    x = torch.zeros(1, 1, 16, dtype=torch.bfloat16, device=DEV).expand(far, 1, 16)
    f, _ = ops.rotary_inv_freq(16)
    cu, w = dev(cu_from_lengths([1])), torch.ones(8, device=DEV)
    rows = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV).expand(far, 8)
    rstd = torch.ones(1, device=DEV).expand(far)
    src, empty = torch.zeros(3, 0, 32, dtype=torch.bfloat16, device=DEV), torch.zeros(far + 1, 1, 0, 16, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(far + 1, 1, 0, 1, dtype=torch.uint8, device=DEV)
    q, idx = torch.zeros(1, 4, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 8, dtype=torch.int32, device=DEV)
    wide = torch.zeros(far + 1, 1, 0, 288, dtype=torch.uint8, device=DEV)
    for bad in (lambda: ops.rotary(x, f, cu, out=x), lambda: ops.rms_norm_fwd(rows, w, EPS, out=rows),
                lambda: ops.rms_norm_bwd(rows, rows, w, rstd, dx=rows, want_dweight=False),
                lambda: ops.kv4_write(src, empty, scale, cu), lambda: ops.kv4_read(empty, scale, cu, 3, out=src),
                lambda: ops.sparse_attn_fwd_kv4(q, wide, wide[..., :18], idx, 0.1)):
        with pytest.raises(ValueError, match="32 bits"):
            bad()


@pytest.mark.parametrize("fmt,group", [("e4m3", 128), ("mxfp8", 32)])
@pytest.mark.parametrize("T,D", [(300001, 128), (9001, 1024)])
def test_norm_in_8_bits_of_a_prompts_rows(fmt, group, T, D):
    """As many rows as a prompt's indexer heads are."""
    rng = np.random.default_rng(T)
    x = apart(bf16(rng.standard_normal((T, D)) * np.exp2(rng.uniform(-6, 6, (T, 1)))), 64)
    w = (rng.standard_normal(D) * np.exp2(rng.integers(-6, 6, D))).astype(np.float32)
    _, _, y = R.norm(f64(x), w.astype(np.float64), EPS)
    got = ops.rms_norm_fwd(x, dev(w), EPS, fmt=fmt)
    s = got["scale"].cpu().numpy()
    s = s.astype(np.float64) if fmt == "e4m3" else np.exp2(s.astype(np.float64) - 127)
    g = y.reshape(T, D // group, group)
    most = np.abs(g).max(2)
    # a <= 448 * 2^e for the smallest e, where 448 = 1.75 * 2^8; either power within the norm's own error of a border
    lo, hi = (np.exp2(np.ceil(np.log2(most * (1 + k * 4 * R.RSTD_REL) / 448))) for k in (-1, 1))
    assert ((s == lo) | (s == hi)).all(), "scales"
    v = torch.from_numpy(got["out"].cpu().numpy()).view(torch.float8_e4m3fn).double().numpy().reshape(g.shape) * s[:, :, None]
    # E4M3: half a step is 2^-4 of the value, or half of 2^-9 below the normal range
    tol = np.abs(g) * (2.0 ** -4 + 4 * R.RSTD_REL) + 2.0 ** -10 * s[:, :, None]
    assert (np.abs(v - g) <= tol).all(), "codes"


def inverse_pi(bits):
    """1 / (2 pi) in units of 2^-bits, by Machin's formula: pi = 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (bits + 64)

    def atan(n):
        term, total, k = one // n, 0, 0
        while term:
            total += (-term if k & 1 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total
    return (one << bits) // (2 * (16 * atan(5) - 4 * atan(239)))


def exact_angle(p, f, turn=inverse_pi(320)):
    """p * f modulo 2 pi in [-pi, pi], from the exact product of the integer and the double."""
    part = (Fraction(int(p)) * Fraction(float(f)) * Fraction(turn, 1 << 320)) % 1
    return 2 * np.pi * float(part - 1 if part > Fraction(1, 2) else part)


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("R_", [16, 64, 256])
def test_rotary_angles_at_far_positions(R_, pairs):
    """Positions whose product with f_i is itself rounded in 64 bits: the definition takes whole turns off exactly."""
    assert exact_angle(1, 1.0) == 1.0 and abs(exact_angle(10 ** 9, 1.0) - np.arctan2(np.sin(1e9), np.cos(1e9))) < 1e-12
    rng = np.random.default_rng(R_)
    lens, pos = [4, 3, 5, 6, 2], [2 ** 31 - 1 - 3, -2 ** 31, 1 << 30, 131071, 987654321]
    T, H, cu = sum(lens), 3, cu_from_lengths(lens)
    at = [pos[b] + i for b, n in enumerate(lens) for i in range(n)]
    x = bf16(rng.standard_normal((T, H, R_)))
    first = np.arange(0, R_, 2) if pairs else np.arange(R_ // 2)
    second = first + 1 if pairs else first + R_ // 2
    x[:, 0, first], x[:, 0, second] = 1.0, 0.0  # cosines and sines themselves
    f, _ = ops.rotary_inv_freq(R_)
    for inverse in (False, True):
        got = f64(ops.rotary(x, f, dev(cu), pos=dev(np.array(pos, np.int32)), interleaved=pairs, inverse=inverse)[0])
        for t, p in enumerate(at):
            theta = np.array([exact_angle(p, v) for v in f64(f)]) * (-1 if inverse else 1)
            c, s = np.cos(theta), np.sin(theta)
            a, b = f64(x[t])[:, first], f64(x[t])[:, second]
            # the angle: 2^-25 of half a turn in fp32 and, of the fixed point, 2^-33 of a turn and p * 2^-61 of f_i
            # (both below 2^-29); cosine, sine and products a few 2^-24 each
            e = np.pi * 2.0 ** -25 + 2.0 ** -28 + 8 * R.F32
            for want, i in ((a * c - b * s, first), (a * s + b * c, second)):
                tol = e * (np.abs(a) + np.abs(b)) + R.BF16 * np.abs(want)
                assert (np.abs(got[t][:, i] - want) <= tol).all(), (p, inverse)
