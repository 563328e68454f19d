"""Norm (with its backward pass) and rotary positions on the GPU against their
64-bit definitions, within bounds that rows_ref derives."""
import math

import numpy as np
import pytest
import torch

import rows_ref as R
from gpu_util import DEV, cu_from_lengths, dev
from sparse_attention_gemm_gb300 import ops

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def draw(rng, *shape, spread=2.0):
    """bf16 rows of different sizes on the device."""
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, (shape[0],) + (1,) * (len(shape) - 1)))
    return torch.from_numpy(x.astype(np.float32)).to(DEV).to(torch.bfloat16)


def apart(x, gap):
    """The same rows, `gap` elements apart, with other values between them."""
    if not gap:
        return x
    wide = torch.full((x.shape[0], x.shape[1] + gap), 7.0, dtype=x.dtype, device=DEV)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def f64(t):
    return t.double().cpu().numpy()


def near(got, want, tol, name):
    g = f64(got)
    assert np.isfinite(g).all(), f"{name}: not finite"
    over = np.abs(g - want) - tol
    assert (over <= 0).all(), f"{name}: {over.max():.3g} over its bound"


WIDTHS = [8, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T,residual,gap", [(1, False, 0), (3, True, 0), (37, True, 64), (301, False, 8)])
def test_norm(D, T, residual, gap):
    rng = np.random.default_rng(D + T)
    x, r = apart(draw(rng, T, D), gap), apart(draw(rng, T, D), 2 * gap) if residual else None
    w = rng.standard_normal(D).astype(np.float32)
    h, rstd, y = R.norm(f64(x), w.astype(np.float64), EPS, None if r is None else f64(r))
    ts, tr, ty = R.norm_bounds(h, rstd, y)
    got = ops.rms_norm_fwd(x, dev(w), EPS, residual=r, want_rstd=True)
    assert set(got) == {"out", "rstd"} | ({"sum"} if residual else set())
    near(got["out"], y, ty, "out")
    near(got["rstd"], rstd, tr, "rstd")
    if residual:
        near(got["sum"], h, ts, "sum")
    # into rows that lie apart: the same bits, and nothing between them
    out, total = apart(torch.zeros(T, D, dtype=torch.bfloat16, device=DEV), 24), apart(torch.zeros(T, D, dtype=torch.bfloat16, device=DEV), 8)
    again = ops.rms_norm_fwd(x, dev(w), EPS, residual=r, out=out, sum_out=total)
    assert again["out"].data_ptr() == out.data_ptr() and torch.equal(out, got["out"])
    assert torch.equal(total, got["sum"] if residual else x)
    for t in (out, total):
        gaps = t.as_strided((T, t.stride(0) - D), (t.stride(0), 1), t.storage_offset() + D)
        assert bool((gaps == 7.0).all())


@pytest.mark.parametrize("fmt,group,D", [("mxfp8", 32, d) for d in (32, 64, 96)] + [
    (f, g, d) for f, g in (("e4m3", 128), ("mxfp8", 32))
    for d in (128, 256, 384, 512, 640, 1024, 1152, 2048, 4096, 5120, 8192, 16384)])
@pytest.mark.parametrize("T,residual", [(1, True), (70, False)])
def test_norm_in_8_bits(fmt, group, D, T, residual):
    rng = np.random.default_rng(D + T)
    x, r = draw(rng, T, D, spread=6.0), draw(rng, T, D) if residual else None
    w = (rng.standard_normal(D) * np.exp2(rng.integers(-12, 12, D))).astype(np.float32)
    w[: group // 2] = 0  # small and empty groups
    if D >= 2 * group:
        w[group:2 * group] = 0
    _, _, y = R.norm(f64(x), w.astype(np.float64), EPS, None if r is None else f64(r))
    got = ops.rms_norm_fwd(x, dev(w), EPS, residual=r, fmt=fmt)
    s = got["scale"].cpu().numpy()
    assert got["out"].dtype == torch.uint8 and s.shape == (T, D // group)
    s = s.astype(np.float64) if fmt == "e4m3" else np.exp2(s.astype(np.float64) - 127)
    R.check_codes(got["out"].cpu().numpy(), s, y, group)
    # the same codes into rows apart and scales of the caller's
    out, scale = apart(torch.zeros(T, D, dtype=torch.uint8, device=DEV), 8), torch.empty_like(got["scale"])
    ops.rms_norm_fwd(x, dev(w), EPS, residual=r, fmt=fmt, out=out, scale=scale)
    assert torch.equal(out, got["out"]) and torch.equal(scale, got["scale"])


@pytest.mark.parametrize("D", [64, 512, 4096])
def test_norm_of_odd_rows(D):
    """Zeros, infinities, NaN, tiny and large values: each row by itself."""
    rng = np.random.default_rng(D)
    x = draw(rng, 9, D)
    x[1], x[2, 5], x[3, 7], x[4, 0] = 0, float("nan"), float("inf"), -float("inf")
    x[5], x[6] = 1e-38, 1e18
    w = dev(np.ones(D, np.float32))
    got = ops.rms_norm_fwd(x, w, EPS, want_rstd=True)
    out, rstd = got["out"].float(), got["rstd"]
    clean = ops.rms_norm_fwd(x[[0, 7, 8]], w, EPS)["out"]
    assert torch.equal(got["out"][[0, 7, 8]], clean)
    assert bool((out[1] == 0).all()) and abs(float(rstd[1]) - 1e3) < 1e-2
    assert bool(out[2].isnan().all())
    for t, c in ((3, 7), (4, 0)):  # an infinite row: rstd 0, 0 * inf is NaN, everything else 0
        assert float(rstd[t]) == 0 and bool(out[t, c].isnan()) and int(out[t].isnan().sum()) == 1
    assert bool((out[5].abs() <= 1e-34).all()) and bool(((out[6] - 1).abs() <= 2.0 ** -8).all())
    if D % 128 == 0:
        q = ops.rms_norm_fwd(x, w, EPS, fmt="e4m3")
        codes = q["out"]
        assert bool(((codes[2] & 127) == 127).all()) and int(((codes[3] & 127) == 127).sum()) == 1
        assert bool((codes[1] == 0).all()) and bool((q["scale"][1] == 2.0 ** -126).all())
        assert torch.equal(codes[[0, 7, 8]], ops.rms_norm_fwd(x[[0, 7, 8]], w, EPS, fmt="e4m3")["out"])


def test_norm_in_8_bits_of_infinite_weights():
    """An infinity in y becomes the largest code and does not touch its group's scale."""
    x = torch.ones(2, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, device=DEV)
    w[3], w[200] = float("inf"), -float("inf")
    got = ops.rms_norm_fwd(x, w, EPS, fmt="e4m3")
    assert bool((got["scale"] == 2.0 ** -8).all())  # 1 <= 448 * 2^-8 < 2
    c = got["out"].view(torch.float8_e4m3fn).float()
    assert bool((c[:, 3] == 448).all()) and bool((c[:, 200] == -448).all()) and bool((c[:, 0] == 256).all())


@pytest.mark.parametrize("D", [64, 256, 1024, 4096, 16384])
def test_norm_in_place(D):
    rng = np.random.default_rng(D)
    x, r, w = draw(rng, 130, D), draw(rng, 130, D), dev(rng.standard_normal(D).astype(np.float32))
    want = ops.rms_norm_fwd(x, w, EPS, residual=r)
    a, b = x.clone(), r.clone()
    got = ops.rms_norm_fwd(a, w, EPS, residual=b, out=a, sum_out=b)
    assert torch.equal(a, want["out"]) and torch.equal(b, want["sum"]) and got["sum"].data_ptr() == b.data_ptr()
    dy, rstd = draw(rng, 130, D), ops.rms_norm_fwd(x, w, EPS, want_rstd=True)["rstd"]
    want = ops.rms_norm_bwd(dy, x, w, rstd, d_sum=r)
    for name in ("dy", "x", "d_sum"):
        t = {"dy": dy.clone(), "x": x.clone(), "d_sum": r.clone()}
        got = ops.rms_norm_bwd(t["dy"], t["x"], w, rstd, d_sum=t["d_sum"], dx=t[name])
        assert torch.equal(t[name], want["dx"]) and torch.equal(got["dweight"], want["dweight"]), name


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T,residual,gap", [(1, True, 0), (45, False, 8), (1500, True, 0)])
def test_norm_backward(D, T, residual, gap):
    rng = np.random.default_rng(D + T)
    x, dy = apart(draw(rng, T, D), gap), apart(draw(rng, T, D), gap)
    ds = apart(draw(rng, T, D), 3 * gap) if residual else None
    w = rng.standard_normal(D).astype(np.float32)
    rstd = ops.rms_norm_fwd(x, dev(w), EPS, want_rstd=True)["rstd"]
    dx, dw, tx, tw = R.norm_back(f64(dy), f64(x), w.astype(np.float64), f64(rstd), None if ds is None else f64(ds))
    got = ops.rms_norm_bwd(dy, x, dev(w), rstd, d_sum=ds)
    near(got["dx"], dx, tx, "dx")
    near(got["dweight"], dw, tw, "dweight")
    out = apart(torch.zeros(T, D, dtype=torch.bfloat16, device=DEV), 8)
    ws = torch.full((ops.rms_norm_bwd_workspace_size(T, D),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):  # the same bits each time, whatever the workspace held
        again = ops.rms_norm_bwd(dy, x, dev(w), rstd, d_sum=ds, dx=out, workspace=ws)
        assert torch.equal(out, got["dx"]) and torch.equal(again["dweight"], got["dweight"])
    alone = ops.rms_norm_bwd(dy, x, dev(w), rstd, d_sum=ds, want_dweight=False)
    assert alone["dweight"] is None and torch.equal(alone["dx"], got["dx"])


def test_norm_backward_of_many_rows():
    """More rows than groups in flight, rows of 128 as query heads are."""
    rng = np.random.default_rng(5)
    x, dy = draw(rng, 70001, 128), draw(rng, 70001, 128)
    w = rng.standard_normal(128).astype(np.float32)
    rstd = ops.rms_norm_fwd(x, dev(w), EPS, want_rstd=True)["rstd"]
    dx, dw, tx, tw = R.norm_back(f64(dy), f64(x), w.astype(np.float64), f64(rstd))
    got = ops.rms_norm_bwd(dy, x, dev(w), rstd)
    near(got["dx"], dx, tx, "dx")
    near(got["dweight"], dw, tw, "dweight")


def test_norm_without_rows():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    got = ops.rms_norm_fwd(x, w, EPS, residual=x, want_rstd=True)
    assert got["out"].shape == (0, 64) and got["rstd"].shape == (0,)
    got = ops.rms_norm_bwd(x, x, w, got["rstd"])
    assert bool((got["dweight"] == 0).all())


# -------------------------------------------------------------------- rotary
def positions_of(cu, pos, T):
    out = [None] * T
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            out[t] = (0 if pos is None else int(pos[b])) + t - int(cu[b])
    return out


def part(rng, T, H, R_, ld, lead):
    """[T, H, R] as a part of heads of ld, after `lead` elements."""
    return draw(rng, T, H, ld)[..., lead:lead + R_]


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("R_,H,H2,lens,pos,pad,ld,lead", [
    (16, 1, 0, [1], None, 0, 16, 0),
    (64, 128, 1, [1, 1, 1, 1], [0, 1, 4095, 131071], 2, 576, 512),
    (64, 3, 2, [70, 0, 5], [0, 9, 1 << 20], 1, 128, 64),
    (128, 24, 2, [33, 300], None, 0, 128, 0),
    (256, 7, 1, [41], [2 ** 31 - 50], 0, 256, 0),
    (1024, 2, 1, [9, 4], [-3, 77], 3, 1032, 8),
    (32, 1, 0, [5000], None, 11, 40, 8),
    (48, 5, 3, [257], [100000], 0, 64, 16),
    (64, 64, 1, [900, 1400], [0, 77], 3, 72, 8),
    (256, 120, 5, [3, 0, 20], [5, 0, 999], 2, 256, 0),
    (1024, 7, 1, [1], [65535], 0, 1024, 0),
    (16, 1000, 24, [130], [7], 4, 16, 0),
])
def test_rotary(pairs, R_, H, H2, lens, pos, pad, ld, lead):
    rng = np.random.default_rng(R_ + H + len(lens))
    T, cu = sum(lens) + pad, cu_from_lengths(lens)
    x, x2 = part(rng, T, H, R_, ld, lead), part(rng, T, H2, R_, ld, lead) if H2 else None
    f, mul = ops.rotary_inv_freq(R_, scaling="yarn" if H2 else "plain", factor=40.0)
    at = positions_of(cu, pos, T)
    dpos = None if pos is None else dev(np.array(pos, np.int32))
    for inverse in (False, True):
        outs = [torch.full((T, h, ld + 8), 7.0, dtype=torch.bfloat16, device=DEV) for h in (H, max(H2, 1))]
        out, out2 = (o[..., lead:lead + R_] for o in outs)
        got = ops.rotary(x, f, dev(cu), pos=dpos, x2=x2, interleaved=pairs, mul=mul, inverse=inverse, out=out,
                         out2=out2 if H2 else None)
        for src, whole, o, g in ((x, outs[0], out, got[0]), (x2, outs[1], out2, got[1])):
            if src is None:
                assert g is None and bool((whole == 7.0).all())
                continue
            want, tol = R.rotary(f64(src), f64(f), at, pairs, inverse, mul)
            rows = np.array([a is not None for a in at])
            assert g.data_ptr() == o.data_ptr()
            near(o[dev(rows)], want[rows], tol[rows], "rotary")
            assert bool((o[dev(~rows)] == 7.0).all())
            assert bool((whole[..., :lead] == 7.0).all()) and bool((whole[..., lead + R_:] == 7.0).all())
        # new outputs and in place: the same bits
        live = dev(np.array([a is not None for a in at]))
        new = ops.rotary(x, f, dev(cu), pos=dpos, x2=x2, interleaved=pairs, mul=mul, inverse=inverse)
        assert torch.equal(new[0][live], out[live])
        keep = torch.empty(T, H, ld, dtype=torch.bfloat16, device=DEV)
        keep[..., lead:lead + R_] = x
        mine = keep[..., lead:lead + R_]
        ops.rotary(mine, f, dev(cu), pos=dpos, interleaved=pairs, mul=mul, inverse=inverse, out=mine)
        assert torch.equal(mine[live], out[live]) and torch.equal(mine[~live], x[~live])


@pytest.mark.parametrize("pairs", [True, False])
def test_rotary_heads_before_tokens_and_shared_rows(pairs):
    """Heads outermost in memory, and one row read for every head."""
    rng = np.random.default_rng(3)
    T, H, cu = 50, 6, dev(cu_from_lengths([20, 30]))
    x = draw(rng, H, T, 64).transpose(0, 1)
    f, _ = ops.rotary_inv_freq(64)
    want = ops.rotary(x.contiguous(), f, cu, interleaved=pairs)[0]
    out = torch.empty(H, T, 64, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert torch.equal(ops.rotary(x, f, cu, interleaved=pairs, out=out)[0], want)
    one = x[:, :1].expand(T, H, 64)
    got = ops.rotary(one, f, cu, interleaved=pairs)[0]
    assert torch.equal(got, want[:, :1].expand(T, H, 64))


def test_rotary_there_and_back():
    """The adjoint of a rotation is its inverse: each way rounds once (2^-8 of the pair's length)."""
    rng = np.random.default_rng(4)
    x, cu = draw(rng, 300, 5, 64), dev(cu_from_lengths([300]))
    f, _ = ops.rotary_inv_freq(64)
    pos = dev(np.array([1 << 30], np.int32))
    there = ops.rotary(x, f, cu, pos=pos)[0]
    back = ops.rotary(there, f, cu, pos=pos, inverse=True)[0]
    size = x.double().unflatten(2, (-1, 2)).norm(dim=3).repeat_interleave(2, 2)
    # the two roundings of a pair, turned: sqrt(2) * 2^-8 of its length, and the one of the way back
    assert bool(((back.double() - x.double()).abs() <= (math.sqrt(2) + 1.01) * 2.0 ** -8 * size).all())


def test_calls_without_tokens():
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    f, _ = ops.rotary_inv_freq(64)
    assert ops.rotary(x, f, dev(cu_from_lengths([0])))[0].shape == (0, 2, 64)


# ------------------------------------------------------------ ways to call them
def test_streams_and_captures():
    """Captured with a workspace each, replayed with new inputs in place and on another stream."""
    rng = np.random.default_rng(7)
    f, mul = ops.rotary_inv_freq(64, scaling="yarn", factor=4.0)
    made = []
    for T, D in ((5, 512), (300, 4096)):
        st = {"x": draw(rng, T, D), "r": draw(rng, T, D), "dy": draw(rng, T, D), "w": dev(rng.standard_normal(D).astype(np.float32)),
              "cu": dev(cu_from_lengths([T])), "ws": torch.empty(ops.rms_norm_bwd_workspace_size(T, D), dtype=torch.uint8, device=DEV)}

        def step(st=st):
            a = ops.rms_norm_fwd(st["x"], st["w"], EPS, residual=st["r"], want_rstd=True)
            b = ops.rms_norm_bwd(st["dy"], a["sum"], st["w"], a["rstd"], workspace=st["ws"])
            c = ops.rotary(a["out"].view(a["out"].shape[0], -1, 64), f, st["cu"], mul=mul)[0]
            d = ops.rms_norm_fwd(st["x"], st["w"], EPS, fmt="mxfp8")
            return [a["out"], a["sum"], b["dx"], b["dweight"], c, d["out"], d["scale"]]

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        made.append((graph, st, step, res))
    side = torch.cuda.Stream()
    for i in range(3):
        for graph, st, step, res in made:
            for k in ("x", "r", "dy"):
                st[k].copy_(torch.randn_like(st[k].float()).to(torch.bfloat16))
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side if i == 1 else torch.cuda.current_stream()):
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
            got = [t.clone() for t in res]
            assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_bindings_refuse():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV), torch.ones(256, device=DEV)
    rstd, f = torch.ones(4, device=DEV), torch.ones(32, dtype=torch.float64, device=DEV)
    cu, q = dev(cu_from_lengths([4])), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    wide = torch.zeros(4, 516, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: ops.rms_norm_fwd(x, w[:128], EPS), lambda: ops.rms_norm_fwd(x, w, 0.0),
                lambda: ops.rms_norm_fwd(x, w, EPS, residual=x[:3]), lambda: ops.rms_norm_fwd(x, w, EPS, out=x[:, :128]),
                lambda: ops.rms_norm_fwd(x[:, ::2], w[:128], EPS), lambda: ops.rms_norm_fwd(x, w, EPS, fmt="fp4"),
                lambda: ops.rms_norm_fwd(wide[:, :256], w, EPS), lambda: ops.rms_norm_fwd(wide[:, 1:257], w, EPS),
                lambda: ops.rms_norm_fwd(x, w, EPS, scale=rstd), lambda: ops.rms_norm_fwd(x.cpu(), w, EPS),
                lambda: ops.rms_norm_fwd(x, w.cpu(), EPS), lambda: ops.rms_norm_fwd(x, w, EPS, sum_out=x, out=x),
                lambda: ops.rms_norm_bwd(x, x, w, rstd[:3]), lambda: ops.rms_norm_bwd(x[:3], x, w, rstd),
                lambda: ops.rms_norm_bwd(x, x, w, rstd, d_sum=x[:, :64]),
                lambda: ops.rms_norm_bwd(x, x, w, rstd, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
                lambda: ops.rotary(q, f[:16], cu), lambda: ops.rotary(q, f, cu, pos=cu), lambda: ops.rotary(q, f, cu, x2=q[:3]),
                lambda: ops.rotary(q, f, cu, out2=q), lambda: ops.rotary(q, f, cu, out=q[:, :1].expand(4, 2, 64)),
                lambda: ops.rotary(q[..., ::2], f[:16], cu), lambda: ops.rotary(q.cpu(), f, cu),
                lambda: ops.rotary(q, f, cu, mul=float("nan")), lambda: ops.rotary(q[..., :24], f[:12], cu)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.rms_norm_fwd(x.float(), w, EPS), lambda: ops.rms_norm_fwd(x, w.to(torch.bfloat16), EPS),
                lambda: ops.rms_norm_bwd(x, x, w, rstd.double()), lambda: ops.rotary(q, f.float(), cu),
                lambda: ops.rotary(q, f, cu.long()), lambda: ops.rotary(q.half(), f, cu)):
        with pytest.raises(TypeError):
            bad()
