"""Cases that measure what stands around sparse attention in a layer: the
root-mean-square norm with its backward pass, rotary positions, a cache of
microscaled 4-bit rows, and sparse attention over that cache.

4-bit cache: codes uint8 [n_blocks, block, Hc, D / 2] (E2M1, element 2i in the
low half of byte i), scale uint8 [n_blocks, block, Hc, D / 32] (E8M0: byte e
stands for 2^(e - 127)); a value is e2m1(code) times its 32 elements' scale.
Position p of sequence b lives in row block_table[b, p // block] * block + p %
block, or in row p without a table.
"""
import math

import torch

own = False

EPS = 1e-6
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]

# The smallest calls are single decode steps, where latency counts; the
# largest are whole prompts, a training batch and a prompt's chunk.
_LISTED = [
    # a decode step's hidden rows: residual added, output in E4M3 with one scale per 128
    {"name": "norm decode 8 bit", "op": "norm", "T": 64, "D": 4096, "ld": 4096, "residual": True, "fmt": "e4m3"},
    # whole prompts' hidden rows, residual added
    {"name": "norm prompts", "op": "norm", "T": 16384, "D": 4096, "ld": 4096, "residual": True, "fmt": "bf16"},
    # training, norm of query heads of 256: many short rows
    {"name": "norm back heads", "op": "norm_back", "T": 24216, "D": 256, "residual": False},
    # training, hidden rows with the residual's gradient
    {"name": "norm back hidden", "op": "norm_back", "T": 8192, "D": 4096, "residual": True},
    # a decode step's queries and latent key: the last 64 of 576, written into the rows that attention takes
    {"name": "rotary decode", "op": "rotary", "T": 32, "seqs": 32, "ctx": 16384, "H": 128, "R": 64, "ld": 576,
     "pairs": True, "scaled": True, "back": False},
    # a long prompt's indexer queries and key, halves of 64 of their 128, positions scaled
    {"name": "rotary index 16k", "op": "rotary", "T": 16384, "seqs": 1, "ctx": 0, "H": 64, "R": 64, "ld": 128,
     "pairs": False, "scaled": True, "back": False},
    # training, gradients of packed grouped heads of 256, the whole head rotated
    {"name": "rotary back gqa", "op": "rotary", "T": 4099, "seqs": 5, "ctx": 0, "H": 24, "R": 256, "ld": 256,
     "pairs": False, "scaled": False, "back": True},
    # one new token for each of 64 running sequences into the cache, and its row as later steps see it
    {"name": "cache decode 64", "op": "cache", "seqs": 64, "tokens": 64, "ctx": 8192, "heads": 1, "dim": 576,
     "block": 64, "table": True, "pad": 0},
    # whole prompts into the cache and back for dense attention over the prefix
    {"name": "cache prompts 16k", "op": "cache", "seqs": 4, "tokens": 16384, "ctx": 0, "heads": 1, "dim": 576,
     "block": 64, "table": True, "pad": 0},
    # one token of one long sequence
    {"name": "attn single token", "op": "attn", "T": 1, "seqs": 1, "ctx": 65536, "H": 64, "heads": 1, "dqk": 576,
     "dv": 512, "K": 2048, "block": 64, "table": True, "sink": True},
    # a decode step of grouped heads with keys and values of 256, flat cache
    {"name": "attn decode gqa", "op": "attn", "T": 96, "seqs": 96, "ctx": 4096, "H": 24, "heads": 2, "dqk": 256,
     "dv": 256, "K": 1027, "block": 16, "table": False, "sink": False},
    # a chunk of a long prompt
    {"name": "attn chunk 2k", "op": "attn", "T": 2048, "seqs": 1, "ctx": 14336, "H": 64, "heads": 1, "dqk": 576,
     "dv": 512, "K": 2048, "block": 64, "table": True, "sink": True},
]


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "rotary", "cache", "attn", "attn"])
    if op == "norm":
        fmt = rng.choice(["bf16", "bf16", "e4m3", "mxfp8"])
        D = 128 * _log(rng, 1, 64) if fmt != "bf16" else 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, min(65536, 16384 * 4096 // D) if fmt == "bf16" else 512)
        return {"op": op, "T": T, "D": D, "ld": D + rng.choice([0, 0, 64]), "residual": rng.random() < 0.6, "fmt": fmt}
    if op == "norm_back":
        D = 8 * _log(rng, 8, 1024)
        return {"op": op, "T": _log(rng, 1, min(65536, 8192 * 4096 // D)), "D": D, "residual": rng.random() < 0.5}
    if op == "rotary":
        R = rng.choice([16, 32, 64, 64, 64, 128, 256])
        H = rng.choice([1, 2, 12, 24, 64, 128])
        T = _log(rng, 1, min(32768, 16384 * 64 * 64 // (H * R)))
        return {"op": op, "T": T, "seqs": rng.randint(1, min(T, 64)), "ctx": rng.choice([0, 5000, 1000000]), "H": H,
                "R": R, "ld": R + rng.choice([0, 64, 512]), "pairs": rng.random() < 0.5, "scaled": rng.random() < 0.5,
                "back": rng.random() < 0.4}
    if op == "cache":
        heads, dim, block = rng.choice([(1, 576, 64), (1, 576, 32), (1, 512, 128), (1, 128, 1), (2, 256, 16),
                                        (4, 256, 64), (8, 128, 32), (1, 96, 16)])
        tokens = _log(rng, 1, min(32768, 16384 * 576 // (heads * dim)))
        return {"op": op, "seqs": rng.randint(1, min(tokens, 64)), "tokens": tokens, "ctx": rng.choice([0, 100, 3000]),
                "heads": heads, "dim": dim, "block": block, "table": rng.random() < 0.7 or block > 1,
                "pad": rng.choice([0, 0, 13])}
    dqk, dv = rng.choice([(576, 512), (576, 512), (512, 512), (256, 256)])
    heads = rng.choice([1, 2]) if dqk == 256 else 1
    H = heads * (rng.choice([1, 6, 12, 16]) if dqk == 256 else rng.choice([16, 32, 64, 100, 128]))
    T = _log(rng, 1, 2048)
    K = min(_log(rng, 16, 2048), max(16, 2048 * 2048 * 64 // (T * max(H, 64))))
    decode = T <= 128 and rng.random() < 0.7
    return {"op": op, "T": T, "seqs": T if decode else rng.randint(1, min(T, 4)), "ctx": _log(rng, 256, 16384), "H": H,
            "heads": heads, "dqk": dqk, "dv": dv, "K": K, "block": rng.choice([1, 16, 32, 64, 128]),
            "table": rng.random() < 0.7, "sink": rng.random() < 0.7}


# ---------------------------------------------------------------- geometry
def _parts(total, n):
    """total split into n uneven positive parts, the same for every seed."""
    w = [1 + (i * 7919) % 13 for i in range(n)]
    left = total - n
    out = [1 + left * x // sum(w) for x in w]
    out[-1] += total - sum(out)
    return out


def _sequences(case):
    """(new tokens, earlier tokens) of each sequence."""
    n = case["seqs"]
    new = _parts(case["tokens"] if case["op"] == "cache" else case["T"], n)
    ctx = [case["ctx"] * (i + 1) // n + (i % 5 if case["ctx"] else 0) for i in range(n)]
    return new, ctx


def _lengths(case):
    """Selected slots of each query: min(K, its position + 1), and none for the odd masked row."""
    new, ctx = _sequences(case)
    n = [min(case["K"], c + i + 1) for c, k in zip(ctx, new) for i in range(k)]
    return [0 if t % 97 == 50 else x for t, x in enumerate(n)]


def _pages(case, new, ctx, gen):
    """Block table (drawn) or flat first rows, and the number of blocks of the cache."""
    block, n = case["block"], case["seqs"]
    need = [(c + k + block - 1) // block for c, k in zip(ctx, new)]
    width, total = max(need), sum(need)
    if not case["table"]:
        first = [sum(need[:i]) * block for i in range(n)]
        return None, torch.tensor(first, dtype=torch.int32, device="cuda"), total
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, None, total


def _rows(n, heads, dim, gen):
    """Rows as a model's projections give them: normal values, rows of different size, a few large channels."""
    x = torch.randn(n, heads, dim, generator=gen, device="cuda")
    x *= 0.5 + torch.rand(n, 1, 1, generator=gen, device="cuda")
    x[..., ::61] *= 4
    return x.to(torch.bfloat16)


def _inv_freq(case):
    """Angle per position of each pair, and the factor of the result: base 10000, or that stretched from 4096
    positions by 40, fast pairs kept, slow ones divided, those between blended (YaRN)."""
    half = case["R"] // 2
    f = [10000.0 ** (-i / half) for i in range(half)]
    if not case["scaled"]:
        return f, 1.0
    factor, first = 40.0, 4096

    def at(turns):  # the pair that makes so many turns over the first positions
        return half * math.log(first / (turns * 2 * math.pi)) / math.log(10000.0)

    lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), case["R"] - 1)
    keep = [1 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(half)]
    return [x * k + x / factor * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0


def _random_cache(blocks, block, heads, dim, gen):
    """A filled cache: drawn rows, quantised."""
    codes = torch.empty(blocks * block, heads, dim // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(blocks * block, heads, dim // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (heads * dim))
    for i in range(0, blocks * block, step):
        n = min(step, blocks * block - i)
        codes[i:i + n], scale[i:i + n] = _quantise(_rows(n, heads, dim, gen).float())
    return codes.view(blocks, block, heads, -1), scale.view(blocks, block, heads, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("norm", "norm_back"):
        T, D = case["T"], case["D"]
        w = 1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")
        if op == "norm_back":
            x = _rows(T, 1, D, gen)[:, 0]
            return {"op": op, "x": x, "w": w, "dy": _rows(T, 1, D, gen)[:, 0],
                    "rstd": torch.rsqrt(x.float().square().mean(1) + EPS),
                    "d_sum": _rows(T, 1, D, gen)[:, 0] if case["residual"] else None}
        # the rows may be the first part of wider ones
        x = _rows(T, 1, case["ld"], gen)[:, 0, :D]
        return {"op": op, "x": x, "w": w, "fmt": case["fmt"], "r": _rows(T, 1, D, gen)[:, 0] if case["residual"] else None}
    new, ctx = _sequences(case)
    if op == "rotary":
        T, H, R, ld = case["T"], case["H"], case["R"], case["ld"]
        f, mul = _inv_freq(case)
        return {"op": op, "q": torch.randn(T, H, R, generator=gen, device="cuda").to(torch.bfloat16),
                "k": torch.randn(T, ld, generator=gen, device="cuda").to(torch.bfloat16)[:, ld - R:].unsqueeze(1),
                "q_out": torch.zeros(T, H, ld, dtype=torch.bfloat16, device="cuda")[..., ld - R:],
                "k_out": torch.zeros(T, 1, ld, dtype=torch.bfloat16, device="cuda")[..., ld - R:],
                "f": torch.tensor(f, dtype=torch.float64, device="cuda"), "mul": mul, "pairs": case["pairs"],
                "back": case["back"], "cu": torch.tensor([0] + new, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32),
                "pos": torch.tensor(ctx, dtype=torch.int32, device="cuda")}
    table, first, blocks = _pages(case, new, ctx, gen)
    cu = torch.tensor([0] + new, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    pos = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    if first is not None:
        pos = pos + first
    s = {"op": op, "cu": cu, "pos": pos, "table": table, "block": case["block"]}
    if op == "cache":
        s["T"] = case["tokens"] + case["pad"]
        s["cache"], s["scale"] = _random_cache(blocks, case["block"], case["heads"], case["dim"], gen)
        s["src"] = _rows(s["T"], case["heads"], case["dim"], gen)
        # the program's buffer for the rows: those behind the last sequence stay as they are
        s["out"] = torch.zeros(s["T"], case["heads"], case["dim"], dtype=torch.bfloat16, device="cuda")
        return s
    T, K, H = case["T"], case["K"], case["H"]
    s["cache"], s["scale"] = _random_cache(blocks, case["block"], case["heads"], case["dqk"], gen)
    s["v"], s["v_scale"] = (None, None) if case["dqk"] != 256 else _random_cache(blocks, case["block"], case["heads"],
                                                                                case["dv"], gen)
    s["q"] = torch.randn(T, H, case["dqk"], generator=gen, device="cuda").to(torch.bfloat16)
    s["sm"] = 1.0 / math.sqrt(case["dqk"])
    s["sink"] = torch.randn(H, generator=gen, device="cuda") if case["sink"] else None
    # query t of sequence b stands at position p and selects positions up to its own
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    p = torch.tensor(ctx, device="cuda")[b] + t - cu[b]
    length = torch.tensor(_lengths(case), device="cuda")
    j = torch.arange(K, device="cuda")
    u = torch.rand(T, K, generator=gen, device="cuda")
    ids = ((j + u) * ((p + 1) / length.clamp(min=1))[:, None]).floor().to(torch.int64)
    ids = torch.minimum(ids, p[:, None])
    if first is not None:
        ids = ids + first.to(torch.int64)[b][:, None]
    s["idx"] = torch.where(j < length[:, None], ids, -1).to(torch.int32)
    s["len"] = length.to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms
def _power(e):
    """2^e in fp32, exactly (e from -126 on)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None] * s["w"]
    out = {"rstd": rstd}
    if s["r"] is not None:
        out["sum"] = h.to(torch.bfloat16)
    if s["fmt"] == "bf16":
        return {**out, "y": y.to(torch.bfloat16)}
    group = 128 if s["fmt"] == "e4m3" else 32
    y = y.view(y.shape[0], -1, group)
    # smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9)
    m, x = torch.frexp(y.abs().amax(2))
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(m > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    scale = _power(e)
    codes = (y / scale[:, :, None]).to(torch.float8_e4m3fn).flatten(1)
    return {**out, "y": codes, "scale": scale if group == 128 else (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _norm_back(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = x * rstd
    g = dy * s["w"]
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0)}


def _rotary(s):
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    p = s["pos"].long()[b] + t - s["cu"].long()[b]
    angle = p.double()[:, None] * s["f"]
    if s["back"]:
        angle = -angle
    c, n = (torch.cos(angle) * s["mul"]).float()[:, None], (torch.sin(angle) * s["mul"]).float()[:, None]
    out = {}
    for name, x, to in (("q", s["q"].float(), s["q_out"]), ("k", s["k"].float(), s["k_out"])):
        half = x.shape[2] // 2
        a, b = (x[..., 0::2], x[..., 1::2]) if s["pairs"] else (x[..., :half], x[..., half:])
        u, v = a * c - b * n, a * n + b * c
        to.copy_(torch.stack((u, v), 3).flatten(2) if s["pairs"] else torch.cat((u, v), 2))
        out[name] = to
    return out


def _row_of(s, t, positions):
    """Cache row of each position of the sequence that holds token t; -1 where there is none."""
    n = s["cu"].numel() - 1
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    inside = b < n
    b = b.clamp(max=n - 1)
    if positions is None:
        positions = s["pos"].long()[b] + t - s["cu"].long()[b]
    block, n_blocks = s["block"], s["cache"].shape[0]
    if s["table"] is None:
        row = positions
    else:
        at = b if positions.dim() == 1 else b[:, None].expand_as(positions)
        page = torch.where(positions < 0, 0, positions // block)
        fits = page < s["table"].shape[1]
        phys = s["table"].long()[at, page.clamp(max=s["table"].shape[1] - 1)]
        row = torch.where(fits & (phys >= 0) & (phys < n_blocks), phys * block + positions % block, -1)
    row = torch.where((positions >= 0) & (row < n_blocks * block), row, -1)
    return torch.where(inside if row.dim() == 1 else inside[:, None], row, -1)


def _quantise(x):
    """Codes and scale bytes of fp32 rows [..., D]: per 32 the smallest e with amax <= 6 * 2^e (6 = 0.75 * 2^3)."""
    g = x.unflatten(-1, (-1, 32))
    m, k = torch.frexp(g.abs().amax(-1))
    e = torch.where(m <= 0.75, k - 3, k - 2)
    e = torch.where(m > 0, e, torch.full_like(e, -126)).clamp(-126, 125)
    a = (g / _power(e)[..., None]).abs()
    # to nearest, ties to the even code
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = (c + 8 * torch.signbit(g).to(torch.uint8)).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], (e + 127).to(torch.uint8)


def _values(codes, scale):
    """fp32 values of codes [..., D / 2] and scale bytes [..., D / 32]."""
    both = torch.tensor(E2M1 + [-x for x in E2M1], device="cuda")
    v = torch.stack((both[(codes & 15).int()], both[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _power(scale.int() - 127)[..., None]).flatten(-2)


def _cache(s):
    cache, scale = s["cache"].flatten(0, 1), s["scale"].flatten(0, 1)
    row = _row_of(s, torch.arange(s["T"], device="cuda"), None)
    keep = (row >= 0).nonzero()[:, 0]
    row = row[keep]
    cache[row], scale[row] = _quantise(s["src"][keep].float())
    s["out"][keep] = _values(cache[row], scale[row]).to(torch.bfloat16)
    return {"out": s["out"]}


def _attn(s):
    q = s["q"]
    T, H, _ = q.shape
    heads, K = s["cache"].shape[2], s["idx"].shape[1]
    group = H // heads
    row = _row_of(s, torch.arange(T, device="cuda"), s["idx"].long())
    valid = (row >= 0) & (torch.arange(K, device="cuda") < s["len"][:, None])
    row = torch.where(valid, row, 0)
    out, lse = [], []
    for h in range(heads):
        k = _values(s["cache"].flatten(0, 1)[:, h][row], s["scale"].flatten(0, 1)[:, h][row])
        v = k[:, :, :512] if s["v"] is None else _values(s["v"].flatten(0, 1)[:, h][row], s["v_scale"].flatten(0, 1)[:, h][row])
        x = torch.matmul(q[:, h * group:(h + 1) * group].float(), k.transpose(1, 2)) * s["sm"]
        x = x.masked_fill(~valid[:, None, :], -math.inf)
        sink = torch.full((group,), -math.inf, device="cuda") if s["sink"] is None else s["sink"][h * group:(h + 1) * group]
        m = torch.maximum(x.amax(2), sink)
        m = torch.where(m == -math.inf, 0.0, m)
        e = torch.exp(x - m[:, :, None])
        z = e.sum(2) + torch.exp(sink - m)
        out.append((torch.matmul(e, v) / torch.where(z > 0, z, 1.0)[:, :, None]).to(torch.bfloat16))
        lse.append(m + torch.log(z))
    return {"out": torch.cat(out, 1), "lse": torch.cat(lse, 1)}


_PLAIN = {"norm": _norm, "norm_back": _norm_back, "rotary": _rotary, "cache": _cache, "attn": _attn}


def run(state):
    s = state
    if not own:
        return _PLAIN[s["op"]](s)
    from sparse_attention_gemm_gb300 import ops

    if s["op"] == "norm":
        r = ops.rms_norm_fwd(s["x"], s["w"], EPS, residual=s["r"], fmt=s["fmt"], want_rstd=True)
        out = {"rstd": r["rstd"]}
        if s["r"] is not None:
            out["sum"] = r["sum"]
        if s["fmt"] == "bf16":
            return {**out, "y": r["out"]}
        scale = r["scale"]
        return {**out, "y": r["out"].view(torch.float8_e4m3fn),
                "scale": scale if s["fmt"] == "e4m3" else scale.view(torch.float8_e8m0fnu)}
    if s["op"] == "norm_back":
        r = ops.rms_norm_bwd(s["dy"], s["x"], s["w"], s["rstd"], d_sum=s["d_sum"])
        return {"dx": r["dx"], "dw": r["dweight"]}
    if s["op"] == "rotary":
        q, k = ops.rotary(s["q"], s["f"], s["cu"], pos=s["pos"], x2=s["k"], interleaved=s["pairs"], mul=s["mul"],
                          inverse=s["back"], out=s["q_out"], out2=s["k_out"])
        return {"q": q, "k": k}
    if s["op"] == "cache":
        ops.kv4_write(s["src"], s["cache"], s["scale"], s["cu"], pos=s["pos"], block_table=s["table"])
        return {"out": ops.kv4_read(s["cache"], s["scale"], s["cu"], s["T"], pos=s["pos"], block_table=s["table"],
                                    out=s["out"])}
    r = ops.sparse_attn_fwd_kv4(s["q"], s["cache"], s["scale"], s["idx"], s["sm"], topk_length=s["len"], sink=s["sink"],
                                v4=s["v"], v_scale=s["v_scale"], cu_seqlens=s["cu"] if s["table"] is not None else None,
                                block_table=s["table"])
    return {"out": r["out"], "lse": r["lse"]}


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "norm":
        n, group = case["T"] * case["D"], {"bf16": 0, "e4m3": 128, "mxfp8": 32}[case["fmt"]]
        out = 2 * n if not group else n + n // group * (4 if group == 128 else 1)
        return {"bytes": 2 * n * (3 if case["residual"] else 1) + out + 4 * (case["D"] + case["T"]), "flops": 5 * n}
    if op == "norm_back":
        n = case["T"] * case["D"]
        return {"bytes": 2 * n * (4 if case["residual"] else 3) + 4 * (case["T"] + 2 * case["D"]), "flops": 10 * n}
    if op == "rotary":
        n = case["T"] * (case["H"] + 1) * case["R"]
        return {"bytes": 4 * n + 4 * case["R"], "flops": 3 * n}
    new, ctx = _sequences(case)
    heads = case["heads"]
    if op == "cache":
        n = case["tokens"] * heads * case["dim"]
        return {"bytes": 4 * n + n // 2 + n // 32, "flops": 4 * n}
    T, H, dqk, dv = (case[k] for k in ("T", "H", "dqk", "dv"))
    length = _lengths(case)
    slots, at, rows = sum(length), 0, 0
    for c, n in zip(ctx, new):  # each cache row once, however many queries select it
        rows += min(c + n, sum(length[at:at + n]))
        at += n
    row = heads * (dqk if dqk != 256 else dqk + dv)
    return {"bytes": 2 * T * H * (dqk + dv) + 4 * T * (H + 1) + 4 * slots + rows * (row // 2 + row // 32),
            "flops": 2 * H * (dqk + dv) * slots}


# ---------------------------------------------------------------- 64 bits
def _nearest(x, table):
    """Value of `table` (ascending magnitudes, one per code) nearest to |x|, ties to the even code, with x's sign."""
    a = x.abs()
    hi = torch.searchsorted(table, a).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.where(torch.signbit(x), -table[c], table[c])


def _scaled_to(x, most):
    """2^e, e the smallest integer from -126 on with max |x| <= most * 2^e over the last dimension."""
    e = torch.ceil(torch.log2(x.abs().amax(-1) / most) - 1e-9)  # 1e-9: an exact power stays whole however log2 rounds
    return torch.exp2(e.clamp(min=-126))


def _decoded(codes, scale):
    tab = torch.tensor([-x if c & 8 else x for c, x in enumerate(E2M1 + E2M1)], dtype=torch.float64, device="cuda")
    n = codes.shape[-1]
    v = torch.empty(*codes.shape[:-1], 2 * n, dtype=torch.float64, device="cuda")
    v[..., 0::2] = tab[(codes % 16).long()]
    v[..., 1::2] = tab[(codes // 16).long()]
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        h = s["x"].double() + (0 if s["r"] is None else s["r"].double())
        norm = torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        y = h / norm[:, None] * s["w"].double()
        out = {"rstd": 1 / norm}
        if s["r"] is not None:
            out["sum"] = h
        if s["fmt"] == "bf16":
            return {**out, "y": y}
        y = y.view(y.shape[0], -1, 128 if s["fmt"] == "e4m3" else 32)
        scale = _scaled_to(y, 448.0)
        e4m3 = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
        codes = _nearest(y / scale[..., None], torch.tensor(e4m3, dtype=torch.float64, device="cuda"))
        return {**out, "y": codes.flatten(1), "scale": scale}
    if op == "norm_back":
        x, dy, w, r = (s[k].double() for k in ("x", "dy", "w", "rstd"))
        r = r[:, None]
        dot = (dy * w * x).sum(1, keepdim=True)
        dx = dy * w * r - x * r ** 3 * dot / x.shape[1]
        if s["d_sum"] is not None:
            dx = dx + s["d_sum"].double()
        return {"dx": dx, "dw": (dy * x * r).sum(0)}
    if op == "rotary":
        new, ctx = _sequences(case)
        p = torch.cat([torch.arange(c, c + n, dtype=torch.float64, device="cuda") for c, n in zip(ctx, new)])
        turn = torch.polar(torch.full((len(p), case["R"] // 2), s["mul"], dtype=torch.float64, device="cuda"),
                           (-1.0 if s["back"] else 1.0) * torch.outer(p, s["f"]))[:, None]
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            x = x.unflatten(2, (-1, 2)) if s["pairs"] else x.unflatten(2, (2, -1)).transpose(2, 3)
            z = torch.view_as_real(torch.view_as_complex(x.contiguous()) * turn)
            out[name] = z.flatten(2) if s["pairs"] else z.transpose(2, 3).flatten(2)
        return out
    if op == "cache":
        x = s["src"].double().unflatten(2, (-1, 32))
        scale = _scaled_to(x, 6.0)[..., None]
        out = (_nearest(x / scale, torch.tensor(E2M1, dtype=torch.float64, device="cuda")) * scale).flatten(2)
        out[case["tokens"]:] = 0
        return {"out": out}
    T, H, dqk = s["q"].shape
    heads, block = s["cache"].shape[2], s["block"]
    group = H // heads
    out = torch.empty(T, H, case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.empty(T, H, dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for b in range(len(cu) - 1):
        for t0 in range(cu[b], cu[b + 1], 16):
            t1 = min(t0 + 16, cu[b + 1])
            n = max(1, int(s["len"][t0:t1].max()))
            ok = torch.arange(n, device="cuda")[None, :] < s["len"][t0:t1, None]
            row = torch.where(ok, s["idx"][t0:t1, :n].long(), 0)
            if s["table"] is not None:
                row = s["table"][b].long()[row // block] * block + row % block
            for h in range(heads):
                k = _decoded(s["cache"].flatten(0, 1)[row, h], s["scale"].flatten(0, 1)[row, h])
                v = k[..., :512] if s["v"] is None else _decoded(s["v"].flatten(0, 1)[row, h], s["v_scale"].flatten(0, 1)[row, h])
                hs = slice(h * group, (h + 1) * group)
                x = torch.einsum("thc,tjc->thj", s["q"][t0:t1, hs].double(), k) / math.sqrt(dqk)
                x = torch.where(ok[:, None, :], x, -math.inf)
                if s["sink"] is not None:
                    x = torch.cat([x, s["sink"].double()[hs][None, :, None].expand(t1 - t0, -1, 1)], 2)
                l = torch.logsumexp(x, 2)
                lse[t0:t1, hs] = l
                e = torch.exp(x[..., :n] - torch.where(l == -math.inf, 0.0, l)[..., None])
                out[t0:t1, hs] = torch.einsum("thj,tjc->thc", e, v)
    return {"out": out, "lse": lse}
