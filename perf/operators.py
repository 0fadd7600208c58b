"""What is measured of the operators around the sparse attention of a decode step: FP4-weight
products, the per-head norm with the position rotation, and attention over every visible entry of
the FP4 cache.  Each case has a plain form (elementary torch operations in 32 bits, angles in 64)
and, with ``own`` true, the call of the library that a user makes.  ``exact`` gives the same
results from the definitions in 64 bits.

FP4: E2M1 codes, two per byte (element 2i in the low nibble), one E4M3 scale per 16 values.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
WINDOW, D_LAT = 128, 512


def listed():
    return [
        # ---- FP4-weight products y = alpha W x
        # one token's indexer queries (8 heads x 128) from a 1,536-wide low-rank query
        {"name": "linear-indexer-q-1", "op": "linear", "tok": 1, "groups": 1, "n_in": 1536, "n_out": 1024,
         "x": "bf16", "y": "f32", "pad": 0},
        # one token's 64 heads x 512 latent queries from the same low-rank query
        {"name": "linear-q-up-1", "op": "linear", "tok": 1, "groups": 1, "n_in": 1536, "n_out": 32768,
         "x": "bf16", "y": "bf16", "pad": 0},
        # the decode batch of 64 sequences, the same projection
        {"name": "linear-q-up-64", "op": "linear", "tok": 64, "groups": 1, "n_in": 1536, "n_out": 32768,
         "x": "bf16", "y": "bf16", "pad": 0},
        # grouped output projection of the fp32 attention output: 16 groups of 4 heads, 16 tokens
        {"name": "linear-out-groups-16", "op": "linear", "tok": 16, "groups": 16, "n_in": 2048, "n_out": 1024,
         "x": "f32", "y": "bf16", "pad": 0},
        # a small chunk of a prompt through a square projection; the largest product
        {"name": "linear-chunk-256", "op": "linear", "tok": 256, "groups": 1, "n_in": 4096, "n_out": 8192,
         "x": "f16", "y": "f16", "pad": 0},
        # ---- per-head norm and rotation
        # one decode token: 64 query heads and the shared latent row
        {"name": "norm-rope-1", "op": "rope", "tok": 1, "hq": 64, "hk": 1, "d": 512, "rot": 64, "x": "bf16",
         "y": "bf16", "norm": True, "halves": False, "inverse": False, "pad": 0, "far": 131072},
        # the attention's fp32 output of 64 tokens turned back by its own position, no norm
        {"name": "rope-back-64", "op": "rope", "tok": 64, "hq": 64, "hk": 0, "d": 512, "rot": 64, "x": "f32",
         "y": "bf16", "norm": False, "halves": False, "inverse": True, "pad": 0, "far": 1048576},
        # odd sizes: 131 tokens, 10 query and 2 key heads of 80, whole head rotated in halves, strided rows
        {"name": "norm-rope-odd", "op": "rope", "tok": 131, "hq": 10, "hk": 2, "d": 80, "rot": 80, "x": "f16",
         "y": "f16", "norm": True, "halves": True, "inverse": False, "pad": 24, "far": 1048576},
        # a prefill chunk of 4,096 tokens, the largest
        {"name": "norm-rope-4096", "op": "rope", "tok": 4096, "hq": 64, "hk": 1, "d": 512, "rot": 64, "x": "bf16",
         "y": "bf16", "norm": True, "halves": False, "inverse": False, "pad": 0, "far": 131072},
        # ---- attention over every visible entry
        # a short context, 16 heads
        {"name": "dense-2k-1", "op": "dense", "batch": 1, "n_q": 1, "heads": 16, "ctx": 2048, "ratio": 2,
         "ragged": False},
        # a ragged batch with three draft positions per sequence, some without a visible entry
        {"name": "dense-ragged-7x3", "op": "dense", "batch": 7, "n_q": 3, "heads": 24, "ctx": 9001, "ratio": 1,
         "ragged": True},
        # 64 sequences of 32K positions, 64 heads: the largest
        {"name": "dense-32k-64", "op": "dense", "batch": 64, "n_q": 1, "heads": 64, "ctx": 32768, "ratio": 2,
         "ragged": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "rope", "dense"])
    if op == "linear":
        while True:
            c = {"op": op, "tok": _log(rng, 1, 256), "groups": rng.choice([1, 1, 1, 2, 5, 8, 16]),
                 "n_in": 16 * _log(rng, 4, 512), "n_out": _log(rng, 40, 32768),
                 "x": rng.choice(["bf16", "bf16", "f16", "f32"]), "y": rng.choice(["bf16", "f16", "f32"]),
                 "pad": rng.choice([0, 0, 8, 5])}
            weights = c["groups"] * c["n_in"] * c["n_out"]
            if weights <= 1536 * 32768 and weights * c["tok"] <= 256 * 4096 * 8192:
                return c
    if op == "rope":
        while True:
            d = rng.choice([64, 80, 96, 128, 192, 256, 512, 512])
            c = {"op": op, "tok": _log(rng, 1, 8192), "hq": rng.choice([1, 3, 8, 16, 24, 32, 64, 128]),
                 "hk": rng.choice([0, 1, 1, 2, 8]), "d": d, "rot": rng.choice([d, d // 2, 64, 32]),
                 "x": rng.choice(["bf16", "f16", "f32"]), "y": rng.choice(["bf16", "f16", "f32"]),
                 "norm": rng.random() < 0.8, "halves": rng.random() < 0.5, "inverse": rng.random() < 0.25,
                 "pad": rng.choice([0, 0, 8, 24, 3]), "far": rng.choice([4096, 131072, 1048576])}
            if c["tok"] * (c["hq"] + c["hk"]) * d * (_SIZE[c["x"]] + _SIZE[c["y"]]) <= 4096 * 65 * 512 * 4:
                return c
    while True:
        c = {"op": op, "batch": _log(rng, 1, 64), "n_q": rng.choice([1, 1, 1, 2, 4, 5]),
             "heads": rng.choice([1, 8, 16, 24, 32, 64, 64]), "ctx": _log(rng, 1, 1048576),
             "ratio": rng.choice([1, 2, 2]), "ragged": rng.random() < 0.5}
        if c["batch"] * c["n_q"] * (c["ctx"] // c["ratio"] + WINDOW) <= 64 * 16384:
            return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _fp4(rows, d, g, spread):
    """codes and scales of `rows` rows of d values: groups of N(0, spread^2) values, each group's own
    size spread further as trained weights and latents have it"""
    codes = torch.empty((rows, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, d // 16), dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 25) // d)
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        x = torch.randn((n, d // 16, 16), device="cuda", generator=g)
        x *= spread * torch.exp2(torch.randn((n, d // 16, 1), device="cuda", generator=g) * 0.5)
        s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        f = s.float().clamp_min(2.0 ** -9)
        m = torch.bucketize(x.abs() / f[..., None], edges, out_int32=True)
        m = (m + 8 * ((x < 0) & (m > 0))).to(torch.uint8).reshape(n, d // 2, 2)
        codes[r0:r0 + n] = m[..., 0] | (m[..., 1] << 4)
        scales[r0:r0 + n] = s.view(torch.uint8)
    return codes, scales


def _padded(shape, pad, dtype, g):
    """N(0, 1) values whose rows lie `pad` elements further apart than they are long"""
    t = torch.randn(shape[:-1] + (shape[-1] + pad,), device="cuda", generator=g).to(dtype)
    return t[..., :shape[-1]]


def prepare(case, seed):
    g = _gen(seed)
    c = case
    if c["op"] == "linear":
        G, K, M, T = c["groups"], c["n_in"], c["n_out"], c["tok"]
        # weights of size n_in^-1/2, held in FP4 as 64 times that (alpha takes it back)
        codes, scales = _fp4(G * M, K, g, 64.0 / math.sqrt(K))
        x = _padded((T, G, K), c["pad"], _T[c["x"]], g)
        y = torch.empty((T, G, M), dtype=_T[c["y"]], device="cuda")
        if G == 1:
            return {"case": c, "x": x[:, 0], "codes": codes, "scales": scales, "alpha": 1.0 / 64.0, "y": y[:, 0]}
        return {"case": c, "x": x, "codes": codes.view(G, M, K // 2), "scales": scales.view(G, M, K // 16),
                "alpha": 1.0 / 64.0, "y": y}
    if c["op"] == "rope":
        T, D, R = c["tok"], c["d"], c["rot"]
        s = {"case": c, "q": _padded((T, c["hq"], D), c["pad"], _T[c["x"]], g),
             "pos": torch.randint(0, c["far"], (T,), device="cuda", generator=g),
             "inv_freq": (10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)).float(),
             "qw": None, "k": None, "kw": None, "ko": None,
             "qo": torch.empty((T, c["hq"], D), dtype=_T[c["y"]], device="cuda")}
        if c["norm"]:
            s["qw"] = 1.0 + 0.2 * torch.randn((D,), device="cuda", generator=g)
        if c["hk"]:
            s["k"] = _padded((T, c["hk"], D), c["pad"], _T[c["x"]], g)
            s["kw"] = 1.0 + 0.2 * torch.randn((D,), device="cuda", generator=g) if c["norm"] else None
            s["ko"] = torch.empty((T, c["hk"], D), dtype=_T[c["y"]], device="cuda")
        return s
    B, Q, H, r = c["batch"], c["n_q"], c["heads"], c["ratio"]
    ctx, cap = c["ctx"], -(-c["ctx"] // r) + 3
    last = torch.full((B,), ctx - 1, dtype=torch.int64, device="cuda")
    if c["ragged"]:
        last = torch.randint(0, ctx, (B,), device="cuda", generator=g)
        last[0] = min(ctx - 1, 100)          # a sequence that sees its window alone
    pos = (last[:, None] - torch.arange(Q - 1, -1, -1, device="cuda")[None]).clamp_min(0)
    codes, scales = _fp4(B * cap, D_LAT, g, 1.0)
    codes, scales = codes.view(B, cap, -1), scales.view(B, cap, -1)
    # the rows from the first unseen entry on hold whatever was there before, NaN scales among it
    n_vis = ((pos.amax(1) - (WINDOW - 1)).clamp_min(0) // r).clamp_max(cap)
    stale = torch.arange(cap, device="cuda")[None] >= n_vis[:, None]
    scales[stale] = 0x7F
    # each sequence's window rows, the oldest first; rows of positions to come hold NaN
    n_win = WINDOW - 1 + Q
    swa_pos0 = (pos.amax(1) - (n_win - 1)).clamp_min(0)
    swa = torch.randn((B, n_win, D_LAT), device="cuda", generator=g).to(torch.bfloat16)
    swa[swa_pos0[:, None] + torch.arange(n_win, device="cuda") > pos.amax(1)[:, None]] = math.nan
    q = torch.randn((B, Q, H, D_LAT), device="cuda", generator=g).to(torch.bfloat16)
    s = {"case": c, "codes": codes, "scales": scales, "pos": pos, "swa": swa, "swa_pos0": swa_pos0, "q": q,
         "scale": D_LAT ** -0.5, "ws": None,
         "out": torch.empty((B, Q, H, D_LAT), dtype=torch.bfloat16, device="cuda"),
         "lse": torch.empty((B, Q, H), dtype=torch.float32, device="cuda")}
    return s


# ---------------------------------------------------------------- the plain forms

def _values(codes, scales):
    """the fp32 values of FP4 rows"""
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                     device=codes.device)
    pairs = torch.stack((t.repeat(16), t.repeat_interleave(16)), -1)          # byte -> its two values
    v = pairs[codes.int()].view(scales.shape + (16,)) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.view(codes.shape[:-1] + (2 * codes.shape[-1],))


def _plain_linear(s):
    w, x = _values(s["codes"], s["scales"]), s["x"].float()
    y = x @ w.T if w.dim() == 2 else torch.matmul(x.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1)
    return (y * s["alpha"]).to(s["y"].dtype)


def _plain_rows(c, x, w, cos, sin):
    v = x.float()
    if c["norm"]:
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w
    R = c["rot"]
    keep, turn = v[..., :c["d"] - R], v[..., c["d"] - R:]
    if c["halves"]:
        a, b = turn[..., :R // 2], turn[..., R // 2:]
        turn = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((keep, turn), -1).to(_T[c["y"]])


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin
    q = _plain_rows(c, s["q"], s["qw"], cos, sin)
    return (q, _plain_rows(c, s["k"], s["kw"], cos, sin)) if c["hk"] else (q,)


def _plain_dense(s):
    c, q, pos = s["case"], s["q"].float(), s["pos"]
    B, Q, H, n = q.shape[0], q.shape[1], q.shape[2], s["codes"].shape[1]
    n_vis = (pos - (WINDOW - 1)).clamp_min(0) // c["ratio"]
    seen = torch.arange(n, device=q.device) < n_vis[..., None]                        # [B, Q, n]
    at = s["swa_pos0"][:, None, None] + torch.arange(s["swa"].shape[1], device=q.device)
    near = (at <= pos[..., None]) & (at > pos[..., None] - WINDOW)                     # [B, Q, n_win]
    win = torch.where(near.any(1)[..., None], s["swa"].float(), 0.0)
    lat = torch.where(seen.any(1)[..., None], _values(s["codes"], s["scales"]), 0.0)   # [B, n, 512]
    rows = q.reshape(B, Q * H, D_LAT)
    a = (rows @ lat.transpose(1, 2)).view(B, Q, H, n) * s["scale"]
    b = (rows @ win.transpose(1, 2)).view(B, Q, H, -1) * s["scale"]
    a = a.masked_fill(~seen[:, :, None], -math.inf)
    b = b.masked_fill(~near[:, :, None], -math.inf)
    top = torch.maximum(a.amax(-1), b.amax(-1))
    base = top.masked_fill(top == -math.inf, 0.0)[..., None]
    a, b = torch.exp(a - base), torch.exp(b - base)
    total = a.sum(-1) + b.sum(-1)
    o = a.view(B, Q * H, n) @ lat + b.view(B, Q * H, -1) @ win
    o = o.view(B, Q, H, D_LAT) / total.masked_fill(total == 0, 1.0)[..., None]
    return o.to(torch.bfloat16), base[..., 0] + torch.log(total)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "rope": _plain_rope, "dense": _plain_dense}[op](s)
    import compressed_sparse_attention_decode_gb300 as csa
    if op == "linear":
        return csa.csa2_linear_fp4(s["x"], s["codes"], s["scales"], s["alpha"], out=s["y"])
    if op == "rope":
        c = s["case"]
        got = csa.csa2_norm_rope(s["q"], s["pos"], s["inv_freq"], q_weight=s["qw"], k=s["k"], k_weight=s["kw"],
                                 eps=1e-6, norm=c["norm"], halves=c["halves"], inverse=c["inverse"], q_out=s["qo"],
                                 k_out=s["ko"])
        return got if c["hk"] else got[:1]
    cache = csa.Cache.of(s["codes"], s["scales"], ratio=s["case"]["ratio"])
    if s["ws"] is None:            # a workspace that the program keeps with its buffers
        B, Q, H = s["q"].shape[:3]
        s["ws"] = csa.workspace(csa.OP_DENSE_ATTN, B, Q, H, 0, cache.capacity)
    return csa.csa2_dense_attn(cache, s["q"], s["pos"], s["swa"], s["swa_pos0"], s["scale"], out=s["out"],
                               lse=s["lse"], ws=s["ws"])


# ---------------------------------------------------------------- what a pass cannot do without

def _visible(c):
    """entries seen by each query, summed over the batch, and by the furthest query of each sequence;
    for ragged positions the mean of their uniform draw"""
    each = max(0, c["ctx"] - WINDOW) / c["ratio"]
    if c["ragged"]:
        each *= 0.5 * (c["batch"] - 1) / c["batch"]
    return each


def work(case):
    c = case
    if c["op"] == "linear":
        T, G, K, M = c["tok"], c["groups"], c["n_in"], c["n_out"]
        return {"bytes": G * M * (K // 2 + K // 16) + T * G * (K * _SIZE[c["x"]] + M * _SIZE[c["y"]]),
                "flops": 2.0 * T * G * K * M}
    if c["op"] == "rope":
        n = c["tok"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": n * (_SIZE[c["x"]] + _SIZE[c["y"]]) + c["tok"] * 8 + 2 * c["rot"] + (8 * c["d"] if c["norm"] else 0),
                "flops": n * (4.0 if c["norm"] else 0.0) + 3.0 * c["tok"] * (c["hq"] + c["hk"]) * c["rot"]}
    B, Q, H = c["batch"], c["n_q"], c["heads"]
    n, win = _visible(c), min(WINDOW, c["ctx"])
    return {"bytes": B * (n * 288 + (win + Q - 1) * 1024) + B * Q * H * (D_LAT * 4 + 4),
            "flops": 4.0 * B * Q * H * D_LAT * (n + win)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _decode(codes, scales):
    """FP4 rows in 64 bits from the formats' definitions: sign, exponent and mantissa bits"""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (n >> 1) & 3, n & 1
    v = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2((e - 1).double()))
    v = torch.where(n >= 8, -v, v)
    s = scales.long()
    e, m = (s >> 3) & 15, (s & 7).double()
    f = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).double()))
    f = torch.where(s >= 128, -f, f)
    f = torch.where((s & 127) == 127, math.nan, f)
    return (v.unflatten(-1, (-1, 16)) * f[..., None]).flatten(-2)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        G, T, M = c["groups"], c["tok"], c["n_out"]
        x = s["x"].double().reshape(T, G, -1)
        codes, scales = s["codes"].reshape(G, M, -1), s["scales"].reshape(G, M, -1)
        y = torch.stack([torch.einsum("tk,mk->tm", x[:, i], _decode(codes[i], scales[i])) for i in range(G)], 1)
        return (s["alpha"] * y).reshape(s["y"].shape)
    if c["op"] == "rope":
        D, R = c["d"], c["rot"]
        # each pair of the rotated tail as one complex number, turned by exp(i p f)
        turn = torch.polar(torch.ones((c["tok"], R // 2), dtype=torch.float64, device="cuda"),
                           (-1.0 if c["inverse"] else 1.0) * s["pos"].double()[:, None] * s["inv_freq"].double())
        outs = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            if x is None:
                continue
            v = x.double()
            if c["norm"]:
                v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            tail = v[..., D - R:]
            pairs = tail.unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["halves"] else tail.unflatten(-1, (R // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
            v[..., D - R:] = (z.transpose(-1, -2) if c["halves"] else z).flatten(-2)
            outs.append(v)
        return tuple(outs)
    B, Q, H = s["q"].shape[:3]
    out = torch.zeros((B, Q, H, D_LAT), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        for i in range(Q):
            p = int(s["pos"][b, i])
            n = max(0, p - (WINDOW - 1)) // c["ratio"]
            lo, at = max(0, p - (WINDOW - 1)), int(s["swa_pos0"][b])
            rows = torch.cat((_decode(s["codes"][b, :n], s["scales"][b, :n]),
                              s["swa"][b, max(lo, at) - at:p + 1 - at].double()))
            a = s["scale"] * torch.einsum("hd,nd->hn", s["q"][b, i].double(), rows)
            lse[b, i] = torch.logsumexp(a, -1)
            out[b, i] = torch.softmax(a, -1) @ rows
    return out, lse
