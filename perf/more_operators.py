"""What is measured of the operators of a speculative step over the FP4 cache: attention of a tree of
drafted tokens (over every visible entry, or over an index list per node), quantising accepted rows
into the cache of a ragged batch, and reading entries back.  Each case has a plain form (elementary
torch operations in 32 bits, exact sums in 64) and, with ``own`` true, the calls of the library that a
user makes.  ``exact`` gives the same results from the definitions in 64 bits.

FP4: E2M1 codes, two per byte (element 2i in the low nibble), one E4M3 scale per 16 values:
scale = E4M3(fp32(largest / 6)), code = the nearest of value / scale, ties to the even code, zero as +0.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
WINDOW, D_LAT = 128, 512


def listed():
    return [
        # ---- a drafted tree over every visible entry
        # one sequence with a short context, eight nodes, 16 heads: the smallest call
        {"name": "tree-2k-1x8", "op": "tree", "batch": 1, "nodes": 8, "heads": 16, "ctx": 2048, "ratio": 2, "k": 0,
         "ragged": False, "out": "bf16"},
        # a ragged batch: lengths from nothing to 9,001 positions of the per-position cache, trees cut short
        {"name": "tree-ragged-7x21", "op": "tree", "batch": 7, "nodes": 21, "heads": 24, "ctx": 9001, "ratio": 1, "k": 0,
         "ragged": True, "out": "bf16"},
        # 16 sequences of 32K positions, 16 nodes each, 64 heads
        {"name": "tree-32k-16x16", "op": "tree", "batch": 16, "nodes": 16, "heads": 64, "ctx": 32768, "ratio": 2, "k": 0,
         "ragged": False, "out": "bf16"},
        # one long sequence and a wide tree: the largest
        {"name": "tree-256k-1x64", "op": "tree", "batch": 1, "nodes": 64, "heads": 64, "ctx": 262144, "ratio": 2, "k": 0,
         "ragged": False, "out": "bf16"},
        # ---- the same over an index list per node, as a layer with an indexer has it
        # two short sequences, lists shorter than their 128 slots for some
        {"name": "tree-list-4k-2x5", "op": "tree", "batch": 2, "nodes": 5, "heads": 32, "ctx": 4096, "ratio": 2, "k": 128,
         "ragged": True, "out": "f32"},
        # the decode layer's own sizes: 512 of 16K entries, 64 heads, 16 sequences of 16 nodes
        {"name": "tree-list-32k-16x16", "op": "tree", "batch": 16, "nodes": 16, "heads": 64, "ctx": 32768, "ratio": 2,
         "k": 512, "ragged": False, "out": "f32"},
        # ---- accepted rows quantised into the cache, and those entries read back
        # one token of each of 64 sequences, every second of which completes a merged pair
        {"name": "append-step-64", "op": "append", "batch": 64, "rows": 1, "path": 1, "ctx": 32768, "ratio": 2, "d_idx": 128,
         "keys": True, "tree": False, "out": "bf16"},
        # the accepted paths of 64 trees of 16 nodes into the per-position cache, with their indexer keys
        {"name": "append-path-64x8", "op": "append", "batch": 64, "rows": 16, "path": 8, "ctx": 32768, "ratio": 1, "d_idx": 128,
         "keys": True, "tree": True, "out": "bf16"},
        # a prompt chunk of 4 sequences that begin anywhere
        {"name": "append-chunk-4x8192", "op": "append", "batch": 4, "rows": 8192, "path": 8192, "ctx": 40000, "ratio": 2,
         "d_idx": 128, "keys": True, "tree": False, "out": "bf16"},
        # ---- entries read back
        # the indexer keys of one short sequence, in fp32
        {"name": "read-keys-1", "op": "read", "batch": 1, "capacity": 2048, "d_idx": 128, "keys": True, "n": 2048,
         "listed": False, "out": "f32"},
        # the rows that the index lists of 16 x 16 queries name, some slots empty
        {"name": "read-list-16x8192", "op": "read", "batch": 16, "capacity": 16384, "d_idx": 128, "keys": False, "n": 8192,
         "listed": True, "out": "bf16"},
        # the latents of 8 sequences of 64K entries
        {"name": "read-all-8x64k", "op": "read", "batch": 8, "capacity": 65536, "d_idx": 128, "keys": False, "n": 65536,
         "listed": False, "out": "f16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "list", "append", "read"])
    if op in ("tree", "list"):
        while True:
            c = {"op": "tree", "batch": _log(rng, 1, 64), "nodes": _log(rng, 1, 128),
                 "heads": rng.choice([1, 8, 16, 24, 32, 48, 64, 64, 128]), "ctx": _log(rng, 1, 1048576),
                 "ratio": rng.choice([1, 2, 2]), "k": _log(rng, 1, 2048) if op == "list" else 0,
                 "ragged": rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "f16", "f32"])}
            n = c["ctx"] // c["ratio"]
            per_node = c["k"] or n
            if c["batch"] * c["nodes"] * c["heads"] * (per_node + WINDOW + c["nodes"]) <= 64 * 64 * 131072 and \
                    c["batch"] * n <= 64 * 16384 and c["batch"] * c["nodes"] * c["k"] <= 1 << 18:
                return c
    if op == "append":
        while True:
            path, tree = _log(rng, 1, 8192), rng.random() < 0.4
            if tree:
                path = 1 + path % 12
            c = {"op": op, "batch": _log(rng, 1, 64), "rows": path + rng.randrange(24) if tree else path, "path": path,
                 "ctx": _log(rng, 1, 65536), "ratio": rng.choice([1, 2, 2]), "d_idx": rng.choice([64, 128, 128]),
                 "keys": rng.random() < 0.7, "tree": tree, "out": rng.choice(["bf16", "f16", "f32"])}
            if c["batch"] * c["path"] * (2 if c["ratio"] == 1 else 1) <= 4 * 8192 and c["batch"] * c["ctx"] <= 64 * 32768:
                return c
    while True:
        cap = _log(rng, 1, 262144)
        c = {"op": op, "batch": _log(rng, 1, 64), "capacity": cap, "d_idx": rng.choice([64, 128]),
             "keys": rng.random() < 0.3, "n": min(cap, _log(rng, 1, 262144)), "listed": rng.random() < 0.5,
             "out": rng.choice(["bf16", "f16", "f32"])}
        if c["listed"]:
            c["n"] = _log(rng, 1, 16384)
        if c["batch"] * max(cap, c["n"] * (2 if c["out"] == "f32" else 1)) <= 8 * 65536:
            return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def _fp4(rows, d, g):
    """codes and scales of `rows` rows of d values: groups of normal values, each group's own size spread
    as latents have it"""
    codes = torch.empty((rows, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, d // 16), dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 25) // d)
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        x = torch.randn((n, d // 16, 16), device="cuda", generator=g)
        x *= torch.exp2(torch.randn((n, d // 16, 1), device="cuda", generator=g) * 0.5)
        s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        m = torch.bucketize(x.abs() / s.float().clamp_min(2.0 ** -9)[..., None], edges, out_int32=True)
        m = (m + 8 * ((x < 0) & (m > 0))).to(torch.uint8).reshape(n, d // 2, 2)
        codes[r0:r0 + n] = m[..., 0] | (m[..., 1] << 4)
        scales[r0:r0 + n] = s.view(torch.uint8)
    return codes, scales


def _prepare_tree(c, g):
    B, N, H, r, ctx = c["batch"], c["nodes"], c["heads"], c["ratio"], c["ctx"]
    cap = -(-ctx // r) + 3
    # committed positions of each sequence; the first drafted token comes at this position
    base = torch.full((B,), ctx, dtype=torch.int64, device="cuda")
    if c["ragged"]:
        base = torch.randint(0, ctx + 1, (B,), device="cuda", generator=g)
        base[0] = min(ctx, 100)                  # a sequence that sees its window alone
    # a parent among the nodes before, or -1 (a child of the last committed token)
    u = torch.rand((B, N), device="cuda", generator=g)
    parent = torch.minimum((u * (torch.arange(N, device="cuda") + 1)).int(), torch.arange(N, device="cuda").int()) - 1
    there = torch.full((B,), N, dtype=torch.int64, device="cuda")
    if c["ragged"]:
        there = torch.randint(1, N + 1, (B,), device="cuda", generator=g)
    parent[torch.arange(N, device="cuda") >= there[:, None]] = -2                     # trees cut short
    depth = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    for i in range(1, N):
        p = parent[:, i:i + 1].long()
        depth[:, i:i + 1] = torch.where(p >= 0, depth.gather(1, p.clamp_min(0)) + 1, 0)
    pos = base[:, None] + depth
    codes, scales = _fp4(B * cap, D_LAT, g)
    codes, scales = codes.view(B, cap, -1), scales.view(B, cap, -1)
    # the entries that no node sees hold whatever was there before, NaN scales among it
    n_vis = ((pos.amax(1) - (WINDOW - 1)).clamp_min(0) // r).clamp_max(cap)
    scales[torch.arange(cap, device="cuda")[None] >= n_vis[:, None]] = 0x7F
    idx = None
    if c["k"]:
        # each node's list: k of the 2k entries that its sequence's candidates are, ascending, the end empty
        k, every = c["k"], ((base - (WINDOW - 1)).clamp_min(0) // r).clamp_max(cap)
        width = min(2 * k, cap)
        pool = torch.rand((B, cap), device="cuda", generator=g).argsort(1)[:, :width].int()
        pick = torch.rand((B, N, width), device="cuda", generator=g).argsort(2)[..., :k]
        idx = pool[:, None].expand(B, N, width).gather(2, pick)
        if width < k:
            idx = torch.cat((idx, idx.new_full((B, N, k - width), cap)), 2)
        idx = torch.where(idx < every[:, None, None], idx, cap).sort(-1).values
        idx = torch.where(idx < cap, idx, -1).int().contiguous()
    # the committed rows of each window, the oldest first; rows past them hold NaN
    swa_pos0 = (base - (WINDOW - 1)).clamp_min(0)
    swa = _randn((B, WINDOW, D_LAT), g, torch.bfloat16)
    swa[swa_pos0[:, None] + torch.arange(WINDOW, device="cuda") >= base[:, None]] = math.nan
    draft = _randn((B, N, D_LAT), g, torch.bfloat16)
    draft[parent < -1] = math.nan
    return {"case": c, "codes": codes, "scales": scales, "pos": pos, "parent": parent.contiguous(), "draft": draft, "idx": idx,
            "swa": swa, "swa_pos0": swa_pos0, "q": _randn((B, N, H, D_LAT), g, torch.bfloat16), "scale": D_LAT ** -0.5,
            "ws": None, "out": torch.empty((B, N, H, D_LAT), dtype=_T[c["out"]], device="cuda"),
            "lse": torch.empty((B, N, H), dtype=torch.float32, device="cuda")}


def _prepare_append(c, g):
    B, R, P, r, d = c["batch"], c["rows"], c["path"], c["ratio"], c["d_idx"]
    cap = (c["ctx"] + P) // r + 1
    pos0 = torch.randint(0, c["ctx"] + 1, (B,), device="cuda", generator=g)
    path, length = None, torch.full((B,), P, dtype=torch.int64, device="cuda")
    if c["tree"]:
        # an accepted path: ascending node numbers, at least one, the end empty
        length = torch.randint(1, P + 1, (B,), device="cuda", generator=g)
        path = torch.rand((B, R), device="cuda", generator=g).argsort(1)[:, :P].sort(1).values.int()
        path[torch.arange(P, device="cuda") >= length[:, None]] = -1
        path = path.contiguous()
    # the entries that the call completes
    first = pos0 // r
    n = ((pos0 + length) // r - first)
    at = torch.arange(P // r + 1, device="cuda")
    written = torch.where(at < n[:, None], first[:, None] + at, -1).int().contiguous()
    s = {"case": c, "rows": _randn((B, R, D_LAT), g, torch.bfloat16), "pos0": pos0, "path": path, "written": written,
         "codes": torch.zeros((B, cap, D_LAT // 2), dtype=torch.uint8, device="cuda"),
         "scales": torch.zeros((B, cap, D_LAT // 16), dtype=torch.uint8, device="cuda"), "w0": None, "w1": None,
         "prev": None, "prev_out": None, "wik": None, "kcodes": None, "kscales": None, "kout": None,
         "out": torch.empty(written.shape + (D_LAT,), dtype=_T[c["out"]], device="cuda")}
    if r == 2:
        s["w0"] = 0.3 + 0.4 * torch.rand((D_LAT,), device="cuda", generator=g)
        s["w1"] = 0.3 + 0.4 * torch.rand((D_LAT,), device="cuda", generator=g)
        s["prev"] = _randn((B, D_LAT), g, torch.bfloat16)
        s["prev_out"] = torch.empty_like(s["prev"])
    if c["keys"]:
        s["wik"] = _fp4(d, D_LAT, g)
        s["kcodes"] = torch.zeros((B, cap, d // 2), dtype=torch.uint8, device="cuda")
        s["kscales"] = torch.zeros((B, cap, d // 16), dtype=torch.uint8, device="cuda")
        s["kout"] = torch.empty(written.shape + (d,), dtype=_T[c["out"]], device="cuda")
    return s


def _prepare_read(c, g):
    B, cap = c["batch"], c["capacity"]
    d = c["d_idx"] if c["keys"] else D_LAT
    codes, scales = _fp4(B * cap, d, g)
    idx = None
    if c["listed"]:
        idx = torch.randint(0, cap, (B, c["n"]), device="cuda", generator=g, dtype=torch.int32)
        idx[torch.rand((B, c["n"]), device="cuda", generator=g) < 0.05] = -1          # empty slots
    latents = tuple(torch.zeros((B, cap, n), dtype=torch.uint8, device="cuda") for n in (256, 32)) if c["keys"] else None
    return {"case": c, "codes": codes.view(B, cap, -1), "scales": scales.view(B, cap, -1), "latents": latents, "idx": idx,
            "out": torch.empty((B, c["n"], d), dtype=_T[c["out"]], device="cuda")}


def prepare(case, seed):
    return {"tree": _prepare_tree, "append": _prepare_append, "read": _prepare_read}[case["op"]](case, _gen(seed))


# ---------------------------------------------------------------- the plain forms

def _values(codes, scales):
    """the fp32 values of FP4 rows"""
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                     device=codes.device)
    pairs = torch.stack((t.repeat(16), t.repeat_interleave(16)), -1)          # byte -> its two values
    v = pairs[codes.int()].view(scales.shape + (16,)) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.view(codes.shape[:-1] + (2 * codes.shape[-1],))


def _chains(parent):
    """[B, N, N]: node i's ancestors and itself; none for a node whose chain does not reach a committed token"""
    B, N = parent.shape
    seen = torch.zeros((B, N, N), dtype=torch.bool, device=parent.device)
    eye = torch.eye(N, dtype=torch.bool, device=parent.device)
    for i in range(N):
        p = parent[:, i].long()
        up = seen.gather(1, p.clamp(0, N - 1)[:, None, None].expand(B, 1, N))[:, 0]
        ok = (p == -1) | ((p >= 0) & (p < i) & up.any(1))
        seen[:, i] = torch.where(ok[:, None], torch.where((p >= 0)[:, None], up, False) | eye[i], False)
    return seen


def _plain_tree(s):
    c, q, pos = s["case"], s["q"].float(), s["pos"]
    B, N, H = q.shape[:3]
    anc = _chains(s["parent"])
    there, length = anc.any(2), anc.sum(2)
    at = s["swa_pos0"][:, None, None] + torch.arange(s["swa"].shape[1], device=q.device)
    near = (at <= (pos - length)[..., None]) & (at > pos[..., None] - WINDOW) & there[..., None]      # [B, N, rows]
    rows = torch.cat((torch.where(near.any(1)[..., None], s["swa"].float(), 0.0),
                      torch.where(anc.any(1)[..., None], s["draft"].float(), 0.0)), 1)
    mask = torch.cat((near, anc), 2)
    b = (q.reshape(B, N * H, D_LAT) @ rows.transpose(1, 2)).view(B, N, H, -1) * s["scale"]
    b = b.masked_fill(~mask[:, :, None], -math.inf)
    if s["idx"] is None:
        n = s["codes"].shape[1]
        n_vis = (pos - (WINDOW - 1)).clamp_min(0) // c["ratio"]
        seen = (torch.arange(n, device=q.device) < n_vis[..., None]) & there[..., None]               # [B, N, n]
        lat = torch.where(seen.any(1)[..., None], _values(s["codes"], s["scales"]), 0.0)
        a = (q.reshape(B, N * H, D_LAT) @ lat.transpose(1, 2)).view(B, N, H, n)
        a = a.mul_(s["scale"]).masked_fill_(~seen[:, :, None], -math.inf)
    else:
        k = s["idx"].shape[2]
        seen = (s["idx"] >= 0) & there[..., None]
        j = s["idx"].long().clamp_min(0).view(B, N * k, 1)
        lat = _values(s["codes"].gather(1, j.expand(-1, -1, D_LAT // 2)), s["scales"].gather(1, j.expand(-1, -1, D_LAT // 16)))
        lat = torch.where(seen.view(B, N * k, 1), lat, 0.0).view(B, N, k, D_LAT)
        a = (q @ lat.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~seen[:, :, None], -math.inf)
    top = torch.maximum(a.amax(-1), b.amax(-1))
    base = top.masked_fill(top == -math.inf, 0.0)[..., None]
    a, b = a.sub_(base).exp_(), torch.exp(b - base)
    total = a.sum(-1) + b.sum(-1)
    o = (a.view(B, N * H, -1) @ lat).view(B, N, H, D_LAT) if s["idx"] is None else a @ lat
    o = o + (b.view(B, N * H, -1) @ rows).view(B, N, H, D_LAT)
    o = o / total.masked_fill(total == 0, 1.0)[..., None]
    return o.to(s["out"].dtype), base[..., 0] + torch.log(total)


def _quantise(x):
    """fp32 rows as codes and scales"""
    g = x.unflatten(-1, (-1, 16))
    scales = (g.abs().amax(-1) / 6.0).clamp_max(448.0).to(torch.float8_e4m3fn)
    f = scales.float()[..., None]
    a = g.abs()
    m = ((a > 0.25 * f).to(torch.uint8) + (a >= 0.75 * f) + (a > 1.25 * f) + (a >= 1.75 * f) + (a > 2.5 * f)
         + (a >= 3.5 * f) + (a > 5.0 * f)) * (f > 0)
    m = (m + 8 * ((g < 0) & (m > 0))).to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    return m[..., 0] | (m[..., 1] << 4), scales.view(torch.uint8)


def _put(plane, at, rows):
    """rows [B, n, d] to the entries at [B, n] of the plane; -1 goes to its last entry, which no call completes"""
    j = torch.where(at >= 0, at.long(), plane.shape[1] - 1)[..., None]
    plane.scatter_(1, j.expand(rows.shape), rows)


def _get(codes, scales, at, dtype):
    """the values of the entries at [B, n], zeros where at is -1"""
    j = at.long().clamp_min(0)[..., None]
    v = _values(codes.gather(1, j.expand(-1, -1, codes.shape[2])), scales.gather(1, j.expand(-1, -1, scales.shape[2])))
    return torch.where((at >= 0)[..., None], v, 0.0).to(dtype)


def _accepted(s):
    """the rows of the accepted path (its order; what lies past its end repeats a row) and its length"""
    B, P = s["case"]["batch"], s["case"]["path"]
    if s["path"] is None:
        return s["rows"], torch.full((B,), P, dtype=torch.int64, device="cuda")
    rows = s["rows"].gather(1, s["path"].long().clamp_min(0)[..., None].expand(B, P, D_LAT))
    return rows, (s["path"] >= 0).sum(1)


def _plain_append(s):
    c = s["case"]
    B, P, r = c["batch"], c["path"], c["ratio"]
    rows, length = _accepted(s)
    outs = []
    if r == 1:
        e = rows.float()
        at = s["written"][:, :P]
    else:
        # with the carried row in front, position pos0 - 1 + j is row j; an entry's first position is even
        both = torch.cat((s["prev"][:, None], rows), 1).float()
        j = 2 * s["written"].long() - (s["pos0"] - 1)[:, None]
        h0 = both.gather(1, j.clamp(0, P)[..., None].expand(-1, -1, D_LAT))
        h1 = both.gather(1, (j + 1).clamp(0, P)[..., None].expand(-1, -1, D_LAT))
        e = (s["w1"].double() * h1.double() + (s["w0"] * h0).double()).float()          # a product, then one fused step
        at = s["written"]
        outs.append(both.gather(1, length[:, None, None].expand(B, 1, D_LAT))[:, 0].to(torch.bfloat16))
    codes, scales = _quantise(e)
    _put(s["codes"], at, codes)
    _put(s["scales"], at, scales)
    if c["keys"]:
        # every product is a multiple of 2^-20 and the sums stay below 2^33: exact in 64 bits
        k = (_values(codes, scales).double() @ _values(*s["wik"]).double().T).float()
        codes, scales = _quantise(k)
        _put(s["kcodes"], at, codes)
        _put(s["kscales"], at, scales)
        outs.append(_get(s["kcodes"], s["kscales"], s["written"], s["kout"].dtype))
    return [_get(s["codes"], s["scales"], s["written"], s["out"].dtype)] + outs


def _plain_read(s):
    if s["idx"] is not None:
        return _get(s["codes"], s["scales"], s["idx"], s["out"].dtype)
    n = s["case"]["n"]
    return _values(s["codes"][:, :n], s["scales"][:, :n]).to(s["out"].dtype)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "append": _plain_append, "read": _plain_read}[op](s)
    import compressed_sparse_attention_decode_gb300 as csa
    c = s["case"]
    if op == "tree":
        cache = csa.Cache.of(s["codes"], s["scales"], ratio=c["ratio"])
        if s["ws"] is None:            # a workspace that the program keeps with its buffers
            s["ws"] = csa.workspace(csa.OP_TREE_ATTN, c["batch"], c["nodes"], c["heads"], c["k"], cache.capacity)
        return csa.csa2_tree_attn(cache, s["q"], s["pos"], s["parent"], s["draft"], s["swa"], s["swa_pos0"], idx=s["idx"],
                                  scale=s["scale"], out=s["out"], lse=s["lse"], ws=s["ws"])
    if op == "append":
        cache = csa.Cache.of(s["codes"], s["scales"], s["kcodes"], s["kscales"], ratio=c["ratio"])
        wik = s["wik"] or (None, None)
        csa.csa2_cache_append(cache, s["rows"], s["pos0"], path=s["path"], prev=s["prev"], prev_out=s["prev_out"], w0=s["w0"],
                              w1=s["w1"], wik_codes=wik[0], wik_scales=wik[1])
        outs = [csa.csa2_cache_read(cache, s["written"], out=s["out"])]
        if c["ratio"] == 2:
            outs.append(s["prev_out"])
        if c["keys"]:
            outs.append(csa.csa2_cache_read(cache, s["written"], keys=True, out=s["kout"]))
        return outs
    planes = s["latents"] + (s["codes"], s["scales"]) if c["keys"] else (s["codes"], s["scales"])
    cache = csa.Cache.of(*planes)
    return csa.csa2_cache_read(cache, s["idx"], count=None if c["listed"] else c["n"], keys=c["keys"], out=s["out"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "read":
        d = c["d_idx"] if c["keys"] else D_LAT
        rows = c["batch"] * min(c["n"], c["capacity"])
        return {"bytes": rows * (d // 2 + d // 16) + c["batch"] * c["n"] * (d * _SIZE[c["out"]] + (4 if c["listed"] else 0)),
                "flops": 1.0 * c["batch"] * c["n"] * d}
    if c["op"] == "append":
        B, r, d = c["batch"], c["ratio"], c["d_idx"] if c["keys"] else 0
        n = B * (0.5 * (c["path"] + 1) if c["tree"] else c["path"])                  # accepted rows, the mean of the draw
        each = (D_LAT + d) * 9 / 16
        # rows in, entries out, the same entries in again and their values out
        return {"bytes": n * D_LAT * 2 + n / r * (2 * each + (D_LAT + d) * _SIZE[c["out"]]) + (B * D_LAT * 4 if r == 2 else 0)
                + d * D_LAT * 9 / 16,
                "flops": n / r * D_LAT * (4.0 + 2.0 * d)}
    B, N, H = c["batch"], c["nodes"], c["heads"]
    each = max(0, c["ctx"] - WINDOW) / c["ratio"]
    nodes, win = 1.0 * N, min(WINDOW, c["ctx"])
    if c["ragged"]:
        each *= 0.5 * (B - 1) / B
        nodes = 0.5 * (N + 1)
    entries = min(2 * c["k"], each) if c["k"] else each
    keys = min(c["k"], each) if c["k"] else each
    return {"bytes": B * (entries * 288 + (win + nodes) * 1024 + nodes * (c["k"] * 4 + H * (2 * D_LAT)))
            + B * N * H * (D_LAT * _SIZE[c["out"]] + 4),
            "flops": 4.0 * B * nodes * H * D_LAT * (keys + win)}


# ---------------------------------------------------------------- the definitions in 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


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


def _nearest(x, grid):
    """the nearest of an ascending grid for every x >= 0 within it; ties to the even place in the grid"""
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    pick = torch.where(up < down, hi, lo)
    return grid[torch.where(up == down, hi + (hi & 1) * -1, pick)]


def _stored(x):
    """what the cache holds of rows x, as values in 64 bits"""
    e4m3 = torch.tensor([m / 8 * 2.0 ** -6 for m in range(8)]
                        + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8 if e < 15 else 7)],
                        dtype=torch.float64, device=x.device)
    e2m1 = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    g = x.double().unflatten(-1, (-1, 16))
    big = (g.abs().amax(-1) / 6.0).float().double().clamp_max(448.0)
    s = _nearest(big, e4m3)[..., None]
    safe = torch.where(s > 0, s, 1.0)
    v = _nearest((g.abs() / safe).clamp_max(6.0), e2m1) * s
    return (torch.sign(g) * v).flatten(-2)


def _exact_tree(c, s):
    B, N, H = s["q"].shape[:3]
    out = torch.zeros((B, N, H, D_LAT), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, H), -math.inf, dtype=torch.float64, device="cuda")
    parents = s["parent"].tolist()
    for b in range(B):
        at = int(s["swa_pos0"][b])
        furthest = max(0, int(s["pos"][b].max()) - (WINDOW - 1)) // c["ratio"]
        lat = None if c["k"] else _decode(s["codes"][b, :furthest], s["scales"][b, :furthest])
        for i in range(N):
            chain, j = [], i
            while j >= 0:
                chain.append(j)
                j = parents[b][j]
            if j != -1:
                continue
            p = int(s["pos"][b, i])
            if c["k"]:
                e = s["idx"][b, i][s["idx"][b, i] >= 0].long()
                entries = _decode(s["codes"][b, e], s["scales"][b, e])
            else:
                entries = lat[:max(0, p - (WINDOW - 1)) // c["ratio"]]
            lo = max(0, p - (WINDOW - 1), at)
            near = torch.cat((s["swa"][b, lo - at:max(lo, p - len(chain) + 1) - at], s["draft"][b, chain])).double()
            q = s["q"][b, i].double()
            a = s["scale"] * torch.cat((q @ entries.T, q @ near.T), 1)
            lse[b, i] = torch.logsumexp(a, -1)
            w = torch.softmax(a, -1)
            out[b, i] = w[:, :len(entries)] @ entries + w[:, len(entries):] @ near
    return out, lse


def _exact_append(c, s):
    B, P, r, d = c["batch"], c["path"], c["ratio"], c["d_idx"]
    n = s["written"].shape[1]
    lat = torch.zeros((B, n, D_LAT), dtype=torch.float64, device="cuda")
    keys = torch.zeros((B, n, d), dtype=torch.float64, device="cuda")
    last = torch.zeros((B, D_LAT), dtype=torch.float64, device="cuda")
    wik = _decode(*s["wik"]) if c["keys"] else None
    for b in range(B):
        if s["path"] is None:
            rows = s["rows"][b, :P]
        else:
            rows = s["rows"][b][[j for j in s["path"][b].tolist() if j >= 0]]
        p = int(s["pos0"][b])
        if r == 2:
            rows = torch.cat((s["prev"][b:b + 1], rows))
            last[b] = rows[-1].double()
            rows = rows[1 - p % 2:]                      # from an even position on
            rows = rows[:len(rows) // 2 * 2].double()
            first = (s["w0"].double() * rows[0::2]).float().double()
            rows = (s["w1"].double() * rows[1::2] + first).float()
        e = _stored(rows)
        lat[b, :len(e)] = e
        if c["keys"]:
            keys[b, :len(e)] = _stored((e @ wik.T).float())
    return [lat] + ([last] if r == 2 else []) + ([keys] if c["keys"] else [])


def _exact_read(c, s):
    if s["idx"] is None:
        return _decode(s["codes"][:, :c["n"]], s["scales"][:, :c["n"]])
    rows = [_decode(s["codes"][b, s["idx"][b].long()], s["scales"][b, s["idx"][b].long()]) for b in range(c["batch"])]
    return torch.stack(rows) * (s["idx"] >= 0)[..., None]


def exact(case, seed):
    return {"tree": _exact_tree, "append": _exact_append, "read": _exact_read}[case["op"]](case, prepare(case, seed))
