"""Attention of drafted trees against a plain 64-bit form of its definition.  Tolerances count roundings, as in
test_gpu_operators: 512 products a score in fp32 (u = 2^-24 each), the softmax weights in fp16 (2^-11 of each, or
2^-25 of one, the largest being at least 1), the sums, and half a step of the output's type."""
import math

import pytest
import torch

from test_gpu_operators import BF, F, HF, U, csa, decode, fp4, gen, randn, within  # noqa: F401

pytestmark = pytest.mark.gpu


def chains(parent):
    """for every node its chain, the node first; none where the chain does not end at a committed token"""
    out = []
    for i in range(len(parent)):
        chain, j = [], i
        while j >= 0:
            chain.append(j)
            j = parent[j] if -1 <= parent[j] < j else -2
        out.append(chain if j == -1 else [])
    return out


def tree64(codes, scales, q, pos, parent, draft, swa, swa_pos0, idx, scale, ratio):
    B, N, H = q.shape[:3]
    out = torch.zeros((B, N, H, 512), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, H), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    cap = codes.shape[1]
    for b in range(B):
        far = min(max(0, int(pos[b].max()) - 127) // ratio, cap)
        every = decode(codes[b, :far], scales[b, :far]) if idx is None else None
        for i, chain in enumerate(chains(parent[b].tolist())):
            if not chain:
                continue
            p = int(pos[b, i])
            if idx is None:
                L = every[:min(max(0, p - 127) // ratio, cap)]
            else:
                e = idx[b, i][(idx[b, i] >= 0) & (idx[b, i] < cap)].long()
                L = decode(codes[b, e], scales[b, e])
            rows = [L]
            if swa is not None:
                p0 = int(swa_pos0[b]) if swa_pos0 is not None else 0
                lo, hi = max(0, p - 127, p0), min(p - len(chain), p0 + swa.shape[1] - 1)
                if hi >= lo:
                    rows.append(swa[b, lo - p0:hi + 1 - p0].double())
            rows.append(draft[b, chain].double())
            L = torch.cat(rows)
            q64 = q[b, i].double()
            s = scale * q64 @ L.T
            lse[b, i] = torch.logsumexp(s, -1)
            w = torch.softmax(s, -1)
            out[b, i] = w @ L
            ds = float((512 * U * abs(scale) * (q64.abs() @ L.abs().T)).max()) + 2.0 ** -20 * float(s.abs().max())
            rel = 2.0 ** -11 + 2 * ds + L.shape[0] * U
            tol[b, i] = rel * (w @ L.abs()) + L.shape[0] * 2.0 ** -25 * L.abs().amax(0)
            ltol[b, i] = 2 * ds + 2.0 ** -20 * (1 + lse[b, i].abs()) + L.shape[0] * U
    return out, lse, tol, ltol


def random_parents(B, N, g):
    u = torch.rand((B, N), device="cuda", generator=g)
    return torch.minimum((u * (torch.arange(N, device="cuda") + 1)).int(), torch.arange(N, device="cuda").int()) - 1


def depths(parent):
    return torch.tensor([[max(0, len(c) - 1) for c in chains(p)] for p in parent.tolist()], device="cuda")


def tree_inputs(B, N, H, cap, base, ratio=2, parent=None, k=None, swa_len=128, seed=0, q_mul=1.0, win_mul=1.0, first=None):
    """base: the committed positions of each sequence.  What no node attends to holds NaN."""
    g = gen(seed)
    base = torch.as_tensor(base, device="cuda", dtype=torch.int64).expand(B).contiguous()
    parent = random_parents(B, N, g) if parent is None else torch.as_tensor(parent, device="cuda", dtype=torch.int32).expand(B, N).contiguous()
    pos = base[:, None] + depths(parent)
    there = torch.tensor([[bool(c) for c in chains(p)] for p in parent.tolist()], device="cuda")
    codes, _ = fp4((B, cap, 512), g)
    scales = torch.randint(0x28, 0x38, (B, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    idx = None
    if k is not None:
        # distinct entries, empty slots and numbers outside the cache in between
        idx = torch.rand((B, N, max(k, cap)), device="cuda", generator=g).argsort(2)[..., :k].int()
        drop = torch.rand(idx.shape, device="cuda", generator=g)
        idx = torch.where(drop < 0.1, -1, torch.where(drop < 0.15, cap + idx, idx)).int().contiguous()
        idx = torch.where(idx < cap, idx, torch.where(drop < 0.1, -1, cap + 5)).int().contiguous()
    else:
        n_vis = ((pos.masked_fill(~there, -1).amax(1) - 127).clamp_min(0) // ratio).clamp_max(cap)
        scales[torch.arange(cap, device="cuda")[None] >= n_vis[:, None]] = 0x7F
    swa = pos0 = None
    if swa_len:
        pos0 = (base - (swa_len - 1)).clamp_min(0) if first is None else torch.as_tensor(first, device="cuda").expand(B).contiguous()
        swa = (randn((B, swa_len, 512), g) * win_mul).to(BF)
        at = pos0[:, None] + torch.arange(swa_len, device="cuda")
        swa[(at >= base[:, None]) | (at < base[:, None] - 127)] = math.nan
    draft = (randn((B, N, 512), g) * win_mul).to(BF)
    draft[~there] = math.nan
    q = (randn((B, N, H, 512), g) * q_mul).to(BF)
    q[~there] = math.nan
    return dict(codes=codes, scales=scales, q=q, pos=pos, parent=parent, draft=draft, swa=swa, swa_pos0=pos0, idx=idx, ratio=ratio)


def call(csa, x, **kw):
    cache = csa.Cache.of(x["codes"], x["scales"], ratio=x["ratio"])
    return csa.csa2_tree_attn(cache, x["q"], x["pos"], x["parent"], x["draft"], x["swa"], x["swa_pos0"], idx=x["idx"], **kw)


def check(csa, x, scale=512 ** -0.5, out_dtype=BF, **kw):
    out, lse = call(csa, x, scale=scale, out_dtype=out_dtype, want_lse=True, **kw)
    ref, rlse, tol, ltol = tree64(x["codes"], x["scales"], x["q"], x["pos"], x["parent"], x["draft"], x["swa"], x["swa_pos0"],
                                  x["idx"], scale, x["ratio"])
    within(out, ref, tol)
    within(lse, rlse, ltol)
    return out, lse


CHAIN = lambda n: list(range(-1, n - 1))


@pytest.mark.parametrize("base", [0, 1, 5, 63, 64, 126, 127, 128, 129, 130, 200, 255, 256, 257, 383, 384, 385, 1000])
@pytest.mark.parametrize("ratio", [1, 2])
def test_tree_short_contexts(csa, base, ratio):
    check(csa, tree_inputs(1, 7, 64, 900, base, ratio=ratio, seed=base))


@pytest.mark.parametrize("H", [1, 3, 8, 15, 16, 17, 24, 32, 63, 64, 65, 100, 128])
@pytest.mark.parametrize("k", [None, 70])
def test_tree_heads(csa, H, k):
    check(csa, tree_inputs(2, 5, H, 700, [900, 40], seed=H, k=k), out_dtype=F)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 9, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128])
def test_tree_nodes(csa, N):
    check(csa, tree_inputs(2, N, 24, 700, [750, 130], ratio=1, seed=N), out_dtype=HF)


@pytest.mark.parametrize("N", [1, 2, 40, 128])
@pytest.mark.parametrize("k", [None, 33])
def test_tree_shapes(csa, N, k):
    """a chain, children of the last committed token only, a comb, pairs"""
    for s, parent in enumerate([CHAIN(N), [-1] * N, [max(-1, i - 2) for i in range(N)], [(i - 1) // 2 if i else -1 for i in range(N)]]):
        check(csa, tree_inputs(1, N, 16, 400, 400, parent=parent, seed=s, k=k))


@pytest.mark.parametrize("k", [None, 20])
def test_tree_nodes_that_are_not_there(csa, k):
    i32 = 1 << 31
    parent = [[-1, 0, -2, 2, 1, 5, 9, 7, -i32, i32 - 1, 4], [-2] * 11, [0, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [-1, 0, 1, 2, 3, -2, 5, 6, 7, 8, -1]]
    x = tree_inputs(4, 11, 64, 500, [600, 300, 100, 127], parent=parent, seed=3, k=k)
    out, lse = check(csa, x)
    gone = torch.tensor([[not c for c in chains(p)] for p in parent], device="cuda")
    assert not out[gone].any() and bool((lse[gone] == -math.inf).all()) and int(gone.sum()) == 7 + 11 + 11 + 5


@pytest.mark.parametrize("k", [0, 1, 7, 63, 64, 65, 512, 2047, 2048])
@pytest.mark.parametrize("H", [64, 20])
def test_tree_lists(csa, k, H):
    x = tree_inputs(2, 3, H, 2500, [3000, 77], seed=k, k=k)
    if k > 1:
        x["idx"][0, 0] = -1                                  # a list with nothing in it
        x["idx"][1, 2, 1:] = -1                              # and one with a single slot
    check(csa, x, out_dtype=F)


def test_tree_lists_larger_than_the_cache_and_extreme_numbers(csa):
    x = tree_inputs(1, 2, 64, 3, 500, seed=1, k=40)
    x["idx"][0, 0, ::3] = (1 << 31) - 1
    x["idx"][0, 1, ::3] = -(1 << 31)
    check(csa, x)


@pytest.mark.parametrize("out_dtype", [BF, HF, F])
@pytest.mark.parametrize("k", [None, 100])
def test_tree_out_types(csa, out_dtype, k):
    check(csa, tree_inputs(2, 3, 64, 500, [700, 500], ratio=1, k=k), out_dtype=out_dtype)


@pytest.mark.parametrize("H,N", [(16, 3), (64, 5), (128, 4), (8, 33)])
def test_tree_long_contexts(csa, H, N):
    check(csa, tree_inputs(1, N, H, 20011, 20009, ratio=1, seed=H))


def test_tree_ragged_batch(csa):
    check(csa, tree_inputs(6, 12, 64, 3100, [3000, 0, 126, 1500, 2999, 64], ratio=1, seed=3, swa_len=300))
    check(csa, tree_inputs(6, 12, 64, 3100, [6200, 0, 126, 1500, 2999, 64], ratio=2, seed=4, k=512))


@pytest.mark.parametrize("k", [None, 64])
def test_tree_window_clipped_absent_and_elsewhere(csa, k):
    check(csa, tree_inputs(2, 6, 64, 400, [600, 300], swa_len=20, k=k))              # fewer rows than the window
    check(csa, tree_inputs(2, 6, 64, 400, [600, 50], swa_len=0, k=k))                # none
    check(csa, tree_inputs(2, 6, 64, 400, [600, 300], swa_len=60, first=[550, 298], k=k))    # rows of the future too
    check(csa, tree_inputs(2, 6, 64, 400, [600, 300], swa_len=60, first=[700, 0], k=k))      # none of the window's
    x = tree_inputs(2, 6, 64, 400, [90, 30], swa_len=128, first=[0, 0], k=k)
    check(csa, {**x, "swa_pos0": None})                                              # (zeros)


def test_tree_positions_far_and_negative(csa):
    """positions past 2^32 see the cache's entries, negative ones none"""
    x = tree_inputs(2, 4, 16, 300, [5_000_000_000, 300], ratio=1, parent=CHAIN(4))
    x["pos"][1] = torch.tensor([-5, -4, -3, -2], device="cuda")
    x["scales"][1].fill_(0x7F)
    check(csa, x)


@pytest.mark.parametrize("q_mul,win_mul", [(1e3, 1.0), (2.0 ** -30, 1.0), (1.0, 2.0 ** 20), (1.0, 2.0 ** -20), (4.0, 64.0)])
@pytest.mark.parametrize("k", [None, 90])
def test_tree_inputs_far_outside_fp16(csa, q_mul, win_mul, k):
    check(csa, tree_inputs(2, 5, 64, 300, [500, 90], q_mul=q_mul, win_mul=win_mul, seed=7, k=k))


def test_tree_rows_of_very_different_size(csa):
    """committed rows and drafts far apart in size, in one window"""
    for a, b in [(2.0 ** 18, 1.0), (1.0, 2.0 ** 18), (2.0 ** -14, 1.0)]:
        x = tree_inputs(1, 6, 64, 300, 500, seed=9)
        x["swa"], x["draft"] = (x["swa"].float() * a).to(BF), (x["draft"].float() * b).to(BF)
        check(csa, x)


@pytest.mark.parametrize("N", [1, 3])
def test_tree_rising_scores_rescale_the_output(csa, N):
    """entries whose scores climb by more than 2^8 from tile to tile: the running max is raised each time"""
    cap = 640
    x = tree_inputs(1, N, 64, cap, cap + 127, ratio=1, seed=11)
    g = gen(11)
    x["codes"].fill_(0x22)                                                            # every value 1
    x["codes"][0, :, 0] = torch.randint(0, 256, (cap,), generator=g, device="cuda", dtype=torch.uint8)
    x["scales"] = (0x20 + 2 * (torch.arange(cap, device="cuda") // 64)).to(torch.uint8)[None, :, None].expand(1, cap, 32).contiguous()
    x["q"].fill_(1.0)
    x["q"][:, :, ::2] *= 0.25
    x["swa"] = x["swa_pos0"] = None
    x["draft"].fill_(0.125)
    check(csa, x, scale=1.0, out_dtype=F)


def test_tree_long_even_tail_next_to_one_large_score(csa):
    """20,000 entries some 18 nats below one draft: together they weigh in the output"""
    cap = 20000
    x = tree_inputs(1, 2, 16, cap, cap + 127, ratio=1, parent=[-1, -1], seed=2)
    x["codes"].fill_(0x22)
    x["scales"].fill_(0x30)                                                           # every value 0.5
    x["q"].fill_(1.0)
    x["draft"].zero_()
    x["draft"][:, :, :36] = 0.5                                                       # scale 1: draft 18, entries 0 (half of q negative)
    x["q"][..., 256:] = -1.0
    x["swa"] = x["swa_pos0"] = None
    check(csa, x, scale=1.0, out_dtype=F)


def test_tree_of_a_chain_equals_dense_queries(csa):
    """a chain of drafts whose rows are put into the window: csa2_dense_attn's queries in a row"""
    x = tree_inputs(3, 5, 64, 900, [900, 60, 300], parent=CHAIN(5), seed=5)
    out, lse = call(csa, x, out_dtype=F, want_lse=True)
    pos0 = x["pos"][:, 0] - 127
    win = torch.zeros((3, 132, 512), dtype=BF, device="cuda")
    for b in range(3):
        base = int(x["pos"][b, 0])
        have = min(base, 127)
        win[b, 127 - have:127] = x["swa"][b, base - have - int(x["swa_pos0"][b]):base - int(x["swa_pos0"][b])]
    win[:, 127:] = x["draft"]
    cache = csa.Cache.of(x["codes"], x["scales"], ratio=2)
    ref, rlse = csa.csa2_dense_attn(cache, x["q"], x["pos"], win, pos0, out_dtype=F, want_lse=True)
    # each within 2^-11 of its weights and the sums' roundings
    assert float((out - ref).abs().max()) <= 2 * 2.0 ** -10 * float(ref.abs().max())
    assert float((lse - rlse).abs().max()) <= 1e-4


def test_tree_cache_past_32_bit_offsets(csa):
    """sequences whose rows lie beyond 2^31 bytes of the code plane, and beyond 2^32"""
    g = gen(8)
    B, cap, n = 3, 6_000_000, 300                           # 1.5 GB of codes a sequence
    codes = torch.empty((B, cap, 256), dtype=torch.uint8, device="cuda")
    codes[:, :] = torch.randint(0, 256, (1, 1, 256), generator=g, device="cuda", dtype=torch.uint8)
    for b in range(B):
        codes[b, :n] = torch.randint(0, 256, (n, 256), generator=g, device="cuda", dtype=torch.uint8)
        codes[b, -n:] = torch.randint(0, 256, (n, 256), generator=g, device="cuda", dtype=torch.uint8)
    x = tree_inputs(B, 4, 64, 8, n + 127, ratio=1, seed=8)
    x.update(codes=codes, scales=torch.full((B, cap, 32), 0x30, dtype=torch.uint8, device="cuda"))
    check(csa, x, out_dtype=F)
    x["idx"] = (cap - 1 - torch.randint(0, n, (B, 4, 100), generator=g, device="cuda")).int()
    check(csa, x, out_dtype=F)


@pytest.mark.parametrize("k", [None, 512])
def test_tree_writes_only_its_outputs(csa, k):
    x = tree_inputs(2, 5, 24, 900, [1500, 200], seed=1, k=k)
    n = 2 * 5 * 24
    o = torch.full((n + 2, 512), 7.0, device="cuda")
    l = torch.full((n + 8,), 7.0, device="cuda")
    need = csa.csa2_workspace_size(csa.OP_TREE_ATTN, 2, 5, 24, -1 if k is None else k, 900)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    ws[:16].zero_()
    want, wl = call(csa, x, out_dtype=F, want_lse=True)
    call(csa, x, out=o[1:-1].view(2, 5, 24, 512), lse=l[4:-4].view(2, 5, 24), ws=ws[:need])
    assert torch.equal(o[1:-1].view_as(want), want) and torch.equal(l[4:-4].view_as(wl), wl)
    assert bool((o[0] == 7).all()) and bool((o[-1] == 7).all()) and bool((l[:4] == 7).all()) and bool((l[-4:] == 7).all())
    assert bool((ws[need:] == 0x5A).all()) and csa.csa2_poll_error(ws) == csa.OK


@pytest.mark.parametrize("k", [None, 300])
def test_tree_repeats_and_replays(csa, k):
    """the same bits call after call; two graphs of different batches that share a workspace, replayed in turn with
    new inputs"""
    a = tree_inputs(3, 9, 64, 2000, [3000, 10, 900], seed=1, k=k)
    b = tree_inputs(1, 9, 64, 2000, [3900], seed=2, k=k)
    ws = csa.workspace(csa.OP_TREE_ATTN, 3, 9, 64, 0, 2000)
    runs, graphs = [], []
    for x in (a, b):
        out, lse = call(csa, x, want_lse=True)
        out2, lse2 = call(csa, x, want_lse=True, ws=ws)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        runs.append((out, lse))
    for x in (a, b):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out, lse = torch.empty_like(x["q"]), torch.empty(x["q"].shape[:3], device="cuda")
        with torch.cuda.stream(s):
            call(csa, x, out=out, lse=lse, ws=ws)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(csa, x, out=out, lse=lse, ws=ws)
        graphs.append((g, out, lse))
    for _ in range(3):
        for (g, out, lse), (want, wl) in zip(graphs, runs):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for (g, out, lse), (want, wl) in zip(graphs, runs):
            assert torch.equal(out, want) and torch.equal(lse, wl)
    # new positions, trees and rows in the same buffers
    y = tree_inputs(3, 9, 64, 2000, [127, 3500, 2100], seed=5, k=k)
    for name in ("codes", "scales", "q", "pos", "parent", "draft", "swa", "swa_pos0") + (("idx",) if k else ()):
        a[name].copy_(y[name])
    graphs[0][0].replay()
    want, wl = call(csa, y, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want) and torch.equal(graphs[0][2], wl)
    assert csa.csa2_poll_error(ws) == csa.OK


def test_tree_on_two_streams(csa):
    """calls at once on two streams, without workspaces and with one each"""
    xs = [tree_inputs(4, 8, 64, 3000, [5000, 300, 4000, 20], seed=s) for s in range(2)]
    want = [call(csa, x, want_lse=True) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    wss = [csa.workspace(csa.OP_TREE_ATTN, 4, 8, 64, -1, 3000) for _ in xs]
    outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(4)] for w in want]
    torch.cuda.synchronize()
    for n in range(4):
        for x, s, ws, o in zip(xs, streams, wss, outs):
            call(csa, x, out=o[n][0], lse=o[n][1], ws=ws if n % 2 else None, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for out, lse in o:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("entries,k", [(8, None), (40, 8), (3000, 2048), (3_000_000, None)])
def test_tree_fp32_outputs_keep_their_bits(csa, entries, k):
    """fp32 outputs, whatever the number of keys.  A score is one product of few bits and at most 1 in size, a value is
    positive, so that what counts is: weights to 2^-22 each, of exponents off by 2^-23 of some 16 at most; runs of 48
    tensor-core sums (one step of fp32, 2^-23, each); then fp32 sums (2^-24 each) of a row's tiles of 128, of the 76 pairs'
    or 152 blocks' shares, twice (outputs and weights); a low part of a weight that underflows, 2^-32 of the largest weight."""
    g = gen(entries)
    N, H = (2, 3) if k is None else (128, 128)
    codes = torch.randint(0, 256, (1, entries, 256), generator=g, device="cuda", dtype=torch.uint8) & 0x77
    codes[..., 0] = torch.randint(0, 256, (1, entries), generator=g, device="cuda", dtype=torch.uint8)    # dims 0 and 1: any sign
    scales = torch.full((1, entries, 32), 0x30, device="cuda", dtype=torch.uint8)                         # 0.5: values to 3
    q = torch.zeros((1, N, H, 512), device="cuda", dtype=BF)
    q[..., 0] = torch.rand((1, N, H), generator=g, device="cuda").to(BF) / 3
    draft = torch.rand((1, N, 512), generator=g, device="cuda").to(BF)
    pos = torch.full((1, N), entries + 127, device="cuda", dtype=torch.int64)
    parent = torch.full((1, N), -1, device="cuda", dtype=torch.int32)
    idx = None if k is None else torch.randint(0, entries, (1, N, k), generator=g, device="cuda", dtype=torch.int32)
    x = dict(codes=codes, scales=scales, q=q, pos=pos, parent=parent, draft=draft, swa=None, swa_pos0=None, idx=idx, ratio=1)
    out, lse = call(csa, x, scale=1.0, out_dtype=F, want_lse=True)
    keys = (entries if k is None else k) + 1
    rel = 2.0 ** -22 + 2 * 16 * 2.0 ** -23 + 48 * 2.0 ** -23 + 2 * (keys / 128 / (76 if k is None else 1) + 152 + 32) * U
    part = 200_000
    for i in range(N) if k is None else (0, 77, N - 1):
        qi, d = q[0, i].double(), draft[0, i].double()
        w = torch.exp(qi @ d)
        s, o = w.clone(), w[:, None] * d
        e = torch.arange(entries, device="cuda") if k is None else idx[0, i].long()
        for at in range(0, e.numel(), part):
            L = decode(codes[0, e[at:at + part]], scales[0, e[at:at + part]])
            w = torch.exp(qi @ L.T)
            s, o = s + w.sum(1), o + w @ L
        ref = o / s[:, None]
        within(out[0, i], ref, rel * ref.abs() + keys * 2.0 ** -32 * 3)
        within(lse[0, i], s.log(), rel + 2.0 ** -22 * (1 + s.log()))


@pytest.mark.parametrize("out_dtype", [BF, F])
def test_tree_lists_in_several_passes(csa, out_dtype):
    """more rows than a pass takes (65,536): the later sequences' results and the earlier ones'"""
    check(csa, tree_inputs(10, 64, 128, 300, [30 * b for b in range(10)], seed=21, k=20), out_dtype=out_dtype)


def test_tree_many_sequences(csa):
    """more sequences than a block has threads, some of them without a node that is there"""
    parent = [[-1, 0], [-2, 0], [-1, -1]]
    B = 1700
    x = tree_inputs(B, 2, 3, 40, [(7 * b) % 190 for b in range(B)], ratio=1, parent=(parent * B)[:B], seed=22)
    check(csa, x)
    x = tree_inputs(B, 2, 3, 40, [(7 * b) % 190 for b in range(B)], ratio=1, parent=(parent * B)[:B], seed=23, k=9)
    check(csa, x)


@pytest.mark.parametrize("k", [None, 50])
@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30, -3.0])
def test_tree_scales(csa, k, scale):
    """none, negative, next to nothing, large enough for one key to take all"""
    check(csa, tree_inputs(2, 4, 64, 500, [600, 77], seed=24, k=k), scale=scale)


def test_tree_same_entry_twice_counts_twice(csa):
    x = tree_inputs(1, 2, 16, 300, 500, seed=25, k=30)
    x["idx"][:, :, 1::2] = x["idx"][:, :, ::2]
    check(csa, x, out_dtype=F)
