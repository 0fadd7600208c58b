"""Attention of drafted trees over window rows and drafts of any size, side by side: what one row is like does not cost another its bits.

The queries have one value, so that a score is one product of few bits, at most 1 in size: what is left are the roundings of
the weights and rows.  With w and L in 64 bits an output is off by
    2^-11 of (w @ |L|), a weight in fp16, and 2^-18 of it: 16 sums of the tensor core (2^-23 each), the exponent's roundings
        (2^-22 of 1.5 each), the exponential's (2^-22), the sum of the weights (2^-22), twice each at most;
    2^-22 of each row's largest magnitude;
    2^-25 a key where a weight times its row's size underflows: n 2^-24 of the largest (w @ |L|), the largest such
        product being 2^7 at least and rows of one size within 2^8.
fp32 outputs have 1e-6 of the norm of w @ |L|, as the header says."""
import math

import pytest
import torch

from test_gpu_operators import BF, F, HF, csa, decode, fp4, gen, randn, within  # noqa: F401
from test_gpu_tree import chains, depths

pytestmark = pytest.mark.gpu
ABSENT = -2


def rows_of(sizes, g):
    """normal values of the given sizes (and at least 2^-6 of them in dim 0, which the scores are made of)"""
    n = randn(tuple(sizes.shape) + (512,), g).double()
    n[..., 0] = n[..., 0].sign() * n[..., 0].abs().clamp(2.0 ** -6, 1.0)
    return (n * sizes[..., None]).to(BF)


def make(base, parent, win, draft, H=64, k=None, cap=600, seed=0):
    """win: the sizes of the committed rows (a number or one each); draft: those of the drafts"""
    g = gen(seed)
    N = len(parent)
    parent = torch.tensor([parent], device="cuda", dtype=torch.int32)
    pos = torch.full((1, N), base, device="cuda", dtype=torch.int64) + depths(parent)
    codes, _ = fp4((1, cap, 512), g)
    codes[..., 0] &= 0xF0                                # dim 0 of the entries: scores of 0
    scales = torch.randint(0x28, 0x38, (1, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    wsize = torch.as_tensor(win, dtype=torch.float64, device="cuda").expand(1, 128)
    dsize = torch.as_tensor(draft, dtype=torch.float64, device="cuda").expand(1, N)
    swa, drafts = rows_of(wsize, g), rows_of(dsize, g)
    q = torch.zeros((1, N, H, 512), device="cuda", dtype=BF)
    for i, chain in enumerate(chains(parent[0].tolist())):
        if chain:
            # (of the committed rows a node sees the later ones; all are counted)
            q[0, i, :, 0] = 1.0 / max([float(wsize.max())] + [float(dsize[0, j]) for j in chain])
    q[..., 0] *= (torch.rand((1, N, H), generator=g, device="cuda") * 2 - 1).to(BF)
    idx = None if k is None else torch.randint(0, cap, (1, N, k), generator=g, device="cuda", dtype=torch.int32)
    return dict(codes=codes, scales=scales, q=q, pos=pos, parent=parent, draft=drafts, swa=swa,
                swa_pos0=torch.tensor([base - 128], device="cuda"), idx=idx)


def reference(x, scale):
    """for each node that is there: its number, w @ L, w @ |L|, w @ (the rows' largest magnitudes), lse, keys"""
    out = []
    for i, chain in enumerate(chains(x["parent"][0].tolist())):
        if not chain:
            continue
        p, p0, cap = int(x["pos"][0, i]), int(x["swa_pos0"][0]), x["codes"].shape[1]
        e = torch.arange(min(max(0, p - 127) // 2, cap), device="cuda") if x["idx"] is None else x["idx"][0, i].long()
        lo, hi = max(0, p - 127), p - len(chain)
        L = torch.cat((decode(x["codes"][0, e], x["scales"][0, e]), x["swa"][0, lo - p0:hi + 1 - p0].double(), x["draft"][0, chain].double()))
        s = scale * x["q"][0, i].double() @ L.T
        w = torch.softmax(s, -1)
        out.append((i, w @ L, w @ L.abs(), w @ L.abs().amax(1, keepdim=True), torch.logsumexp(s, -1), L.shape[0]))
    return out


def check(csa, x, scale=1.0):
    cache = csa.Cache.of(x["codes"], x["scales"], ratio=2)
    for dtype in (BF, HF, F):
        out, lse = csa.csa2_tree_attn(cache, x["q"], x["pos"], x["parent"], x["draft"], x["swa"], x["swa_pos0"], idx=x["idx"],
                                      scale=scale, out_dtype=dtype, want_lse=True)
        for i, ref, size, top, rlse, n in reference(x, scale):
            if dtype == F:
                err = (out[0, i].double() - ref).norm(dim=1) / size.norm(dim=1)
                assert float(err.max()) <= 1e-6, (i, float(err.max()))
            elif dtype == BF or float(size.max()) < 2.0 ** 14:
                within(out[0, i], ref, (2.0 ** -11 + 2.0 ** -18) * size + 2.0 ** -22 * top + n * 2.0 ** -24 * size.amax(1, keepdim=True))
            within(lse[0, i], rlse, 2.0 ** -20 * (1 + rlse.abs()))


LISTS = pytest.mark.parametrize("k", [None, 0, 40])
BASES = pytest.mark.parametrize("base", [100, 400])      # without entries and with


@LISTS
@BASES
@pytest.mark.parametrize("size", [-97, -60, -20, -12, -11, -10, -4, 0, 3, 14, 20, 60])
def test_rows_of_one_size_with_nodes_that_are_not_there(csa, size, base, k):
    """rows of 2^size, their largest values on both sides of a power of two, and a node left out between others"""
    check(csa, make(base, [-1, ABSENT, 0, -1, 2], 2.0 ** size, 2.0 ** size, k=k, seed=size + 100))


@LISTS
@BASES
@pytest.mark.parametrize("size", [-40, 12, 20, 30, 40, 50, 90])
def test_a_sibling_of_another_size(csa, size, base, k):
    """node 1 and its child are 2^size, all other rows near 1: nodes of the other branch do not see them"""
    check(csa, make(base, [-1, -1, 0, 1, 2], 1.0, [1.0, 2.0 ** size, 1.0, 2.0 ** size, 1.0], k=k, seed=size + 50))


@LISTS
@BASES
def test_rows_of_every_size_in_one_chain(csa, base, k):
    """committed rows of 2^-12 to 2^12, drafts of 2^-30 to 2^30"""
    win = 2.0 ** (torch.arange(128) % 25 - 12).double()
    check(csa, make(base, [-1, 0, 1, 2, 3, 4, 5], win, [2.0 ** (10 * i - 30) for i in range(7)], k=k, H=20, seed=5))


@LISTS
@BASES
@pytest.mark.parametrize("size", [20, 40, 120])
def test_a_large_row_without_weight(csa, size, base, k):
    """a node that sees a row of 2^size whose score leaves it no weight, and rows near 1 that have it all"""
    x = make(base, [-1, 0, -1], 1.0, [1.0, 2.0 ** size, 1.0], k=k, seed=size)
    x["q"][0, 1, :, 0] = 1.0
    x["draft"][0, 1, 0] = -(2.0 ** size)
    x["swa"][..., 0] = x["swa"][..., 0].abs()
    check(csa, x)


@LISTS
def test_queries_and_rows_of_opposite_sizes(csa, k):
    """queries of 2^100 against rows of 2^-97, and the other way about: scores near 1 (no entries: theirs are 0)"""
    for size in (-97, 100):
        check(csa, make(100, [-1, 0, -1], 2.0 ** size, 2.0 ** size, k=0 if k else k, seed=3), scale=-1.0)


@pytest.mark.parametrize("k", [None, 10])
def test_positions_that_contradict_the_tree(csa, k):
    """a chain of 128 whose nodes all claim one position, or positions in reverse, beside a tree that is as it should
    be: that one's results, and the same bits at every call"""
    x = make(400, list(range(-1, 127)), 1.0, 1.0, H=8, k=k, seed=9)
    two = {n: None if v is None else torch.cat((v, v)) for n, v in x.items()}
    cache = csa.Cache.of(two["codes"], two["scales"], ratio=2)

    def call(pos, parent):
        return csa.csa2_tree_attn(cache, two["q"], pos, parent, two["draft"], two["swa"], two["swa_pos0"], idx=two["idx"],
                                  scale=1.0, out_dtype=F, want_lse=True)

    want, wl = call(two["pos"], two["parent"])
    for pos, parent in ((torch.full_like(x["pos"], 400), x["parent"]), (x["pos"].flip(1), x["parent"]),
                        (x["pos"].flip(1), torch.full_like(x["parent"], -1)), (x["pos"] * 0 - (1 << 62), x["parent"]),
                        (x["pos"] * 0 + (1 << 62), x["parent"])):
        got = [call(torch.cat((pos, x["pos"])), torch.cat((parent, x["parent"]))) for _ in range(3)]
        for out, lse in got:
            # (two outputs within 1e-6; the shares of the work are others)
            assert float((out[1] - want[1]).norm()) <= 2e-6 * float(want[1].norm()) and float((lse[1] - wl[1]).abs().max()) <= 1e-5
            assert torch.equal(out, got[0][0]) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("k", [None, 0, 40])
@pytest.mark.parametrize("size,score", [(s, n) for s in (0, 13, -13) for n in range(15, 33 if s == 0 else 22)])
def test_scores_beyond_the_last_place_of_their_exponents(csa, score, size, k):
    """scores of 2^score: neighbours in fp32 lie up to 2^9 apart, so that a reference below the largest may be none or far;
    keys that tie have all the weight (rows of an exponent of their own have their bits below 2^22, as the header says)"""
    x = make(400, [-1, 0, -1], 2.0 ** size, 2.0 ** size, H=128, k=k, seed=score)
    x["q"] *= 2.0 ** score
    check(csa, x)
