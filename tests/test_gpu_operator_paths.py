"""Calls of the operators around the attention that reach their less trodden paths: many short shares a
block and several passes of the dense attention, against the same 64-bit forms as test_gpu_operators."""
import math

import pytest
import torch

from test_gpu_operators import BF, HF, F, U, check_linear, csa, decode, dense_case, fp4, gen, randn, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- FP4-weight products

@pytest.mark.parametrize("T", [3, 20, 70])
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("K", [512, 4096])
def test_linear_small_tokens_with_a_small_alpha(csa, T, xt, K):
    """a token's power of two times alpha lies below fp32's normal range, the results do not"""
    x = (randn((T, 1, K), gen(K)) * 2.0 ** -112).to(xt)
    check_linear(csa, T, 1, K, 40, xt, F, x=x, alpha=1.37 * 2.0 ** -14)


@pytest.mark.parametrize("T", [3, 20, 70])
@pytest.mark.parametrize("K", [512, 4096])
def test_linear_large_tokens_with_a_large_alpha(csa, T, K):
    """... or above its range: rows without weights still give zeros, the others the infinity that they round to"""
    g = gen(K)
    codes, scales = fp4((40, K), g)
    scales[::3] = 0
    y = csa.csa2_linear_fp4(randn((T, K), g) * 2.0 ** 105, codes, scales, 2.0 ** 36)
    assert not y[:, ::3].any()
    y[:, ::3] = math.inf
    assert bool(torch.isinf(y).all())


@pytest.mark.parametrize("xt", [BF, HF, F])
@pytest.mark.parametrize("T,G,K,M", [(2048, 1, 1536, 1000), (8192, 1, 272, 520), (2050, 3, 112, 129)])
def test_linear_prompt_chunks(csa, T, G, K, M, xt):
    check_linear(csa, T, G, K, M, xt, xt, seed=T)


@pytest.mark.parametrize("xt,T", [(BF, 40), (HF, 40), (F, 40), (HF, 16)])
def test_linear_many_tokens_take_weights_just_quantised(csa, xt, T):
    """the quantiser and the product of many tokens back to back, new weights each time: as with a wait in between"""
    g = gen(6)
    x = randn((T, 1536), g, xt)
    ws = [randn((15000, 1536), g) for _ in range(4)]
    codes = torch.empty((15000, 768), dtype=torch.uint8, device="cuda")
    scales = torch.empty((15000, 96), dtype=torch.uint8, device="cuda")
    want = []
    for w in ws:
        csa.csa2_quantize_fp4(w, codes, scales)
        torch.cuda.synchronize()
        want.append(csa.csa2_linear_fp4(x, codes, scales, out_dtype=F))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for w in ws:
            csa.csa2_quantize_fp4(w, codes, scales)
            got.append(csa.csa2_linear_fp4(x, codes, scales, out_dtype=F))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("D,R,T", [(512, 64, 1), (512, 64, 300), (80, 40, 40), (36, 12, 40), (1024, 64, 9), (66, 10, 40)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_takes_weights_just_written(csa, D, R, T, halves):
    """weights, frequencies and positions that the kernel just before the call writes, other ones each time, for
    the wide and the narrow accesses: as with a wait in between, eagerly and in a graph"""
    g = gen(D)
    n = 12
    x, y = randn((T, 5, D), g, BF), torch.empty((n, T, 5, D), dtype=F, device="cuda")
    k, z = randn((T, 1, D), g, BF), torch.empty((n, T, 1, D), dtype=F, device="cuda")
    ws = [[randn((D,), g) for _ in range(n)] for _ in range(2)]
    fs = [torch.rand((R // 2,), generator=g, device="cuda") for _ in range(n)]
    ps = [torch.randint(0, 1 << 20, (T,), generator=g, device="cuda") for _ in range(n)]
    qw, kw, f, p = (torch.empty_like(v[0]) for v in (ws[0], ws[1], fs, ps))

    def steps(sync):
        for i in range(n):
            # the one just before the call changes from step to step
            todo = [(f, fs), (p, ps), (kw, ws[1]), (qw, ws[0])]
            for dst, src in todo[i % 4:] + todo[:i % 4]:
                dst.copy_(src[i])
            if sync:
                torch.cuda.synchronize()
            csa.csa2_norm_rope(x, p, f, qw, k, kw, halves=halves, q_out=y[i], k_out=z[i])

    steps(True)
    torch.cuda.synchronize()
    want = y.clone(), z.clone()
    for _ in range(10):
        y.zero_(), z.zero_()
        steps(False)
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        steps(False)
    for _ in range(10):
        y.zero_(), z.zero_()
        gr.replay()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])


# ---------------------------------------------------------------- attention over every visible entry

def test_dense_hands_many_short_shares_over(csa):
    """1,024 queries of one or two FP4 tiles and a window each: every block goes through some fourteen shares, its
    loaders ahead of the other warps; each call gives what the first gave, and no wait gives up"""
    g = gen(21)
    B, Q, H, cap = 4, 256, 8, 128
    codes, _ = fp4((B, cap, 512), g)
    scales = torch.randint(0x28, 0x38, (B, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    cache = csa.Cache.of(codes, scales, ratio=2)
    pos = torch.randint(128, 383, (B, Q), generator=g, device="cuda")
    q, swa = randn((B, Q, H, 512), g, BF), randn((B, 383, 512), g, BF)
    ws = csa.workspace(csa.OP_DENSE_ATTN, B, Q, H, 0, cap)
    first, _ = csa.csa2_dense_attn(cache, q, pos, swa, None, ws=ws)
    for _ in range(50):
        again, _ = csa.csa2_dense_attn(cache, q, pos, swa, None, ws=ws)
        assert torch.equal(first, again)
    assert bool(torch.isfinite(first).all()) and csa.csa2_poll_error(ws) == csa.OK


@pytest.mark.parametrize("B,Q,H", [(7, 100, 16),      # more (query, 64 heads) pairs than threads: two a thread
                                   (1, 1024, 8), (1, 1025, 8),                 # one pass to the last pair, and one pair more
                                   (3, 700, 16), (2, 390, 100)])               # passes that begin inside a sequence
def test_dense_many_queries(csa, B, Q, H):
    pos = torch.arange(Q)[None] // 3 + 61 * torch.arange(B)[:, None]
    pos[0, :5] = -4                                                            # see nothing
    pos[-1, Q // 2:] = torch.randint(0, 420, (Q - Q // 2,), generator=torch.Generator().manual_seed(Q))
    dense_case(csa, B, Q, H, 280, pos, ratio=1, out_dtype=F, seed=Q, swa_len=440)


@pytest.mark.parametrize("n", [1 << 13, 1 << 17])
def test_dense_long_even_tail_below_one_entry(csa, n):
    """one entry 18 nats above n - 1 equal ones, which have dims of their own: 152 queries, so that a block takes a
    whole one.  Each of the tail's weights is 2^-26 of the largest, its part of the output n times that."""
    Q = 152
    codes = torch.zeros((1, n, 256), dtype=torch.uint8, device="cuda")
    codes[0, 0, :128], codes[0, 1:, 128:] = 0x22, 0x22                # ones in dims 0-255, in dims 256-511
    scales = torch.full((1, n, 32), 0x38, dtype=torch.uint8, device="cuda")
    q = torch.zeros((1, Q, 16, 512), device="cuda").to(BF)
    q[..., :256] = 9.0 / 128
    pos = torch.full((1, Q), n + 127, dtype=torch.int64, device="cuda")
    out, lse = csa.csa2_dense_attn(csa.Cache.of(codes, scales, ratio=1), q, pos, None, None, 1.0, out_dtype=F, want_lse=True)
    tail = (n - 1) * math.exp(-18.0)
    want = torch.full((512,), 1.0 / (1.0 + tail), dtype=torch.float64, device="cuda")
    want[256:] = tail / (1.0 + tail)
    # scores exact (256 equal products), P half a step of fp16 or 2^-25 where the largest is 2^7 or more, fp32 sums
    tol = want * (2.0 ** -11 + n * U + 2.0 ** -20) + n * 2.0 ** -32
    within(out, want.expand(out.shape), tol.expand(out.shape))
    assert float((lse.double() - 18.0 - math.log1p(tail)).abs().max()) <= tail * n * U + 2.0 ** -18
