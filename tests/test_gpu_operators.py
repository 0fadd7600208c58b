"""The operators around the attention (FP4-weight products, per-head norm with rotation, attention
over every visible entry) against plain 64-bit forms of their definitions.

Tolerances count roundings: u = 2^-24 for fp32 arithmetic, torch.finfo(t).eps / 2 for the one
rounding of an output to type t."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_decode_gb300 as m
    from compressed_sparse_attention_decode_gb300 import build as b
    b.build()
    m.load()
    assert torch.cuda.is_available()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, dtype=F):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def fp4(shape, g):
    """random codes and finite scales (every code; scales from subnormal to 28, either sign)"""
    codes = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0, 0x60, shape[:-1] + (shape[-1] // 16,), generator=g, device="cuda", dtype=torch.uint8)
    scales |= 128 * torch.randint(0, 2, scales.shape, generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def decode(codes, scales):
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = mags[n & 7] * torch.where(n >= 8, -1.0, 1.0)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2)


def within(got, want, tol):
    """|got - want| <= tol + half a step of got's type, elementwise; NaN and infinities in the same places"""
    got64 = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got64), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got64[inf], want[inf])
    f = torch.finfo(got.dtype)
    lim = tol + want.abs() * f.eps / 2 + f.smallest_normal * f.eps
    over = ((got64 - want).abs() - lim)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, float(((got64 - want).abs() / lim)[fin].max())


# ---------------------------------------------------------------- FP4-weight products

def check_linear(csa, T, G, K, M, xt, yt, pad=0, seed=0, alpha=0.37, x=None, scales=None):
    g = gen(seed)
    codes, sc = fp4((G, M, K), g)
    scales = sc if scales is None else scales
    if x is None:
        x = randn((T, G, K + pad), g, xt)[..., :K]
    y = torch.full((T, G, M + pad), 7.0, dtype=yt, device="cuda")
    out = y[..., :M]
    if G == 1:
        got = csa.csa2_linear_fp4(x[:, 0], codes[0], scales[0], alpha, out=out[:, 0])[:, None]
    else:
        got = csa.csa2_linear_fp4(x, codes, scales, alpha, out=out)
    w, x64 = decode(codes, scales), x.double()
    a32 = float(torch.tensor(alpha, dtype=F))
    want = torch.einsum("tgk,gmk->tgm", x64, w) * a32
    size = torch.einsum("tgk,gmk->tgm", x64.abs(), w.abs()) * abs(a32)
    # n_in products summed in fp32 in any order (and truncated sums of a tensor core), the two fp16
    # parts of an fp32 x (2^-22 of the element, and of the token's largest value 2^-39), alpha
    within(got, want, size.nan_to_num(0.0, 0.0) * ((K + 8) * U + 2.0 ** -21))
    if pad:
        assert bool((y[..., M:] == 7.0).all())       # nothing past the rows
    return got


@pytest.mark.parametrize("xt", [BF, HF, F])
@pytest.mark.parametrize("yt", [BF, HF, F])
def test_linear_types(csa, xt, yt):
    check_linear(csa, 3, 1, 208, 75, xt, yt)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 129, 257])
@pytest.mark.parametrize("xt", [BF, F])
def test_linear_tokens(csa, T, xt):
    check_linear(csa, T, 1, 528, 130, xt, F, seed=T)


@pytest.mark.parametrize("K", [0, 16, 32, 48, 64, 112, 128, 240, 256, 1040, 4096, 8208])
@pytest.mark.parametrize("T", [1, 20, 70])
def test_linear_inner_sizes(csa, K, T):
    check_linear(csa, T, 1, K, 33, BF, F, seed=K)


@pytest.mark.parametrize("M,K", [(1, 20912), (17, 20928), (700, 5120), (20000, 48), (9999, 1040), (3, 32768)])
def test_linear_few_tokens_of_long_and_short_rows(csa, M, K):
    check_linear(csa, 3, 1, K, M, BF, F, seed=K)


@pytest.mark.parametrize("M,K", [(5, 16), (33, 48), (35, 112), (1003, 1040)])
@pytest.mark.parametrize("T", [1, 12])
def test_linear_groups_off_16_byte_boundaries(csa, M, K, T):
    """groups whose codes and scales start between 16-byte boundaries, up to the last byte of the tensors"""
    check_linear(csa, T, 3, K, M, BF, F, seed=M)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 1003, 5000])
@pytest.mark.parametrize("T", [1, 40])
def test_linear_outer_sizes(csa, M, T):
    check_linear(csa, T, 1, 320, M, HF, F, seed=M)


@pytest.mark.parametrize("K", [112, 128, 384, 640, 1168])        # one and odd numbers of 128-value chunks
@pytest.mark.parametrize("T,xt", [(20, BF), (20, F), (70, HF), (200, BF)])
def test_linear_blocks_with_several_tiles(csa, K, T, xt):
    check_linear(csa, T, 1, K, 60001, xt, BF, seed=K)


@pytest.mark.parametrize("T,G,K,M", [(1, 3, 160, 50), (5, 16, 512, 64), (40, 5, 96, 100), (130, 2, 1024, 200)])
@pytest.mark.parametrize("xt", [BF, HF, F])
def test_linear_groups(csa, T, G, K, M, xt):
    check_linear(csa, T, G, K, M, xt, BF, seed=G)


@pytest.mark.parametrize("pad", [1, 3, 4, 8])
@pytest.mark.parametrize("xt,yt", [(BF, HF), (F, F)])
@pytest.mark.parametrize("T", [2, 24, 80])
def test_linear_strided_and_unaligned_rows(csa, pad, xt, yt, T):
    check_linear(csa, T, 2, 272, 37, xt, yt, pad=pad, seed=pad)


@pytest.mark.parametrize("pad", [0, 3, 8, 24])
@pytest.mark.parametrize("T,G,K,M", [(24, 2, 288, 37), (80, 3, 96, 130), (130, 1, 1056, 70), (300, 2, 160, 129)])
def test_linear_strided_fp16_tokens(csa, pad, T, G, K, M):
    check_linear(csa, T, G, K, M, HF, F, pad=pad, seed=pad)


@pytest.mark.parametrize("T", [5, 8, 9, 16])
@pytest.mark.parametrize("xt,pad", [(BF, 0), (HF, 0), (HF, 3), (F, 0)])
@pytest.mark.parametrize("G,K,M", [(1, 1536, 14001), (3, 1552, 5000)])
def test_linear_some_tokens_of_a_large_matrix(csa, T, xt, pad, G, K, M):
    check_linear(csa, T, G, K, M, xt, BF, pad=pad, seed=T)


@pytest.mark.parametrize("T", [5, 24, 80])
@pytest.mark.parametrize("xt", [BF, HF, F])
def test_linear_tokens_shared_by_the_groups(csa, T, xt):
    x = randn((T, 1, 256), gen(T), xt).expand(T, 3, 256)
    check_linear(csa, T, 3, 256, 50, xt, F, x=x)


@pytest.mark.parametrize("T", [2, 20, 70])
@pytest.mark.parametrize("xt", [BF, F])
def test_linear_wide_range_of_tokens(csa, T, xt):
    """tokens whose values lie far outside fp16's range, each at its own size"""
    g = gen(9)
    x = randn((T, 1, 512), g)
    x *= torch.exp2(torch.linspace(-90, 90, T, device="cuda"))[:, None, None]
    check_linear(csa, T, 1, 512, 40, xt, F, x=x.to(xt), alpha=1.0)


@pytest.mark.parametrize("T", [3, 20, 70])
@pytest.mark.parametrize("xt", [BF, HF, F])
def test_linear_non_finite(csa, T, xt):
    """an infinity and a NaN in x stay in their token's results; a NaN scale in its row's"""
    g = gen(4)
    K, M = 192, 40
    codes, scales = fp4((1, M, K), g)
    x = randn((T, 1, K), g, xt)
    x[0, 0, 5] = math.inf
    x[1, 0, 100] = math.nan
    scales[0, 7, 3] = 0x7F
    got = csa.csa2_linear_fp4(x[:, 0], codes[0], scales[0], out_dtype=F)
    want = torch.einsum("tk,mk->tm", x[:, 0].double(), decode(codes[0], scales[0]))
    size = torch.einsum("tk,mk->tm", x[:, 0].double().abs().nan_to_num(0, 0), decode(codes[0], scales[0]).abs().nan_to_num(0))
    within(got, want, size * ((K + 8) * U + 2.0 ** -21))
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(got[:, 7]).all())


def test_linear_zero_tokens_and_repeatability(csa):
    g = gen(2)
    codes, scales = fp4((100, 256), g)
    assert csa.csa2_linear_fp4(torch.zeros((0, 256), device="cuda"), codes, scales).shape == (0, 100)
    x = randn((19, 256), g)
    a = csa.csa2_linear_fp4(x, codes, scales)
    for _ in range(3):
        assert torch.equal(a, csa.csa2_linear_fp4(x, codes, scales))


def test_linear_takes_weights_just_quantised(csa):
    """the quantiser and the product back to back on one stream, new weights each time"""
    g = gen(6)
    x = randn((4, 512), g, BF)
    codes = torch.empty((256, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((256, 32), dtype=torch.uint8, device="cuda")
    ws = [randn((256, 512), g) for _ in range(6)]
    got = []
    for w in ws:
        csa.csa2_quantize_fp4(w, codes, scales)
        got.append((csa.csa2_linear_fp4(x, codes, scales, out_dtype=F), codes.clone(), scales.clone()))
    for y, c, s in got:
        want = x.double() @ decode(c, s).T
        within(y, want, (x.double().abs() @ decode(c, s).abs().T) * (520 * U + 2.0 ** -21))


# ---------------------------------------------------------------- norm and rotation

def rope64(x, w, pos, f, R, norm, halves, inverse, eps):
    v = x.double()
    D = v.shape[-1]
    if norm:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        if w is not None:
            v = v * w.double()
    size = v.abs().clone()
    if R:
        ang = pos.double()[:, None] * f.double() * (-1 if inverse else 1)
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        t = v[..., D - R:]
        a, b = (t[..., :R // 2], t[..., R // 2:]) if halves else (t[..., 0::2], t[..., 1::2])
        x1, x2, n = a * c - b * s, a * s + b * c, a.abs() + b.abs()
        if halves:
            turned, sz = torch.cat((x1, x2), -1), torch.cat((n, n), -1)
        else:
            turned, sz = torch.stack((x1, x2), -1).flatten(-2), torch.stack((n, n), -1).flatten(-2)
        v = torch.cat((v[..., :D - R], turned), -1)
        size = torch.cat((size[..., :D - R], sz), -1)
    return v, size


def check_rope(csa, T, hq, hk, D, R, xt, yt, norm=True, halves=False, inverse=False, pad=0, far=1 << 20, seed=0, weight=True,
               eps=1e-6, inplace=False, pos=None):
    g = gen(seed)
    f = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / max(R, 1))).float() if R else None
    if pos is None:
        pos = torch.randint(0, far, (T,), generator=g, device="cuda")
    sets = []
    for h in (hq, hk):
        x = randn((T, h, D + pad), g, xt)[..., :D]
        w = 1 + 0.3 * randn((D,), g) if norm and weight else None
        y = x if inplace else torch.full((T, h, D + pad), 7.0, dtype=yt, device="cuda")[..., :D]
        sets.append((x, w, y))
    want = [rope64(x, w, pos, f, R, norm, halves, inverse, eps) for x, w, _ in sets]
    (q, qw, qo), (k, kw, ko) = sets
    csa.csa2_norm_rope(q, pos if R else None, f, qw, k if hk else None, kw if hk else None, eps=eps, norm=norm,
                       halves=halves, inverse=inverse, q_out=qo, k_out=ko if hk else None)
    for (v, size), (_, _, y) in zip(want[:2 if hk else 1], sets):
        # D squares summed in fp32 (half of it after the root), the root, products; the rotation's
        # cosines to 2^-22 and its own roundings
        within(y, v, size * ((D / 2 + 16) * U + 2.0 ** -21))


@pytest.mark.parametrize("xt", [BF, HF, F])
@pytest.mark.parametrize("yt", [BF, HF, F])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_types(csa, xt, yt, halves):
    check_rope(csa, 5, 3, 2, 128, 64, xt, yt, halves=halves)


@pytest.mark.parametrize("D,R", [(2, 2), (4, 0), (6, 4), (64, 64), (80, 80), (80, 40), (96, 32), (100, 10), (130, 6), (192, 64),
                                 (256, 2), (512, 64), (512, 512), (520, 8), (1022, 1022), (1024, 64)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_sizes(csa, D, R, halves):
    check_rope(csa, 3, 5, 1, D, R, BF, F, halves=halves, seed=D + R)
    check_rope(csa, 2, 1, 0, D, R, F, HF, halves=halves, inverse=True, norm=False, seed=D)


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 0), (1, 64, 1), (131, 10, 2), (700, 1, 1), (64, 128, 8), (3000, 3, 0), (257, 64, 1)])
def test_norm_rope_rows(csa, T, hq, hk):
    check_rope(csa, T, hq, hk, 64, 32, BF, BF, seed=T)
    check_rope(csa, T, hq, hk, 512, 64, BF, BF, seed=T + 1)


@pytest.mark.parametrize("pad", [1, 3, 4, 8, 24])
@pytest.mark.parametrize("xt,yt", [(BF, F), (F, BF), (HF, HF)])
def test_norm_rope_strided_rows(csa, pad, xt, yt):
    for halves in (False, True):
        check_rope(csa, 6, 3, 2, 96, 32, xt, yt, pad=pad, halves=halves)


@pytest.mark.parametrize("D,pad", [(512, 0), (80, 3)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_in_place(csa, D, pad, halves):
    check_rope(csa, 40, 9, 1, D, 64, BF, BF, pad=pad, halves=halves, inplace=True)


def test_norm_rope_far_positions(csa):
    pos = torch.tensor([0, 1, (1 << 24) - 1, (1 << 24) + 1, (1 << 31) + 12345, (1 << 36) + 7, -3, -(1 << 30)], device="cuda")
    for halves in (False, True):
        check_rope(csa, 8, 2, 0, 128, 128, F, F, pos=pos, halves=halves)


def test_norm_rope_without_weight_zero_rows_and_back(csa):
    check_rope(csa, 4, 2, 1, 64, 64, BF, F, weight=False, eps=0.0)
    q = torch.zeros((3, 2, 64), device="cuda")
    f = torch.ones(16, device="cuda")
    pos = torch.arange(3, device="cuda")
    assert not csa.csa2_norm_rope(q, pos, f)[0].any()                       # zeros / sqrt(eps)
    assert csa.csa2_norm_rope(q[:0], pos[:0], f)[0].shape == (0, 2, 64)
    x = randn((3, 2, 64), gen(1))
    there, _ = csa.csa2_norm_rope(x, pos * 100000, f, norm=False)
    back, _ = csa.csa2_norm_rope(there, pos * 100000, f, norm=False, inverse=True)
    assert float((back - x).abs().max()) <= 4 * 2.0 ** -21 * float(x.abs().max())


# ---------------------------------------------------------------- attention over every visible entry

def dense64(codes, scales, q, pos, swa, swa_pos0, scale, ratio):
    B, Q, H = q.shape[:3]
    out = torch.zeros((B, Q, H, 512), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    ltol = torch.zeros_like(lse)
    for b in range(B):
        for i in range(Q):
            p = int(pos[b, i])
            n = min(max(0, p - 127) // ratio, codes.shape[1])
            p0 = int(swa_pos0[b]) if swa_pos0 is not None else 0
            lo, hi = max(0, p - 127, p0), min(p, p0 + (swa.shape[1] if swa is not None else 0) - 1)
            L = decode(codes[b, :n], scales[b, :n])
            if hi >= lo:
                L = torch.cat((L, swa[b, lo - p0:hi + 1 - p0].double()))
            if L.shape[0] == 0:
                continue
            q64 = q[b, i].double()
            s = scale * q64 @ L.T
            lse[b, i] = torch.logsumexp(s, -1)
            w = torch.softmax(s, -1)
            out[b, i] = w @ L
            # scores: 512 products summed in fp32; P: half a step of fp16 (2^-11) plus, below 2^-14 of the
            # running max, at most 2^-25 each, where the largest P is at least 1; the sums' own roundings
            ds = float((512 * U * abs(scale) * (q64.abs() @ L.abs().T)).max()) + 2.0 ** -20 * float(s.abs().max())
            rel = 2.0 ** -11 + 2 * ds + L.shape[0] * U
            tol[b, i] = rel * (w @ L.abs()) + L.shape[0] * 2.0 ** -25 * L.abs().amax(0)
            ltol[b, i] = 2 * ds + 2.0 ** -20 * (1 + lse[b, i].abs()) + L.shape[0] * U
    return out, lse, tol, ltol


def dense_case(csa, B, Q, H, cap, pos, ratio=2, swa_len=None, out_dtype=BF, seed=0, q_mul=1.0, win_mul=1.0, splits_check=True):
    g = gen(seed)
    pos = torch.as_tensor(pos, device="cuda", dtype=torch.int64).expand(B, Q).contiguous()
    codes, _ = fp4((B, cap, 512), g)
    scales = torch.randint(0x28, 0x38, (B, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    # what no query of the sequence sees holds NaN
    n_vis = ((pos.amax(1) - 127).clamp_min(0) // ratio).clamp_max(cap)
    scales[torch.arange(cap, device="cuda")[None] >= n_vis[:, None]] = 0x7F
    swa_len = 127 + Q if swa_len is None else swa_len
    pos0 = (pos.amax(1) - (swa_len - 1)).clamp_min(0)
    swa = (randn((B, swa_len, 512), g) * win_mul).to(BF) if swa_len else None
    if swa is not None:
        swa[pos0[:, None] + torch.arange(swa_len, device="cuda") > pos.amax(1)[:, None]] = math.nan
    q = (randn((B, Q, H, 512), g) * q_mul).to(BF)
    cache = csa.Cache.of(codes, scales, ratio=ratio)
    scale = 512 ** -0.5
    out, lse = csa.csa2_dense_attn(cache, q, pos, swa, pos0, scale, out_dtype=out_dtype, want_lse=True)
    ref, rlse, tol, ltol = dense64(codes, scales, q, pos, swa, pos0, scale, ratio)
    within(out, ref, tol)
    within(lse, rlse, ltol)
    return out, lse


@pytest.mark.parametrize("p", [0, 1, 5, 63, 64, 126, 127, 128, 129, 130, 200, 255, 256, 257, 383, 384, 385, 1000])
@pytest.mark.parametrize("ratio", [1, 2])
def test_dense_short_contexts(csa, p, ratio):
    dense_case(csa, 1, 1, 64, 600, p, ratio=ratio, seed=p)


@pytest.mark.parametrize("H", [1, 3, 8, 15, 16, 17, 32, 63, 64, 65, 100, 128])
def test_dense_heads(csa, H):
    dense_case(csa, 2, 2, H, 700, [[900, 901], [40, 41]], ratio=2, seed=H)


@pytest.mark.parametrize("out_dtype", [BF, HF, F])
def test_dense_out_types(csa, out_dtype):
    dense_case(csa, 2, 1, 64, 500, [[700], [500]], ratio=1, out_dtype=out_dtype)


def test_dense_many_splits_and_long_context(csa):
    dense_case(csa, 1, 1, 16, 20011, 20010, ratio=1, seed=1)
    dense_case(csa, 1, 2, 64, 40000, [[70001, 70002]], ratio=2, seed=2)


def test_dense_ragged_batch(csa):
    pos = torch.tensor([[3000, 3001, 3002], [0, 1, 2], [126, 127, 128], [1500, 1501, 1502], [2999, 5, 700]])
    dense_case(csa, 5, 3, 24, 3100, pos, ratio=1, seed=3, swa_len=400)


def test_dense_window_clipped_absent_and_nothing_visible(csa):
    dense_case(csa, 2, 1, 64, 400, [[600], [300]], swa_len=20)          # fewer rows than the window
    out, lse = dense_case(csa, 2, 1, 64, 400, [[600], [50]], swa_len=0)    # none: the second query sees nothing
    assert not out[1].any() and bool((lse[1] == -math.inf).all())
    g = gen(1)
    codes, scales = fp4((1, 8, 512), g)
    out, lse = csa.csa2_dense_attn(csa.Cache.of(codes, scales), randn((1, 1, 4, 512), g, BF),
                                   torch.tensor([[-5]], device="cuda"), None, None, want_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("q_mul,win_mul", [(1e3, 1.0), (2.0 ** -30, 1.0), (1.0, 2.0 ** 20), (1.0, 2.0 ** -20), (4.0, 64.0)])
def test_dense_inputs_far_outside_fp16(csa, q_mul, win_mul):
    dense_case(csa, 2, 1, 64, 300, [[500], [90]], q_mul=q_mul, win_mul=win_mul, seed=7)


def test_dense_rising_scores_rescale_the_output(csa):
    """entries whose scores climb by more than 2^8 from tile to tile: the running max is raised each time"""
    g = gen(11)
    cap, H = 640, 64
    codes = torch.full((1, cap, 256), 0x22, dtype=torch.uint8, device="cuda")       # every value 1
    scales = (0x20 + 2 * (torch.arange(cap, device="cuda") // 64)).to(torch.uint8)[None, :, None].expand(1, cap, 32).contiguous()
    codes[0, :, 0] = torch.randint(0, 256, (cap,), generator=g, device="cuda", dtype=torch.uint8)
    q = torch.full((1, 1, H, 512), 1.0, device="cuda").to(BF)
    q[0, 0, ::2] *= 0.25
    pos = torch.tensor([[cap + 127]], device="cuda")
    cache = csa.Cache.of(codes, scales, ratio=1)
    out, lse = csa.csa2_dense_attn(cache, q, pos, None, None, 1.0, out_dtype=F, want_lse=True)
    ref, rlse, tol, ltol = dense64(codes, scales, q, pos, None, None, 1.0, 1)
    within(out, ref, tol)
    within(lse, rlse, ltol)


def test_dense_equals_sparse_over_all_entries(csa):
    """the selection's attention with every visible entry selected gives the same output (both within 2e-3)"""
    g = gen(5)
    B, H, cap, p = 3, 64, 1000, 1200
    codes, _ = fp4((B, cap, 512), g)
    scales = torch.randint(0x28, 0x38, (B, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    cache = csa.Cache.of(codes, scales, ratio=2)
    q, swa = randn((B, 1, H, 512), g, BF), randn((B, 128, 512), g, BF)
    pos = torch.full((B, 1), p, dtype=torch.int64, device="cuda")
    n = (p - 127) // 2
    idx = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, 1, n).contiguous()
    ref, rl = csa.csa2_sparse_attn(cache, q, pos, idx, swa, p - 127, want_lse=True)
    out, lse = csa.csa2_dense_attn(cache, q, pos, swa, torch.full((B,), p - 127, device="cuda"), out_dtype=F, want_lse=True)
    assert float(((out - ref).abs().amax(-1) / ref.abs().amax(-1)).max()) <= 4e-3
    assert float((lse - rl).abs().max()) <= 1e-4


def test_dense_cache_past_32_bit_offsets(csa):
    """sequences whose rows lie beyond 2^31 bytes of the code plane, and beyond 2^32"""
    g = gen(8)
    B, cap = 3, 6_000_000                                   # 1.5 GB of codes per sequence
    codes = torch.empty((B, cap, 256), dtype=torch.uint8, device="cuda")
    codes[:, :] = torch.randint(0, 256, (1, 1, 256), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((B, cap, 32), 0x30, dtype=torch.uint8, device="cuda")
    n = 300
    for b in range(B):
        codes[b, :n] = torch.randint(0, 256, (n, 256), generator=g, device="cuda", dtype=torch.uint8)
    pos = torch.full((B, 1), n + 127, dtype=torch.int64, device="cuda")
    q = randn((B, 1, 64, 512), g, BF)
    cache = csa.Cache.of(codes, scales, ratio=1)
    out, lse = csa.csa2_dense_attn(cache, q, pos, None, None, out_dtype=F, want_lse=True)
    ref, rlse, tol, ltol = dense64(codes, scales, q, pos, None, None, 512 ** -0.5, 1)
    within(out, ref, tol)
    within(lse, rlse, ltol)


# ---------------------------------------------------------------- together, on streams and in graphs

def test_rows_written_for_the_attention_are_seen_by_it(csa):
    """the norm / the product writes the queries that the sparse attention stages before it waits for its
    predecessor: back to back, with other values each time, the attention sees this call's rows"""
    g = gen(3)
    B, H = 32, 64
    codes, _ = fp4((B, 700, 512), g)
    scales = torch.randint(0x28, 0x38, (B, 700, 32), generator=g, device="cuda", dtype=torch.uint8)
    cache = csa.Cache.of(codes, scales, ratio=2)
    pos = torch.full((B, 1), 1300, dtype=torch.int64, device="cuda")
    idx = torch.arange(512, dtype=torch.int32, device="cuda").expand(B, 1, 512).contiguous()
    f = (10000.0 ** (-torch.arange(0, 64, 2, device="cuda") / 64.0)).float()
    xs = [randn((B, H, 512), g, BF) for _ in range(8)]
    wins = [randn((B, 128, 512), g, BF) for _ in range(8)]
    wc, wsc = fp4((512, 512), g)
    ws = csa.workspace(csa.OP_SPARSE_ATTN, B, 1, H, 512, 700)
    q = torch.empty((B, 1, H, 512), dtype=BF, device="cuda")
    win = torch.empty((B, 128, 512), dtype=BF, device="cuda")

    def step(x, w, out, sync):
        csa.csa2_norm_rope(x, pos[:, 0], f, q_out=q[:, 0], k=w, k_out=win)
        if sync:
            torch.cuda.synchronize()
        csa.csa2_sparse_attn(cache, q, pos, idx, win, 1173, out=out, ws=ws)

    def step2(x, w, out, sync):
        csa.csa2_linear_fp4(x.view(B * H, 512), wc, wsc, 0.05, out=q.view(B * H, 512))
        if sync:
            torch.cuda.synchronize()
        csa.csa2_sparse_attn(cache, q, pos, idx, w, 1173, out=out, ws=ws)

    for fn in (step, step2):
        outs = torch.empty((2, 8, B, 1, H, 512), device="cuda")
        for sync in (1, 0):
            for i in range(8):
                fn(xs[i], wins[i], outs[sync, i], sync)
            torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        gr = torch.cuda.CUDAGraph()
        again = torch.empty_like(outs[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            fn(xs[0], wins[0], again[0], False)
        torch.cuda.current_stream().wait_stream(s)
        with torch.cuda.graph(gr):
            for i in range(8):
                fn(xs[i], wins[i], again[i], False)
        for _ in range(5):
            again.zero_()
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, outs[1])


def test_operators_on_another_stream(csa):
    g = gen(12)
    s = torch.cuda.Stream()
    codes, scales = fp4((300, 256), g)
    x = randn((12, 256), g, BF)
    lat, _ = fp4((1, 400, 512), g)
    cache = csa.Cache.of(lat, torch.full((1, 400, 32), 0x30, dtype=torch.uint8, device="cuda"), ratio=1)
    q, pos = randn((1, 1, 64, 512), g, BF), torch.tensor([[500]], device="cuda")
    torch.cuda.synchronize()
    a = (csa.csa2_linear_fp4(x, codes, scales), csa.csa2_norm_rope(q[0], None, None)[0],
         csa.csa2_dense_attn(cache, q, pos, None, None)[0])
    torch.cuda.synchronize()
    ws = csa.workspace(csa.OP_DENSE_ATTN, 1, 1, 64, 0, 400)
    torch.cuda.synchronize()
    b = (csa.csa2_linear_fp4(x, codes, scales, stream=s), csa.csa2_norm_rope(q[0], None, None, stream=s)[0],
         csa.csa2_dense_attn(cache, q, pos, None, None, ws=ws, stream=s)[0])
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    assert csa.csa2_poll_error(ws, s) == csa.OK


def test_scratch_belongs_to_the_stream_of_the_call(csa):
    """calls without a workspace on a side stream, while the current stream takes and overwrites whatever memory
    is free: their scratch is not handed to it"""
    g = gen(13)
    s = torch.cuda.Stream()
    codes, scales = fp4((2048, 2048), g)
    x = randn((100, 2048), g)
    want = csa.csa2_linear_fp4(x, codes, scales)
    lat, _ = fp4((4, 3000, 512), g)
    cache = csa.Cache.of(lat, torch.full((4, 3000, 32), 0x30, dtype=torch.uint8, device="cuda"), ratio=1)
    q, pos = randn((4, 1, 64, 512), g, BF), torch.full((4, 1), 3100, dtype=torch.int64, device="cuda")
    dense = csa.csa2_dense_attn(cache, q, pos, None, None)[0]
    torch.cuda.synchronize()
    n = csa.csa2_workspace_size(csa.OP_LINEAR_FP4, 100, 1, 2, 0, 2048)
    m = csa.csa2_workspace_size(csa.OP_DENSE_ATTN, 4, 1, 64, 0, 3000)
    outs = [(torch.empty_like(want), torch.empty_like(dense)) for _ in range(20)]
    torch.cuda.synchronize()
    for y, o in outs:
        csa.csa2_linear_fp4(x, codes, scales, out=y, stream=s)
        csa.csa2_dense_attn(cache, q, pos, None, None, out=o, stream=s)
        for size in (n, m):
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    for y, o in outs:
        assert torch.equal(y, want) and torch.equal(o, dense)
