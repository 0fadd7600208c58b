"""A layer's step at one position after the other: the window is where the position puts it, with indices
and without, eagerly and in one captured graph."""
import types

import pytest
import torch

from test_gpu_layer import chain64, csa, fill  # noqa: F401
from test_gpu_operators import fp4, gen, randn

pytestmark = pytest.mark.gpu

K = 512                                          # indices per query: every visible entry up to position 1,152


def make(csa, B, with_indices, seed=0):
    """a layer as its class makes it, nothing set by hand but the inputs"""
    from compressed_sparse_attention_decode_gb300.layer import DecodeLayer
    g = gen(seed)
    codes, _ = fp4((B, 600, 512), g)
    scales = torch.randint(0x28, 0x38, (B, 600, 32), generator=g, device="cuda", dtype=torch.uint8)
    idx = torch.full((B, 1, K), -1, dtype=torch.int32, device="cuda") if with_indices else None
    layer = DecodeLayer(csa.Cache.of(codes, scales, ratio=2), randn((64 * 512, 256), g) / 16, randn((8, 96, 4096), g) / 64,
                        1 + 0.2 * randn((512,), g), 1 + 0.2 * randn((512,), g), idx=idx, out_dtype=torch.float32)
    return layer, g


def advance(layer, pos, g):
    """the inputs of a step at these positions"""
    fill(layer, g)
    layer.pos.copy_(pos)
    if layer.idx is not None:
        j = torch.arange(K, dtype=torch.int32, device="cuda").expand(layer.B, 1, K)
        layer.idx.copy_(torch.where(j < ((pos - 127).clamp_min(0) // 2)[:, None, None], j, -1))


def check(layer, run):
    view = types.SimpleNamespace(**{k: getattr(layer, k) for k in ("B", "H", "x", "row", "pos", "win", "wq", "wo", "q_weight",
                                                                   "k_weight", "inv_freq", "eps", "cache", "groups")})
    view.win_pos0 = layer.pos - 127              # the last row of win is this token's
    ref = chain64(view)
    run()
    torch.cuda.synchronize()
    # the roundings of test_gpu_layer's chain
    assert float((layer.y.double() - ref).norm() / ref.norm()) <= 4 * 2.0 ** -8 + 2.0 ** -11


def positions(B, step):
    """of every sequence: around the window's length, past it, moving on by one, and all different"""
    p = [0, 5, 126, 127, 128, 255, 256, 900, 901, 902, 1040, 60][step]
    return torch.full((B,), p, device="cuda") if step % 2 == 0 else (p + 37 * torch.arange(B, device="cuda")) % 1150


@pytest.mark.parametrize("with_indices", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_layer_follows_the_position(csa, with_indices, captured):
    layer, g = make(csa, 5, with_indices)
    if captured:
        advance(layer, positions(5, 8), g)
        layer.capture()
    for step in range(12):
        advance(layer, positions(5, step), g)
        check(layer, layer.run)


@pytest.mark.parametrize("H", [3, 32, 64, 128])          # CUDA cores, tiles with a join, the pair of blocks
@pytest.mark.parametrize("n_q", [1, 3])
def test_sparse_window_at_the_query(csa, H, n_q):
    """each sequence's window ends at its own last query: as one call a sequence with that position given"""
    g = gen(H)
    B = 6
    codes, _ = fp4((B, 300, 512), g)
    scales = torch.randint(0x28, 0x38, (B, 300, 32), generator=g, device="cuda", dtype=torch.uint8)
    idx = torch.randint(-1, 300, (B, n_q, 64), generator=g, device="cuda", dtype=torch.int32)
    q, swa = randn((B, n_q, H, 512), g, torch.bfloat16), randn((B, 130, 512), g, torch.bfloat16)
    last = torch.tensor([2, 60, 127, 129, 131, 1 << 33], device="cuda")
    pos = last[:, None] + torch.arange(1 - n_q, 1, device="cuda")
    out, lse = csa.csa2_sparse_attn(csa.Cache.of(codes, scales), q, pos, idx, swa, csa.WINDOW_AT_QUERY, want_lse=True)
    for b, p in enumerate(last.tolist()):
        s = slice(b, b + 1)
        first = max(0, p - 129)                          # rows of negative positions are not there
        one, l1 = csa.csa2_sparse_attn(csa.Cache.of(codes[s], scales[s]), q[s], pos[s], idx[s],
                                       swa[s, 129 - (p - first):].contiguous(), first, want_lse=True)
        assert torch.equal(out[s], one) and torch.equal(lse[s], l1)
