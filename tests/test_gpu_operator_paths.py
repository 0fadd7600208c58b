"""Calls of the operators around the attention that reach their less trodden paths: many short shares a
block and several passes of the dense attention, against the same 64-bit forms as test_gpu_operators."""
import pytest
import torch

from test_gpu_operators import BF, HF, F, U, csa, decode, dense_case, fp4, gen, randn, within  # noqa: F401

pytestmark = pytest.mark.gpu


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
