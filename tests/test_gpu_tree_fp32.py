"""What fp32 outputs of drafted trees keep, against 64-bit sums of the same keys.  The queries have one value and the scores
are of few bits, so that the roundings of weights and sums are what is left:
    a sum of 48 tensor-core steps loses a unit in its last place a step at most, 2^-23 of what it has reached: of values of one sign
    24.5 x 2^-23 = 2.9e-6 of it where it grows evenly, whatever the number of keys;
    weights and their exponentials 2^-22 each: 3.4e-6 in all;
    2^-32 of the largest weight of a run of 384 keys for each of them (half of fp16's smallest step, that weight being 2^7 at least),
    with index lists 2^-35 of the largest of all (2^10 at least)."""
import pytest
import torch

from test_gpu_operators import BF, F, csa, decode, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def inputs(entries, N, H, k, g, window):
    """positive values to 3; dims 0 and 1 (which the scores are made of) 0 in the entries"""
    codes = torch.randint(0, 256, (1, entries, 256), generator=g, device="cuda", dtype=torch.uint8) & 0x77
    codes[..., 0] = 0
    scales = torch.full((1, entries, 32), 0x30, device="cuda", dtype=torch.uint8)
    x = dict(q=torch.zeros((1, N, H, 512), device="cuda", dtype=BF), q_pos=torch.full((1, N), entries + 127, device="cuda"),
             parent=torch.full((1, N), -1, device="cuda", dtype=torch.int32),
             draft=torch.rand((1, N, 512), generator=g, device="cuda").to(BF),
             swa=torch.rand((1, 127, 512), generator=g, device="cuda").to(BF) if window else None,
             swa_pos0=torch.full((1,), entries, device="cuda") if window else None,
             idx=None if k is None else torch.randint(0, entries, (1, N, k), generator=g, device="cuda", dtype=torch.int32))
    return codes, scales, x


def reference(codes, scales, x, i, scale=1.0, part=100_000):
    """node i's w @ L and lse in 64 bits"""
    q = x["q"][0, i].double()
    rows = x["draft"][0, i:i + 1].double()
    if x["swa"] is not None:
        rows = torch.cat((x["swa"][0, -127:].double(), rows))
    w = torch.exp(scale * q @ rows.T)
    s, o = w.sum(1), w @ rows
    e = torch.arange(codes.shape[1], device="cuda") if x["idx"] is None else x["idx"][0, i].long()
    for at in range(0, e.numel(), part):
        L = decode(codes[0, e[at:at + part]], scales[0, e[at:at + part]])
        w = torch.exp(scale * q @ L.T)
        s, o = s + w.sum(1), o + w @ L
    return o / s[:, None], s.log()


@pytest.mark.parametrize("entries,k", [(300, None), (20_000, None), (200_000, None), (1_000_000, None), (3000, 512), (3000, 2048)])
@pytest.mark.parametrize("window", [False, True])
def test_fp32_outputs_keep_their_bits_at_any_length(csa, entries, k, window):
    """scores to 1 in size, every key counts"""
    g = gen(entries)
    N, H = 5, 13
    codes, scales, x = inputs(entries, N, H, k, g, window)
    codes[..., 0] = torch.randint(0, 256, (1, entries), generator=g, device="cuda", dtype=torch.uint8)
    x["q"][..., 0] = (torch.rand((1, N, H), generator=g, device="cuda") / 3).to(BF)
    out, lse = csa.csa2_tree_attn(csa.Cache.of(codes, scales, ratio=1), scale=1.0, out_dtype=F, want_lse=True, **x)
    for i in range(N):
        ref, rlse = reference(codes, scales, x, i)
        err = (out[0, i].double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert float(err.max()) <= 3.4e-6, (i, float(err.max()))
        assert float((lse[0, i].double() - rlse).abs().max()) <= 1e-6 * (1 + float(rlse.abs().max()))


@pytest.mark.parametrize("entries,k", [(200_000, None), (1_000_000, None), (3000, 2048)])
@pytest.mark.parametrize("nats", [16.0, 20.0, 22.25, 23.0])
def test_fp32_outputs_with_one_large_key_and_a_long_tail(csa, entries, k, nats):
    """the draft is `nats` above every entry and has no values but the one that its score is made of: the output is the
    tail's, of weights that are small numbers beside the largest"""
    g = gen(int(nats))
    N, H = 128, 128 if k is None else 64                     # (many rows, so that the work is not split within the keys)
    codes, scales, x = inputs(entries, N, H, k, g, False)
    x["q"][..., 0] = nats / 16                               # (few bits)
    x["draft"].zero_()
    x["draft"][..., 0] = 16.0
    out, lse = csa.csa2_tree_attn(csa.Cache.of(codes, scales, ratio=1), scale=1.0, out_dtype=F, want_lse=True, **x)
    for i in (0, 77, 127):
        ref, rlse = reference(codes, scales, x, i)
        # the draft's run has 383 entries, of values up to 3; other runs' largest weights are the tail's own.  Of the tail: the sums,
        # and the draft's exponent near 2^5, rounded to 2^-19 and its factor to 2^-24 (0.7 of either for a weight)
        tol = (383 * 2.0 ** -32 if k is None else k * 2.0 ** -35) * 3 + 7e-6 * ref.abs()
        over = ((out[0, i].double() - ref).abs() / tol)[:, 1:]
        assert float(over.max()) <= 1, (i, float(over.max()), float(ref[:, 1:].abs().max()))
        assert float((lse[0, i].double() - rlse).abs().max()) <= 1e-6 * (1 + float(rlse.abs().max()))
