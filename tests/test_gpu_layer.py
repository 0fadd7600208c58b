"""The operators run together as a layer runs them: the projections, the norm with the rotation, the
attention over given indices or over every visible entry, the rotation back and the grouped output
projection, against the same chain in 64 bits on the same FP4 weights and cache."""
import pytest
import torch

from test_gpu_operators import decode, dense64, fp4, gen, randn, rope64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_decode_gb300 as m
    from compressed_sparse_attention_decode_gb300 import build as b
    b.build()
    m.load()
    return m


def make(csa, B, H, r_q, groups, r_out, cap, p, dense, seed):
    from compressed_sparse_attention_decode_gb300.layer import DecodeLayer
    g = gen(seed)
    codes, _ = fp4((B, cap, 512), g)
    scales = torch.randint(0x28, 0x38, (B, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    cache = csa.Cache.of(codes, scales, ratio=2)
    wq, wo = randn((H * 512, r_q), g) * r_q ** -0.5, randn((groups, r_out, H // groups * 512), g) * (H // groups * 512) ** -0.5
    n = (p - 127) // 2
    idx = None if dense else torch.arange(n, dtype=torch.int32, device="cuda").expand(B, 1, n).contiguous()
    layer = DecodeLayer(cache, wq, wo, 1 + 0.2 * randn((512,), g), 1 + 0.2 * randn((512,), g), idx=idx, swa_pos0=p - 127,
                        out_dtype=torch.float32)
    layer.pos.fill_(p)
    layer.win_pos0.fill_(p - 127)
    fill(layer, g)
    return layer, g


def fill(layer, g):
    layer.x.copy_(randn(layer.x.shape, g))
    layer.row.copy_(randn(layer.row.shape, g))
    layer.win.copy_(randn(layer.win.shape, g))


def chain64(layer):
    """the layer in 64 bits, rounding to bf16 where the layer hands bf16 on, and the 2-norm error that its
    roundings leave: each bf16 hand-over half a step (2^-9 at most of a value; rms 2^-9 / sqrt(3) of its
    binade's top), the attention's fp16 weights 2^-11"""
    B, H = layer.B, layer.H
    wq = decode(*layer.wq[:2]) * layer.wq[2]
    q = (layer.x.double() @ wq.T).to(torch.bfloat16).view(B, H, 512)
    q, _ = rope64(q, layer.q_weight, layer.pos, layer.inv_freq, 64, True, False, False, layer.eps)
    k, _ = rope64(layer.row, layer.k_weight, layer.pos, layer.inv_freq, 64, True, False, False, layer.eps)
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    win = layer.win.clone()
    win[:, -1:] = k
    o = dense64(layer.cache.lat_codes, layer.cache.lat_scales, q.view(B, 1, H, 512), layer.pos.view(B, 1), win,
                layer.win_pos0, 512 ** -0.5, 2)[0][:, 0]
    o, _ = rope64(o, None, layer.pos, layer.inv_freq, 64, False, False, True, 0.0)
    wo = decode(*layer.wo[:2]) * layer.wo[2]
    return torch.einsum("bgk,gmk->bgm", o.view(B, layer.groups, -1), wo)


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("B,H,groups", [(1, 64, 16), (20, 64, 8)])
def test_layer_matches_the_chain(csa, B, H, groups, dense):
    layer, g = make(csa, B, H, 256, groups, 96, 600, 900, dense, B)
    for _ in range(2):
        ref = chain64(layer)
        layer.enqueue()
        torch.cuda.synchronize()
        # two bf16 roundings of q (its own 2^-8 half steps reach o through scores of unit size) and two of o:
        # each at most 2^-8 relative, the weights' fp16 2^-11
        assert float((layer.y.double() - ref).norm() / ref.norm()) <= 4 * 2.0 ** -8 + 2.0 ** -11
        fill(layer, g)


def test_layer_graph_replays_new_inputs(csa):
    layer, g = make(csa, 20, 64, 256, 16, 64, 600, 900, True, 3)
    layer.enqueue()
    torch.cuda.synchronize()
    first = layer.y.clone()
    inputs = [t.clone() for t in (layer.x, layer.row, layer.win)]
    layer.capture()
    fill(layer, g)
    layer.run()
    torch.cuda.synchronize()
    assert not torch.equal(layer.y, first)
    for t, v in zip((layer.x, layer.row, layer.win), inputs):
        t.copy_(v)
    layer.run()
    torch.cuda.synchronize()
    assert torch.equal(layer.y, first)
