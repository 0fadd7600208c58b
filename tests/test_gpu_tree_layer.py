"""The operators of a speculative step run together, as a layer runs them: trees drafted, an accepted path committed to the
window and the cache, the next trees over what was committed; against the same chain in 64 bits, against the layer that
decodes one token at a time, and captured and replayed."""
import pytest
import torch

from test_gpu_operators import decode, fp4, gen, randn, rope64
from test_gpu_tree import chains, csa, depths, random_parents, tree64  # noqa: F401

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(csa, B, n, H=16, r_q=128, groups=4, r_out=40, cap=700, ratio=2, seed=0, idx=None, kind="TreeLayer"):
    from compressed_sparse_attention_decode_gb300 import layer as L
    g = gen(seed)
    codes, _ = fp4((B, cap, 512), g)
    scales = torch.randint(0x28, 0x38, (B, cap, 32), generator=g, device="cuda", dtype=torch.uint8)
    cache = csa.Cache.of(codes, scales, *fp4((B, cap, 128), g), ratio=ratio)
    a = (cache, randn((H * 512, r_q), g) * r_q ** -0.5, randn((groups, r_out, H // groups * 512), g) * (H // groups * 512) ** -0.5,
         1 + 0.2 * randn((512,), g), 1 + 0.2 * randn((512,), g))
    if kind == "TreeLayer":
        return L.TreeLayer(*a, n, idx=idx, out_dtype=torch.float32), g
    return L.DecodeLayer(*a, idx=idx, out_dtype=torch.float32), g


def draw(layer, g):
    """new trees over what is committed"""
    layer.parent.copy_(random_parents(layer.B, layer.n, g))
    layer.pos.copy_(layer.committed[:, None] + depths(layer.parent))
    layer.x.copy_(randn(layer.x.shape, g))
    layer.row.copy_(randn(layer.row.shape, g))


def chain64(layer):
    """the layer in 64 bits, rounding to bf16 where the layer hands bf16 on"""
    B, n, H = layer.B, layer.n, layer.H
    T = B * n
    q = (layer.x.double().view(T, -1) @ (decode(*layer.wq[:2]) * layer.wq[2]).T).to(BF).view(T, H, 512)
    q, _ = rope64(q, layer.q_weight, layer.pos.view(T), layer.inv_freq, 64, True, False, False, layer.eps)
    k, _ = rope64(layer.row.view(T, 1, 512), layer.k_weight, layer.pos.view(T), layer.inv_freq, 64, True, False, False, layer.eps)
    o = tree64(layer.cache.lat_codes, layer.cache.lat_scales, q.to(BF).view(B, n, H, 512), layer.pos, layer.parent,
               k.to(BF).view(B, n, 512), layer.win, layer.committed - 128, layer.idx, 512 ** -0.5, layer.cache.ratio)[0]
    o, _ = rope64(o.to(BF).view(T, H, 512), None, layer.pos.view(T), layer.inv_freq, 64, False, False, True, 0.0)
    y = torch.einsum("bgk,gmk->bgm", o.to(BF).double().view(T, layer.groups, -1), decode(*layer.wo[:2]) * layer.wo[2])
    return y.view(B, n, layer.groups, -1)


def close(y, ref):
    # bf16 roundings of q (twice), of the output (twice, both sides rounding on their own): each at most 2^-8 of a value; the
    # attention's fp16 weights 2^-11
    assert float((y.double() - ref).norm() / ref.norm()) <= 6 * 2.0 ** -8 + 2.0 ** -11


def accepted(layer, g, m):
    """a path from the root down: of each sequence the chain of a drawn node, cut to m steps, its end empty"""
    path = torch.full((layer.B, m), -1, dtype=torch.int32)
    for b, parent in enumerate(layer.parent.tolist()):
        node = int(torch.randint(0, layer.n, (1,), generator=g, device="cuda"))
        chain = chains(parent)[node][::-1][:m]
        path[b, :len(chain)] = torch.tensor(chain, dtype=torch.int32)
    return path.cuda()


@pytest.mark.parametrize("ratio", [1, 2])
@pytest.mark.parametrize("lists", [False, True])
def test_steps_of_trees_and_commits(csa, ratio, lists):
    B, n = 3, 9
    idx = torch.full((B, n, 64), -1, dtype=torch.int32, device="cuda") if lists else None
    layer, g = make(csa, B, n, ratio=ratio, idx=idx)
    layer.committed.copy_(torch.tensor([0, 131, 600], device="cuda"))
    layer.win.copy_(randn(layer.win.shape, g))
    cache = layer.cache
    prev = randn((B, 512), g, BF)
    w = [torch.rand(512, device="cuda", generator=g) for _ in range(2)] if ratio == 2 else [None, None]
    wik = fp4((128, 512), g)
    wik = (wik[0], wik[1] & 0x7F)                    # (csa2_quantize_fp4 writes no negative scale)
    for step in range(5):
        draw(layer, g)
        if lists:
            seen = ((layer.committed - 127).clamp_min(0) // ratio).clamp_min(1)
            layer.idx.copy_((torch.rand(layer.idx.shape, device="cuda", generator=g) * seen[:, None, None]).int())
            layer.idx[..., 40:] = -1
        ref = chain64(layer)
        layer.enqueue()
        torch.cuda.synchronize()
        close(layer.y, ref)
        # the accepted path into the window and the cache, and what the cache then holds
        path, h = accepted(layer, g, 5), randn((B, n, 512), g, BF)
        before, win, draft, p0 = [t.clone() for t in (cache.lat_codes, cache.lat_scales)], layer.win.clone(), layer.draft.clone(), layer.committed.clone()
        carried = prev.clone()
        layer.commit(path, h, prev=prev if ratio == 2 else None, w0=w[0], w1=w[1], wik_codes=wik[0], wik_scales=wik[1])
        rows = csa.csa2_cache_read(cache, out_dtype=torch.float32)
        keys = csa.csa2_cache_read(cache, keys=True, out_dtype=torch.float32)
        for b in range(B):
            take = [j for j in path[b].tolist() if j >= 0]
            assert torch.equal(layer.win[b], torch.cat((win[b], draft[b, take]))[-128:])
            assert int(layer.committed[b]) == int(p0[b]) + len(take)
            r, p = h[b, take], int(p0[b])
            if ratio == 2:
                r = torch.cat((carried[b:b + 1], r))
                assert torch.equal(prev[b], r[-1])
                p, r = (p, r[1:]) if p % 2 == 0 else (p - 1, r)
                r = r[:len(r) // 2 * 2].double()
                r = (w[1].double() * r[1::2] + (w[0].double() * r[0::2]).float().double()).float()
            else:
                r = r.float()
            e = p // ratio
            want = decode(*csa.csa2_quantize_fp4(r.contiguous())).float() if len(r) else r
            assert torch.equal(rows[b, e:e + len(r)], want)
            if len(r):
                # the sum is exact in 64 bits (products of 2^-20, below 2^33): the key as csa2_quantize_fp4 makes it
                k = csa.csa2_quantize_fp4((want.double() @ decode(*wik).T).float().contiguous())
                assert torch.equal(keys[b, e:e + len(r)], decode(*k).float())
            same = torch.ones(700, dtype=torch.bool, device="cuda")
            same[e:e + len(r)] = False
            assert torch.equal(cache.lat_codes[b, same], before[0][b, same]) and torch.equal(cache.lat_scales[b, same], before[1][b, same])


@pytest.mark.parametrize("lists", [False, True])
def test_a_single_node_is_a_decode_step(csa, lists):
    """a tree of one node and the layer of one token, the same weights and window: outputs within both's roundings"""
    B = 4
    idx = torch.arange(64, dtype=torch.int32, device="cuda").expand(B, 1, 64).contiguous() if lists else None
    tree, g = make(csa, B, 1, H=64, groups=8, idx=idx, seed=5)
    one, _ = make(csa, B, 1, H=64, groups=8, idx=idx, seed=5, kind="DecodeLayer")
    pos = torch.tensor([300, 500, 901, 1200], device="cuda")
    win = randn((B, 128, 512), g, BF)
    x, row = randn(tree.x.shape, g, BF), randn((B, 1, 512), g, BF)
    tree.x.copy_(x)
    tree.row.copy_(row)
    tree.parent.fill_(-1)
    tree.pos.copy_(pos[:, None])
    tree.committed.copy_(pos)
    tree.win.copy_(win)
    one.x.copy_(x[:, 0])
    one.row.copy_(row)
    one.pos.copy_(pos)
    one.win[:, :-1] = win[:, 1:]                     # its last row is the token's own
    tree.enqueue()
    one.enqueue()
    torch.cuda.synchronize()
    # two bf16 roundings of the output, an fp32 one in between for the layer with indices
    assert float((tree.y[:, 0] - one.y).norm() / one.y.norm()) <= 3 * 2.0 ** -8


def test_captured_steps_follow_new_trees(csa):
    """one captured step, replayed over new trees, positions and windows: as the eager calls"""
    layer, g = make(csa, 3, 12, seed=2)
    layer.committed.copy_(torch.tensor([5, 400, 777], device="cuda"))
    layer.win.copy_(randn(layer.win.shape, g))
    draw(layer, g)
    layer.capture()
    for _ in range(4):
        draw(layer, g)
        layer.run()
        got = layer.y.clone()
        layer.enqueue()
        torch.cuda.synchronize()
        assert torch.equal(got, layer.y)
        layer.commit(accepted(layer, g, 4))
    assert csa.csa2_poll_error(layer.ws) == csa.OK


def test_operators_chained_on_a_stream(csa):
    """append, tree attention over what was appended, read-back: one stream, nothing in between, many times; against the
    same calls with a wait after each"""
    g = gen(9)
    B, n, H, cap = 4, 6, 64, 500
    w = [torch.rand(512, device="cuda", generator=g) for _ in range(2)]
    inputs = []
    for i in range(6):
        base = torch.tensor([400, 401, 650, 899], device="cuda") + i
        parent = random_parents(B, n, g)
        inputs.append(dict(rows=randn((B, 5, 512), g, BF), pos0=base - 5, prev=randn((B, 512), g, BF), parent=parent,
                           pos=base[:, None] + depths(parent), draft=randn((B, n, 512), g, BF), swa=randn((B, 128, 512), g, BF),
                           swa_pos0=base - 128, q=randn((B, n, H, 512), g, BF),
                           idx=torch.arange(200, 264, dtype=torch.int32, device="cuda").expand(B, n, 64).contiguous()))

    def run(sync):
        cache = csa.Cache(B, cap, 128, ratio=2)
        cache.lat_codes.fill_(0x21)
        cache.lat_scales.fill_(0x30)
        outs = []
        wait = torch.cuda.synchronize if sync else (lambda: None)
        for x in inputs:
            csa.csa2_cache_append(cache, x["rows"], x["pos0"], prev=x["prev"], prev_out=torch.empty_like(x["prev"]), w0=w[0], w1=w[1])
            wait()
            for idx in (None, x["idx"]):
                outs.append(csa.csa2_tree_attn(cache, x["q"], x["pos"], x["parent"], x["draft"], x["swa"], x["swa_pos0"], idx=idx)[0])
                wait()
            outs.append(csa.csa2_cache_read(cache))
            wait()
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
