"""A speculative step on a stream of the caller's: the layer's calls and the commit behind them, while the current
stream does other things."""
import pytest
import torch

from test_gpu_operators import fp4, randn
from test_gpu_tree import csa  # noqa: F401
from test_gpu_tree_layer import BF, accepted, draw, make

pytestmark = pytest.mark.gpu


def test_steps_and_commits_on_another_stream(csa):
    """commit takes the stream that enqueue ran on: nothing of it waits for, or runs on, the current one"""
    B, n, steps = 2, 7, 3
    results = []
    for stream in (None, torch.cuda.Stream()):
        layer, g = make(csa, B, n, seed=4)
        layer.committed.copy_(torch.tensor([130, 611], device="cuda"))
        layer.win.copy_(randn(layer.win.shape, g))
        prev, w = randn((B, 512), g, BF), [torch.rand(512, device="cuda", generator=g) for _ in range(2)]
        wik = fp4((128, 512), g)
        drawn = []
        for _ in range(steps):                               # (positions of every step, whatever is accepted)
            draw(layer, g)
            path = accepted(layer, g, 5)
            drawn.append([t.clone() for t in (layer.parent, layer.x, layer.row, path, randn((B, n, 512), g, BF))])
            layer.committed += ((path >= 0).long().sum(1))
            drawn[-1].append(layer.pos.clone())
        layer.committed.copy_(torch.tensor([130, 611], device="cuda"))
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(200_000_000)                # what runs on the current stream runs before all of this
        ys = []
        for parent, x, row, path, h, pos in drawn:
            with torch.cuda.stream(stream):
                layer.parent.copy_(parent), layer.x.copy_(x), layer.row.copy_(row), layer.pos.copy_(pos)
            layer.enqueue(stream=stream)
            layer.commit(path, h, prev=prev, w0=w[0], w1=w[1], wik_codes=wik[0], wik_scales=wik[1], stream=stream)
            with torch.cuda.stream(stream):
                ys.append(layer.y.clone())
        if stream is not None:
            assert not stream.query()                        # (nothing waited for it)
            stream.synchronize()
        torch.cuda.synchronize()
        results.append(ys + [layer.win, layer.committed, prev, layer.cache.lat_codes, layer.cache.ikey_codes, layer.cache.ikey_scales])
    for a, b in zip(*results):
        assert torch.equal(a, b)
