"""The operators of a speculative step refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def csa():
    from compressed_sparse_attention_decode_gb300 import build as b
    import compressed_sparse_attention_decode_gb300 as m
    b.build()
    m.load()
    return m


P = ctypes.c_void_p(256)


def at(n):
    return ctypes.c_void_p(n)


def struct(csa, ik=256, batch=2, cap=1000, d_idx=128, ratio=2):
    return csa._CacheStruct(256, 256, ik, ik, batch, cap, 512, d_idx, ratio)


def tree(csa, cache=None, q=P, n_q=4, heads=64, pos=P, parent=P, draft=P, idx=None, k=-1, swa=P, pos0=P, swa_len=128, scale=0.04,
         out=P, ot=0, lse=None, ws=P, ws_bytes=1 << 40):
    c = struct(csa) if cache is None else cache
    return csa.load().csa2_tree_attn(ctypes.byref(c) if c else None, q, n_q, heads, pos, parent, draft, idx, k, swa, pos0, swa_len,
                                     scale, out, ot, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(cache=False), dict(q=None), dict(pos=None), dict(parent=None), dict(draft=None), dict(out=None),
                                dict(n_q=0), dict(n_q=129), dict(heads=0), dict(heads=129), dict(k=-2), dict(k=2049, idx=P),
                                dict(k=4), dict(swa_len=-1), dict(swa=None), dict(scale=float("nan")), dict(ot=3),
                                dict(q=at(264)), dict(draft=at(264)), dict(swa=at(264)), dict(out=at(264)), dict(pos=at(260)),
                                dict(pos0=at(260)), dict(parent=at(258)), dict(idx=at(258), k=4), dict(lse=at(258))])
def test_tree_refusals(csa, kw):
    assert tree(csa, **kw) == csa.ERR_INVALID_ARG


def test_tree_cache_and_workspace(csa):
    assert tree(csa, cache=struct(csa, batch=65536)) == csa.ERR_INVALID_ARG
    assert tree(csa, cache=struct(csa, ratio=3)) == csa.ERR_INVALID_ARG
    assert tree(csa, cache=csa._CacheStruct(256, 256, 0, 0, 2, 1000, 256, 128, 2)) == csa.ERR_UNSUPPORTED
    for k in (csa.EVERY_ENTRY, 0, 1, 512):
        need = csa.csa2_workspace_size(csa.OP_TREE_ATTN, 2, 4, 64, k, 1000)
        assert need > 0
        for ws in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=at(264))):
            if k != 0 or "ws_bytes" not in ws:
                assert tree(csa, k=k, idx=P, **ws) == csa.ERR_WORKSPACE
    # with k = 0 a workspace serves both forms
    assert csa.csa2_workspace_size(csa.OP_TREE_ATTN, 2, 4, 64, 0, 1000) >= csa.csa2_workspace_size(csa.OP_TREE_ATTN, 2, 4, 64, -1, 1000)
    for bad in [(2, 129, 64, 0, 1000), (2, 4, 0, 0, 1000), (2, 4, 129, 0, 1000), (2, 4, 64, -2, 1000), (2, 4, 64, 2049, 1000),
                (2, 4, 64, 0, 0), (0, 4, 64, 0, 1000)]:
        assert csa.csa2_workspace_size(csa.OP_TREE_ATTN, *bad) == 0
    # bounded: the largest trees need no more than some hundred MB
    assert csa.csa2_workspace_size(csa.OP_TREE_ATTN, 64, 128, 128, -1, 1 << 20) < 400 << 20


def append(csa, cache=None, rows=P, n_rows=8, path=P, n_path=4, pos0=P, prev=P, prev_out=P, w0=P, w1=P, wc=None, ws=None):
    c = struct(csa) if cache is None else cache
    return csa.load().csa2_cache_append(ctypes.byref(c) if c else None, rows, n_rows, path, n_path, pos0, prev, prev_out, w0, w1, wc,
                                        ws, None)


@pytest.mark.parametrize("kw", [dict(cache=False), dict(rows=None), dict(rows=at(264)), dict(n_rows=-1), dict(n_path=-1),
                                dict(path=None, n_path=9), dict(path=at(258)), dict(pos0=None), dict(pos0=at(260)), dict(prev=None),
                                dict(prev=at(264)), dict(prev_out=at(264)), dict(w0=None), dict(w1=None), dict(w0=at(264)),
                                dict(w1=at(264)), dict(wc=P), dict(ws=P), dict(wc=at(264), ws=P), dict(wc=P, ws=at(258))])
def test_append_refusals(csa, kw):
    assert append(csa, **kw) == csa.ERR_INVALID_ARG


def test_append_cache_checks(csa):
    assert append(csa, cache=struct(csa, ratio=4)) == csa.ERR_INVALID_ARG
    assert append(csa, cache=struct(csa, batch=65536)) == csa.ERR_INVALID_ARG
    assert append(csa, cache=struct(csa, ik=0), wc=P, ws=P) == csa.ERR_INVALID_ARG          # no planes for the keys
    assert append(csa, cache=struct(csa, d_idx=96)) == csa.ERR_UNSUPPORTED


def read(csa, cache=None, what=0, idx=None, first=0, n=10, out=P, ot=0):
    c = struct(csa) if cache is None else cache
    return csa.load().csa2_cache_read(ctypes.byref(c) if c else None, what, idx, first, n, out, ot, None)


@pytest.mark.parametrize("kw", [dict(cache=False), dict(what=2), dict(what=-1), dict(idx=at(258)), dict(first=-1), dict(n=-1),
                                dict(n=1001), dict(first=1000, n=1), dict(first=1 << 62, n=1 << 62), dict(n=1 << 62, idx=P),
                                dict(out=None), dict(out=at(264)), dict(ot=3)])
def test_read_refusals(csa, kw):
    assert read(csa, **kw) == csa.ERR_INVALID_ARG


def test_read_of_keys_needs_their_planes(csa):
    assert read(csa, cache=struct(csa, ik=0), what=csa.INDEXER_KEYS) == csa.ERR_INVALID_ARG


def test_empty_calls_enqueue_nothing(csa):
    lib = csa.load()
    n = lib.csa2_launch_count()
    assert read(csa, n=0, out=None) == csa.OK and read(csa, idx=P, n=0) == csa.OK and read(csa, first=1000, n=0) == csa.OK
    assert append(csa, n_path=0) == csa.OK                                     # the carried row stays where it is
    assert append(csa, cache=struct(csa, ratio=1), n_rows=0, rows=None, n_path=0, prev=None, w0=None, w1=None) == csa.OK
    assert lib.csa2_launch_count() == n


def test_binding_checks_shapes_and_types(csa):
    u8, bf = dict(dtype=torch.uint8), dict(dtype=torch.bfloat16)
    refused = lambda what: pytest.raises(ValueError, match=what)
    cache = csa.Cache.of(torch.zeros(2, 8, 256, **u8), torch.zeros(2, 8, 32, **u8), torch.zeros(2, 8, 64, **u8), torch.zeros(2, 8, 8, **u8))
    bare = csa.Cache.of(cache.lat_codes, cache.lat_scales)
    a = dict(q=torch.zeros(2, 3, 4, 512, **bf), q_pos=torch.zeros(2, 3, dtype=torch.int64), parent=torch.zeros(2, 3, dtype=torch.int32),
             draft=torch.zeros(2, 3, 512, **bf), swa=torch.zeros(2, 5, 512, **bf), swa_pos0=torch.zeros(2, dtype=torch.int64))
    with refused("GPU"):
        csa.csa2_tree_attn(cache, **a)
    with refused("GPU"):
        csa.csa2_tree_attn(cache, **a, idx=torch.zeros(2, 3, 0, dtype=torch.int32), want_lse=True)
    for bad in [dict(q=a["q"].float()), dict(q=a["q"][:1]), dict(q=a["q"].transpose(1, 2)), dict(q_pos=a["q_pos"].int()),
                dict(q_pos=a["q_pos"][:, :2]), dict(parent=a["q_pos"]), dict(parent=a["parent"].T), dict(draft=a["draft"][:, :2]),
                dict(draft=a["draft"].half()), dict(swa=a["swa"].float()), dict(swa_pos0=a["swa_pos0"].int()),
                dict(idx=torch.zeros(2, 3, 4, dtype=torch.int64)), dict(idx=torch.zeros(2, 2, 4, dtype=torch.int32)),
                dict(out=torch.zeros(2, 3, 4, 256)), dict(lse=torch.zeros(2, 3)), dict(ws=torch.zeros(64, **u8)[::2])]:
        with refused("contiguous"):
            csa.csa2_tree_attn(cache, **{**a, **bad})
    with refused("bf16, fp16 or fp32"):
        csa.csa2_tree_attn(cache, **a, out_dtype=torch.float64)
    b = dict(rows=torch.zeros(2, 3, 512, **bf), pos0=torch.zeros(2, dtype=torch.int64), path=torch.zeros(2, 4, dtype=torch.int32),
             prev=torch.zeros(2, 512, **bf), prev_out=torch.zeros(2, 512, **bf), w0=torch.zeros(512), w1=torch.zeros(512),
             wik_codes=torch.zeros(128, 256, **u8), wik_scales=torch.zeros(128, 32, **u8))
    with refused("GPU"):
        csa.csa2_cache_append(cache, **b)
    for bad in [dict(rows=b["rows"].float()), dict(rows=b["rows"][:1]), dict(rows=b["rows"][:, ::2]), dict(pos0=b["pos0"].int()),
                dict(path=b["path"].long()), dict(path=b["path"][:1]), dict(prev=b["prev"][:1]), dict(prev_out=b["prev"].half()),
                dict(w0=torch.zeros(256)), dict(w1=torch.zeros(512, dtype=torch.float64)), dict(wik_codes=torch.zeros(64, 256, **u8)),
                dict(wik_scales=torch.zeros(128, 16, **u8))]:
        with refused("contiguous"):
            csa.csa2_cache_append(cache, **{**b, **bad})
    with refused("both or neither"):
        csa.csa2_cache_append(cache, **{**b, "wik_scales": None})
    with refused("indexer keys"):
        csa.csa2_cache_append(bare, **b)
    idx = torch.zeros(2, 3, 4, dtype=torch.int32)
    with refused("GPU"):
        csa.csa2_cache_read(cache, idx, keys=True)
    with refused("GPU"):
        csa.csa2_cache_read(bare, first=8)
    for kw in [dict(idx=idx.long()), dict(idx=idx[:1]), dict(idx=idx.transpose(1, 2)), dict(idx=idx, out=torch.zeros(2, 3, 512)),
               dict(count=3, out=torch.zeros(2, 3, 512)[..., ::2])]:
        with refused("contiguous"):
            csa.csa2_cache_read(cache, **kw)
    with refused("indexer keys"):
        csa.csa2_cache_read(bare, keys=True)
    with refused("of idx, or"):
        csa.csa2_cache_read(cache, idx, count=3)
    for kw in [dict(first=-1), dict(first=9), dict(first=2, count=7), dict(count=-1)]:
        with refused("inside the cache"):
            csa.csa2_cache_read(cache, **kw)


def test_calls_need_the_native_module(csa, monkeypatch, tmp_path):
    monkeypatch.setattr(csa, "_native", None)
    monkeypatch.setattr(csa, "_HERE", str(tmp_path))
    cache = csa.Cache.of(torch.zeros(1, 1, 256), torch.zeros(1, 1, 32))
    for call in (lambda: csa.csa2_tree_attn(cache, None, None, None, None, None, None), lambda: csa.csa2_cache_append(cache, None, None),
                 lambda: csa.csa2_cache_read(cache)):
        with pytest.raises(RuntimeError, match="_native.so is not built"):
            call()
