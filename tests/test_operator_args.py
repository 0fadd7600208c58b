"""The operators around the attention refuse bad arguments on the host, before any CUDA call."""
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


def linear(lib, x=P, xt=0, n_tok=1, groups=1, n_in=64, n_out=8, codes=P, scales=P, alpha=1.0, y=P, yt=0, ws=None,
           ws_bytes=0):
    return lib.csa2_linear_fp4(x, xt, n_in, n_in, n_tok, groups, n_in, n_out, codes, scales, alpha, y, yt, n_out, n_out, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(xt=3), dict(yt=-1), dict(n_tok=-1), dict(groups=0), dict(groups=65536),
                                dict(n_in=24), dict(n_in=-16), dict(n_in=(1 << 24) + 16), dict(n_out=-1), dict(codes=None), dict(scales=None),
                                dict(codes=ctypes.c_void_p(264)), dict(scales=ctypes.c_void_p(264)), dict(alpha=float("nan")), dict(alpha=float("inf")),
                                dict(y=None), dict(x=ctypes.c_void_p(257)), dict(x=ctypes.c_void_p(258), xt=2),
                                dict(y=ctypes.c_void_p(258), yt=2)])
def test_linear_refusals(csa, kw):
    assert linear(csa.load(), **kw) == csa.ERR_INVALID_ARG


def test_linear_workspace(csa):
    size = lambda T, K, xt: csa.csa2_workspace_size(csa.OP_LINEAR_FP4, T, 1, xt, 0, K)
    assert size(1, 4096, 0) == 0 and size(16, 8192, 1) == 0
    for T, K, xt in [(17, 64, 0), (300, 4096, 2), (100, 0, 1), (1, 1 << 20, 0)]:
        need = size(T, K, xt)
        assert need > 0
        for kw in [dict(), dict(ws=P, ws_bytes=need - 1), dict(ws=ctypes.c_void_p(264), ws_bytes=need)]:
            assert linear(csa.load(), n_tok=T, n_in=K, xt=xt, **kw) == csa.ERR_WORKSPACE


def test_empty_calls_enqueue_nothing(csa):
    lib = csa.load()
    n = lib.csa2_launch_count()
    assert linear(lib, n_tok=0) == csa.OK and linear(lib, n_out=0) == csa.OK
    assert rope(lib, n_tok=0) == csa.OK
    assert rope(lib, q=rows(csa, heads=0)) == csa.OK
    assert lib.csa2_launch_count() == n


def rows(csa, x=256, y=256, w=0, heads=4, d=64):
    return csa._HeadRows(x, y, w, heads * d, d, heads * d, d, heads)


def rope(lib, q="default", k=None, xt=0, yt=0, n_tok=2, d=64, rot=32, pos=P, inv=P, eps=1e-6, flags=0):
    import compressed_sparse_attention_decode_gb300 as csa
    q = rows(csa) if q == "default" else q
    r = lambda v: None if v is None else ctypes.byref(v)
    return lib.csa2_norm_rope(r(q), r(k), xt, yt, n_tok, d, rot, pos, inv, eps, flags, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(xt=3), dict(yt=9), dict(n_tok=-1), dict(d=0), dict(d=63), dict(d=1026),
                                dict(rot=66), dict(rot=31), dict(rot=-2), dict(pos=None), dict(inv=None),
                                dict(pos=ctypes.c_void_p(260)), dict(inv=ctypes.c_void_p(258)), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(flags=8)])
def test_norm_rope_refusals(csa, kw):
    assert rope(csa.load(), **kw) == csa.ERR_INVALID_ARG


def test_norm_rope_refuses_bad_row_sets(csa):
    lib = csa.load()
    bad = [rows(csa, x=0), rows(csa, y=0), rows(csa, heads=-1), rows(csa, w=257), rows(csa, x=257), rows(csa, heads=1 << 21)]
    for r in bad:
        assert rope(lib, q=r) == csa.ERR_INVALID_ARG
        assert rope(lib, k=r) == csa.ERR_INVALID_ARG
    assert rope(lib, q=rows(csa, x=258), xt=2) == csa.ERR_INVALID_ARG
    assert rope(lib, q=rows(csa, w=256), flags=csa.ROPE_NO_NORM) == csa.ERR_INVALID_ARG   # a weight without the norm


def dense(lib, cache="default", q=P, n_q=1, heads=64, pos=P, swa=P, pos0=P, swa_len=128, scale=0.04, out=P, ot=0, lse=None,
          ws=P, ws_bytes=1 << 40):
    import compressed_sparse_attention_decode_gb300 as csa
    c = csa._CacheStruct(256, 256, 0, 0, 2, 1000, 512, 128, 2) if cache == "default" else cache
    return lib.csa2_dense_attn(ctypes.byref(c) if c is not None else None, q, n_q, heads, pos, swa, pos0, swa_len, scale,
                               out, ot, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(cache=None), dict(q=None), dict(pos=None), dict(out=None), dict(n_q=0), dict(heads=0),
                                dict(heads=129), dict(swa_len=-1), dict(swa=None), dict(scale=float("nan")), dict(ot=3),
                                dict(q=ctypes.c_void_p(264)), dict(swa=ctypes.c_void_p(264)), dict(out=ctypes.c_void_p(264)),
                                dict(pos=ctypes.c_void_p(260)), dict(pos0=ctypes.c_void_p(260)), dict(lse=ctypes.c_void_p(258))])
def test_dense_refusals(csa, kw):
    assert dense(csa.load(), **kw) == csa.ERR_INVALID_ARG


def test_dense_workspace_and_cache_checks(csa):
    lib = csa.load()
    need = csa.csa2_workspace_size(csa.OP_DENSE_ATTN, 2, 1, 64, 0, 1000)
    assert need > 0
    assert dense(lib, ws_bytes=need - 1) == csa.ERR_WORKSPACE
    assert dense(lib, ws=None) == csa.ERR_WORKSPACE
    assert dense(lib, ws=ctypes.c_void_p(264)) == csa.ERR_WORKSPACE
    assert dense(lib, cache=csa._CacheStruct(256, 256, 0, 0, 2, 1000, 256, 128, 2)) == csa.ERR_UNSUPPORTED
    assert dense(lib, cache=csa._CacheStruct(256, 256, 0, 0, 2, 1000, 512, 128, 3)) == csa.ERR_INVALID_ARG
    assert csa.csa2_workspace_size(csa.OP_DENSE_ATTN, 2, 1, 0, 0, 1000) == 0
    # the shares of a pass are bounded: a chunk of many queries needs no more than a few hundred MB
    assert csa.csa2_workspace_size(csa.OP_DENSE_ATTN, 1, 8192, 64, 0, 65536) < 400 << 20


def test_binding_checks_shapes_and_types(csa):
    u8 = dict(dtype=torch.uint8)
    x, c, s = torch.zeros(3, 64), torch.zeros(5, 32, **u8), torch.zeros(5, 4, **u8)
    refused = lambda what: pytest.raises(ValueError, match=what)
    with refused("GPU"):                       # all is well but for the device
        csa.csa2_linear_fp4(x, c, s)
    with refused("GPU"):
        csa.csa2_linear_fp4(x[:, None].expand(3, 2, 64), c.expand(2, 5, 32).contiguous(), s.expand(2, 5, 4).contiguous())
    for bad in [(x.double(), c, s), (x, c[:, :16], s), (x, c, s[:, :2]), (x, c.int(), s), (x.T.contiguous().T, c, s),
                (x[:, :40], c, s), (torch.zeros(3, 2, 64), c, s)]:
        with refused("n_in|uint8|bf16|contiguous"):
            csa.csa2_linear_fp4(*bad)
    with refused("out"):
        csa.csa2_linear_fp4(x, c, s, out=torch.zeros(3, 6))
    with refused("out"):
        csa.csa2_linear_fp4(x, c, s, out=torch.zeros(3, 5), out_dtype=torch.float16)
    with refused("tensor"):
        csa.csa2_linear_fp4([1.0], c, s)
    with pytest.raises(TypeError):
        csa.csa2_linear_fp4(x, c, s, "alpha")
    with refused("codes"):
        csa.csa2_linear_fp4(torch.zeros(3, 2, 64), torch.zeros(3, 5, 32, **u8), torch.zeros(3, 5, 4, **u8))
    q, pos, f = torch.zeros(3, 4, 64), torch.zeros(3, dtype=torch.int64), torch.zeros(16)
    with refused("GPU"):
        csa.csa2_norm_rope(q, pos, f, k=torch.zeros(3, 1, 64), q_weight=torch.zeros(64))
    for kw in [dict(q=q, pos=pos.int(), inv_freq=f), dict(q=q, pos=pos[:2], inv_freq=f), dict(q=q, pos=None, inv_freq=f),
               dict(q=q, pos=pos, inv_freq=f.double()), dict(q=q.transpose(1, 2), pos=pos, inv_freq=f),
               dict(q=q, pos=pos, inv_freq=f, q_weight=torch.zeros(32)), dict(q=q, pos=pos, inv_freq=f, k=q.half()),
               dict(q=q, pos=pos, inv_freq=f, k=torch.zeros(2, 4, 64)), dict(q=q.double(), pos=pos, inv_freq=f)]:
        with refused("contiguous|bf16|k has|a head set"):
            csa.csa2_norm_rope(**kw)
    cache = csa.Cache.of(torch.zeros(2, 8, 256, **u8), torch.zeros(2, 8, 32, **u8))
    bq, p = torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int64)
    with refused("GPU"):
        csa.csa2_dense_attn(cache, bq, p, torch.zeros(2, 4, 512, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64))
    for a in [(bq.float(), p, None, None), (bq[:1], p, None, None), (bq, p.int(), None, None), (bq, p[:1], None, None),
              (bq, p, torch.zeros(2, 4, 512), None), (bq, p, None, torch.zeros(2, dtype=torch.int32))]:
        with refused("contiguous"):
            csa.csa2_dense_attn(cache, *a)
