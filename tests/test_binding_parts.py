"""The parts of the binding stand alone: the library is built, loaded and called without its C++ module."""
import os

import pytest
import torch


@pytest.fixture
def built():
    from compressed_sparse_attention_decode_gb300 import build as b
    b.build()
    return b


def test_library_loads_without_the_native_module(built, monkeypatch, tmp_path):
    import compressed_sparse_attention_decode_gb300 as csa
    monkeypatch.setattr(csa, "_lib", None)
    monkeypatch.setattr(csa, "_native", None)
    monkeypatch.setattr(csa, "_HERE", str(tmp_path))          # where _native.so is looked for
    assert csa.load().csa2_abi_version() == 200
    assert csa.csa2_workspace_size(csa.OP_SPARSE_ATTN, 1, 1, 64, 512, 1000) > 0
    for call in (lambda: csa.csa2_linear_fp4(None, None, None), lambda: csa.csa2_norm_rope(None, None, None),
                 lambda: csa.csa2_dense_attn(csa.Cache.of(torch.zeros(1, 1, 256), torch.zeros(1, 1, 32)), None, None, None, None)):
        with pytest.raises(RuntimeError, match="_native.so is not built"):
            call()


def test_library_is_built_where_the_native_module_fails(built, monkeypatch, tmp_path):
    def fails():
        raise RuntimeError("no compiler for it")
    monkeypatch.setattr(built, "_binding", fails)
    monkeypatch.setattr(built, "LIB", str(tmp_path / "libcsa2.so"))
    with pytest.raises(RuntimeError, match="no compiler for it"):
        built.build()
    assert os.path.exists(built.LIB)


def test_native_module_is_built_again_for_another_pytorch(built, monkeypatch, tmp_path):
    """its build is kept while sources, Python and PyTorch stay what they were, and made again for others"""
    calls = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def compiler(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done

    monkeypatch.setattr(built, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(built, "BUILD", str(tmp_path))
    monkeypatch.setattr(built.subprocess, "run", compiler)
    for version, made in [("2.9.1", 1), ("2.9.1", 1), ("2.11.0", 2), ("2.11.0", 2), ("2.9.1", 3)]:
        monkeypatch.setattr(torch, "__version__", version)
        built._binding()
        assert len(calls) == made


def test_binding_refuses_memory_that_is_not_there_or_shared(built):
    import compressed_sparse_attention_decode_gb300 as csa
    u8 = dict(dtype=torch.uint8)
    x, c, s = torch.zeros(20, 64), torch.zeros(5, 32, **u8), torch.zeros(5, 4, **u8)
    cache = csa.Cache.of(torch.zeros(2, 8, 256, **u8), torch.zeros(2, 8, 32, **u8))
    q, p = torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int64)
    one = torch.zeros(1, **u8)
    for ws in (one.expand(1 << 24), torch.zeros(64, **u8)[::2]):
        with pytest.raises(ValueError, match="ws: contiguous"):
            csa.csa2_linear_fp4(x, c, s, ws=ws)
        with pytest.raises(ValueError, match="ws: contiguous"):
            csa.csa2_dense_attn(cache, q, p, None, None, ws=ws)
    with pytest.raises(ValueError, match="apart"):
        csa.csa2_linear_fp4(x, c, s, out=torch.zeros(1, 5).expand(20, 5))
    with pytest.raises(ValueError, match="apart"):
        csa.csa2_linear_fp4(torch.zeros(3, 2, 64), c.expand(2, 5, 32).contiguous(), s.expand(2, 5, 4).contiguous(),
                            out=torch.zeros(3, 1, 5).expand(3, 2, 5))
    h = torch.zeros(3, 4, 64)
    for kw in (dict(q_out=torch.zeros(3, 1, 64).expand(3, 4, 64)), dict(k=h, k_out=torch.zeros(1, 4, 64).expand(3, 4, 64))):
        with pytest.raises(ValueError, match="apart"):
            csa.csa2_norm_rope(h, None, None, **kw)
    # one row may have any stride
    with pytest.raises(ValueError, match="GPU"):
        csa.csa2_linear_fp4(x[:1], c, s, out=torch.zeros(1, 5).expand(1, 5))
