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
