"""csa2_sparse_attn's window position: what is refused on the host."""
import ctypes

import pytest


@pytest.mark.parametrize("swa_pos0", [-1, -(1 << 63) + 1])
def test_negative_window_positions_are_refused(swa_pos0):
    import compressed_sparse_attention_decode_gb300 as csa
    from compressed_sparse_attention_decode_gb300 import build as b
    b.build()
    p = ctypes.c_void_p(256)
    cache = csa._CacheStruct(256, 256, 0, 0, 1, 1000, 512, 128, 2)
    assert csa.load().csa2_sparse_attn(ctypes.byref(cache), p, 1, 64, p, p, 64, p, swa_pos0, 128, 0.04, p, None, p, 1 << 40,
                                       None) == csa.ERR_INVALID_ARG
