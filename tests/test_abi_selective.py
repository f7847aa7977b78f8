"""Host-side validation of the calls that read listed groups or drafted trees, without a GPU:
a null cache handle is rejected before anything else, and the library and the binding export
the three calls."""
import ctypes

import pytest

K = pytest.importorskip("kv_cache_compression_snapkv_gb300")


def test_null_cache_is_rejected():
    P = ctypes.c_void_p(256)   # never dereferenced: the null cache is rejected first
    lib = K._lib
    assert lib.kvc_select_groups(None, 0, 1, P, 4, P, None) == 1
    assert lib.kvc_decode_groups(None, 0, 1, P, 4, P, P, None) == 1
    assert lib.kvc_tree_attn(None, 0, 1, 4, P, P, P, P, P, None) == 1


@pytest.mark.parametrize("name", ["kvc_select_groups", "kvc_decode_groups", "kvc_tree_attn"])
def test_exported(name):
    assert name in K.exported_symbols() and name in K.__all__
    assert callable(getattr(K, name))
