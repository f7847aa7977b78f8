"""Host-side validation of the calls that bound a long generation's attention, without a GPU: a null
cache handle is rejected before anything else, and the library and the binding export them."""
import ctypes

import pytest

K = pytest.importorskip("kv_cache_compression_snapkv_gb300")


def test_null_cache_is_rejected():
    P = ctypes.c_void_p(256)   # never dereferenced: the null cache is rejected first
    lib = K._lib
    assert lib.kvc_prefill_window(None, 0, 4, 16, P, P, P, P, None) == 1
    assert lib.kvc_decode_window(None, 0, 1, 4, 16, P, P, None) == 1
    assert lib.kvc_decode_weights(None, 0, 1, P, 4, P, P, P, None) == 1
    assert lib.kvc_evict_groups(None, P, 0, 1, 4, 0, 4, P, P, P, None) == 1


@pytest.mark.parametrize("name", ["kvc_prefill_window", "kvc_decode_window", "kvc_decode_weights",
                                  "kvc_evict_groups"])
def test_exported(name):
    assert name in K.exported_symbols() and name in K.__all__
    assert callable(getattr(K, name))
