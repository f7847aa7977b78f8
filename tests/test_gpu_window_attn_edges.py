"""Prompt attention over a sliding window where something is wrong: waits that give up."""
import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from test_gpu_window_attn import make, new_cache, prompt  # noqa: E402


def test_a_wait_that_gives_up_is_an_earlier_calls():
    """The call that launched the kernel returns as it would have (its packing does not look at the error
    word in between), and the error is reported once."""
    for n in (600, 3000, 20000):
        q, k, v = make(11, 8, 2, 128, n)
        cache = new_cache(q, k, 64)
        want = prompt(cache, q, k, v, 4, 96)
        for _ in range(5):
            K.kvc_cache_reset(cache)
            K.kvc_set_wait_limit(cache, 0)
            prompt(cache, q, k, v, 4, 96)
            assert K.kvc_layer_info_get(cache, 0)["prefilled"] == 1
            torch.cuda.synchronize()
            with pytest.raises(K.KvcError) as e:
                K.kvc_check_device(cache)
            assert e.value.status == 7
            K.kvc_check_device(cache)
            K.kvc_set_wait_limit(cache, -1)
            K.kvc_cache_reset(cache)
            assert torch.equal(prompt(cache, q, k, v, 4, 96), want)
            K.kvc_check_device(cache)
