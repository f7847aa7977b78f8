"""Prompt attention over a sliding window where something goes wrong: waits that give up."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

WAITS = """
import torch
import kv_cache_compression_snapkv_gb300 as K
from test_gpu_window_attn import make, new_cache, prompt

q, k, v = make(11, 8, 2, 128, 3000)
cache = new_cache(q, k, 64)
want = prompt(cache, q, k, v, 4, 96)
for _ in range(3):
    K.kvc_cache_reset(cache)
    K.kvc_set_wait_limit(cache, 0)
    prompt(cache, q, k, v, 4, 96)
    assert K.kvc_layer_info_get(cache, 0)["prefilled"] == 1
    try:
        K.kvc_check_device(cache)
        raise SystemExit("no error was reported")
    except K.KvcError as e:
        assert e.status == 7
    K.kvc_check_device(cache)
    K.kvc_set_wait_limit(cache, -1)
    K.kvc_cache_reset(cache)
    assert torch.equal(prompt(cache, q, k, v, 4, 96), want)
    K.kvc_check_device(cache)
"""


@pytest.mark.parametrize("blocking", ["0", "1"])
def test_a_wait_that_gives_up_is_an_earlier_calls(blocking):
    """The call that launched the kernel returns as it would have, however early the error word is there
    (with blocking launches it is before the call's second one), and the error is reported once."""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([os.path.dirname(here), here])
    r = subprocess.run([sys.executable, "-c", WAITS], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, CUDA_LAUNCH_BLOCKING=blocking, PYTHONPATH=path))
    assert r.returncode == 0, r.stdout + r.stderr
