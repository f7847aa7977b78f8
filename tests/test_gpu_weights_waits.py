"""kvc_decode_weights where staging waits give up: what a (layer, sequence, kv head) received is added
whole or not at all, so that a running sum never takes what an earlier call left in the scratch."""
import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import make_cache  # noqa: E402

CASES = [
    dict(q_heads=4, kv_heads=2, d=64, n=300, alpha=16, bits=4, batch=3),                 # weights in the same launch
    dict(q_heads=1, kv_heads=1, d=128, n=300, alpha=16, bits=2),                         # one unit over several CTAs
    dict(q_heads=4, kv_heads=2, d=64, n=3000, alpha=16, bits=2),                         # weights in a second one
    dict(q_heads=16, kv_heads=2, d=64, n=2500, alpha=5, bits=4, batch=2, layers=2),
    dict(q_heads=8, kv_heads=8, d=64, n=75, alpha=3, bits=2, batch=200, layers=3),       # a warp holds several units
    dict(q_heads=2, kv_heads=2, d=64, n=1100, alpha=3, bits=16, batch=60),
]


def slots_of(cache):
    i = K.kvc_layer_info_get(cache, 0)
    return i["packed_tokens"] // 32 + -(-i["window_tokens"] // 32)


def call(cache, q, before, after):
    D = cache.dims
    out = torch.empty(q.shape, device="cuda")
    K.kvc_decode_weights(cache, 0, D.n_layers, q, before.shape[-1], before, after, out)
    return after


def gave_up(cache):
    try:
        K.kvc_check_device(cache)
    except K.KvcError as e:
        assert e.status == 7
        return True
    return False


@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_sums_survive(case):
    cache, g = make_cache(31, **case)
    D = cache.dims
    q, other = ((spread * torch.randn(D.n_layers, D.batch, D.n_q_heads, D.head_dim, generator=g,
                                      device="cuda")).bfloat16() for spread in (1.0, 3.0))
    before = torch.rand(D.n_layers, D.batch, D.n_kv_heads, slots_of(cache) + 2, generator=g, device="cuda")
    want = call(cache, q, before, torch.empty_like(before))
    call(cache, other, before, torch.empty_like(before))       # what the scratch holds now is of other queries
    assert not gave_up(cache)
    for limit in (0, 1, 4, 20):
        K.kvc_set_wait_limit(cache, limit)
        after = call(cache, q, before, torch.full_like(before, float("nan")))
        failed = gave_up(cache)
        K.kvc_set_wait_limit(cache, 1 << 20)
        whole, none = (after == want).all(-1), (after == before).all(-1)
        assert bool((whole | none).all()), limit
        assert failed or bool(whole.all())
        if limit == 0:
            assert failed and bool(none.all())
        call(cache, other, before, after)
    # in place: the sum of a generation is still there, and the step can be made again
    total = before.clone()
    K.kvc_set_wait_limit(cache, 0)
    call(cache, q, total, total)
    assert gave_up(cache) and torch.equal(total, before)
    K.kvc_set_wait_limit(cache, -1)
    assert torch.equal(call(cache, q, total, total), want)
    assert not gave_up(cache)
