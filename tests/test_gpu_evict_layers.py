"""Eviction of some layers of a cache, from the first or not: stores, rings, weights and marks are those of
the layers named, with arrays that begin at the call's first layer."""
import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import attend, contents, make_cache  # noqa: E402
from test_gpu_stream import check_evicted, evict, expected_groups, slots_of, small_cache  # noqa: E402


def rows_of(cache, layer, ids, E):
    """Keys and values of the tokens that stay of every unit."""
    k, v, *_ = contents(cache, layer)
    tail = torch.arange(32 * E, k.shape[2])
    out = []
    for b in range(k.shape[0]):
        for h in range(k.shape[1]):
            at = torch.cat([(ids[b, h][:, None].long() * 32 + torch.arange(32)).reshape(-1), tail]).cuda()
            out.append((k[b, h, at], v[b, h, at]))
    return out


@pytest.mark.parametrize("bits", [[4, 4, 4, 4], [2, 16, 4, 16]])
@pytest.mark.parametrize("begin,count", [(3, 1), (1, 2), (0, 1), (2, 2)])
def test_part_of_the_layers(bits, begin, count):
    cache, g = make_cache(22, q_heads=4, kv_heads=2, d=64, n=300, alpha=5, bits=2, layers=4, batch=2, layer_bits=bits)
    n = max(slots_of(cache, i) for i in range(4))
    w = torch.rand(count, 2, 2, n, generator=g, device="cuda")
    small = small_cache(cache, 4)
    stay = torch.full_like(w, -5.0)
    groups = torch.full((count, 2, 2, 4), -7, dtype=torch.int32, device="cuda")
    K.kvc_evict_groups(cache, small, begin, count, 4, 1, n, w, stay, groups)
    torch.cuda.synchronize()
    assert [K.kvc_layer_info_get(small, i)["prefilled"] for i in range(4)] == [int(begin <= i < begin + count) for i in range(4)]
    for i in range(count):
        info = K.kvc_layer_info_get(cache, begin + i)
        exact = info["bits"] == 16
        E = info["window_tokens"] // 32 if exact else info["packed_tokens"] // 32
        ids = expected_groups(w[i].cpu(), E, 4, 1)
        assert torch.equal(groups[i].cpu(), ids)
        k, v, *_ = contents(small, begin + i)
        for u, (kk, vv) in enumerate(rows_of(cache, begin + i, ids, E)):
            assert torch.equal(k[u // 2, u % 2], kk) and torch.equal(v[u // 2, u % 2], vv)
        left = slots_of(cache, begin + i) - E
        rest = w[i, :, :, E:E + left].cpu()
        want = torch.cat([w[i].cpu().gather(-1, ids.long()), rest, torch.zeros(2, 2, n - 4 - left)], -1)
        assert torch.equal(stay[i].cpu(), want)
    # the other layers of the small cache are still free for a call of their own
    others = [i for i in range(4) if not begin <= i < begin + count]
    for i in others:
        K.kvc_evict_groups(cache, small, i, 1, 4, 1, n, w[:1], stay[:1], groups[:1])
    torch.cuda.synchronize()
    for i in range(count):
        ids = expected_groups(w[i].cpu(), 9, 4, 1)      # (nine groups at every precision)
        k, v, *_ = contents(small, begin + i)
        for u, (kk, vv) in enumerate(rows_of(cache, begin + i, ids, 9)):
            assert torch.equal(k[u // 2, u % 2], kk) and torch.equal(v[u // 2, u % 2], vv)


def test_marks_go_with_their_layer():
    """Layer 1 alone holds values past fp16's range, and it is evicted by itself: its units carry the
    marks that the tree attention goes by, and the other layer's, evicted after it, none."""
    g = torch.Generator(device="cuda").manual_seed(23)
    dims = K.make_dims(2, 1, 4, 2, 128, 300, 16, 7, 2, 32, 64, 4)
    cache = K.kvc_cache_create(dims, [300, 300])
    for layer in range(2):
        k = torch.randn(1, 2, 300, 128, generator=g, device="cuda").bfloat16()
        v = torch.randn(1, 2, 300, 128, generator=g, device="cuda").bfloat16()
        if layer == 1:
            v[:, 1, 70:90] = v[:, 1, 70:90].abs() * 30000
        K.kvc_prefill_compress(dims, [300, 300], layer, None, k, v, cache)
    n = slots_of(cache, 0)
    w = torch.arange(n, 0, -1, device="cuda").float().expand(1, 1, 2, n).contiguous()
    small = small_cache(cache, 6)
    for layer in (1, 0):
        stay, groups = torch.empty_like(w), torch.empty(1, 1, 2, 6, dtype=torch.int32, device="cuda")
        K.kvc_evict_groups(cache, small, layer, 1, 6, 0, n, w, stay, groups)
    q = torch.randn(2, 1, 4, 3, 128, generator=g, device="cuda").bfloat16()
    kd = torch.randn(2, 1, 2, 3, 128, generator=g, device="cuda").bfloat16()
    parents = torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    K.kvc_tree_attn(small, 0, 2, 3, parents, q, kd, kd, out)
    for layer in range(2):
        keys, values, *_ = contents(small, layer)
        assert bool((values > 65504).any()) == (layer == 1) and bool(torch.isfinite(values).all())
        for i in range(3):
            qq = q[layer, :, :, i].double().reshape(1, 2, 2, 128)
            kk = torch.cat([keys, kd[layer, :, :, :i + 1].double()], 2)
            vv = torch.cat([values, kd[layer, :, :, :i + 1].double()], 2)
            want, size, av = attend(qq, kk, vv)
            # roundings of keys, values and weights (2^-11 each, drafted ones 2^-8), of the output (2^-8)
            lim = av * (2 * size * 2.0 ** -10 + 2.0 ** -7) + 2.0 ** -8 * want.abs() + 2.0 ** -20 * values.abs().amax()
            assert bool(((out[layer, :, :, i].double().reshape(want.shape) - want).abs() <= lim).all())


def test_all_layers_at_once_are_the_same():
    cache, g = make_cache(24, q_heads=4, kv_heads=2, d=128, n=500, alpha=5, bits=4, layers=3)
    n = slots_of(cache, 0)
    w = torch.rand(3, 1, 2, n, generator=g, device="cuda")
    whole = small_cache(cache, 5)
    stay, groups = evict(cache, whole, 5, 2, w)
    torch.cuda.synchronize()
    check_evicted(cache, whole, 5, 2, w, stay, groups)
    parts = small_cache(cache, 5)
    for begin, count in ((1, 2), (0, 1)):
        s, i = torch.empty_like(w[:count]), torch.empty_like(groups[:count])
        K.kvc_evict_groups(cache, parts, begin, count, 5, 2, n, w[begin:begin + count], s, i)
        assert torch.equal(s, stay[begin:begin + count]) and torch.equal(i, groups[begin:begin + count])
    for layer in range(3):
        a, b = K.kvc_export_layer(whole, layer), K.kvc_export_layer(parts, layer)
        for name in a:
            assert torch.equal(a[name], b[name]), name
