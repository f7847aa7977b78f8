"""Decode attention over the first and the last cached tokens, decode attention that accumulates what
the groups receive, and eviction by that weight, against plain 64-bit forms over the exported cache."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import U32, attend, contents, make_cache, sum_bound  # noqa: E402

CASES = [
    dict(q_heads=4, kv_heads=4, d=64, n=528, alpha=16, bits=2),
    dict(q_heads=8, kv_heads=2, d=128, n=1000, alpha=32, bits=2),
    dict(q_heads=8, kv_heads=1, d=128, n=2500, alpha=0, bits=4),
    dict(q_heads=4, kv_heads=2, d=64, n=777, alpha=9, bits=4, batch=3, layers=2),
    dict(q_heads=2, kv_heads=2, d=128, n=40, alpha=0, bits=2, batch=2),        # one group
    dict(q_heads=2, kv_heads=2, d=128, n=1, alpha=0, bits=4),                  # one token
    dict(q_heads=4, kv_heads=1, d=128, n=320, alpha=0, bits=2),                # an empty window
    dict(q_heads=4, kv_heads=2, d=128, n=300, alpha=16, bits=2, appended=90),  # flushed groups
    dict(q_heads=4, kv_heads=2, d=64, n=300, alpha=16, bits=2, layers=3, layer_bits=[2, 16, 4]),
    dict(q_heads=16, kv_heads=2, d=64, n=333, alpha=3, bits=16, batch=2),      # every token exact
    dict(q_heads=1, kv_heads=1, d=64, n=40000, alpha=5, bits=2),               # many groups
]
IDS = [f"{i}" for i in range(len(CASES))]


def queries(cache, g, spread=1.0):
    D = cache.dims
    return (spread * torch.randn(D.n_layers, D.batch, D.n_q_heads, D.head_dim, generator=g,
                                 device="cuda")).bfloat16()


def window(cache, q, sinks, last, stream=None):
    D = cache.dims
    out = torch.full((D.n_layers, D.batch, D.n_q_heads, D.head_dim), float("nan"), device="cuda")
    K.kvc_decode_window(cache, 0, D.n_layers, sinks, last, q, out, stream)
    return out


def slots_of(cache, layer):
    i = K.kvc_layer_info_get(cache, layer)
    return i["packed_tokens"] // 32 + -(-i["window_tokens"] // 32)


def weights(cache, q, before, stream=None):
    D = cache.dims
    out = torch.full((D.n_layers, D.batch, D.n_q_heads, D.head_dim), float("nan"), device="cuda")
    after = torch.full_like(before, float("nan"))
    K.kvc_decode_weights(cache, 0, D.n_layers, q, before.shape[-1], before, after, out, stream)
    return out, after


def check(cache, q, out, seen_of):
    """`out` against the 64-bit form over the tokens seen_of(T). Weights carry three fp16 parts, codes
    one product of two roundings: a logit off by e moves a weight by e of itself, so the output by
    twice that of the weighted |v|; the parts of a weight add 2^-22, sums U32 per term in order."""
    D = cache.dims
    g = D.n_q_heads // D.n_kv_heads
    for layer in range(D.n_layers):
        keys, values, *_ = contents(cache, layer)
        T = keys.shape[2]
        seen = seen_of(T).cuda()
        qd = q[layer].double().reshape(D.batch, D.n_kv_heads, g, D.head_dim)
        if not bool(seen.any()):
            assert bool((out[layer] == 0).all())
            continue
        want, size, av = attend(qd, keys[:, :, seen], values[:, :, seen])
        got = out[layer].double().reshape(want.shape)
        assert bool(torch.isfinite(got).all())
        # queries times scales as fp16 pairs: 2^-22 of each product; fp32 sums of them
        e = sum_bound(size, D.head_dim, 2.0 ** -22)
        lim = av * (2 * e + 2.0 ** -20) + values[:, :, seen].abs().amax((2, 3), keepdim=True) * 2.0 ** -20
        assert bool(((got - want).abs() <= lim).all()), ((got - want).abs() / lim).max()


RANGES = [(0, 1), (4, 100), (45, 77), (32, 64), (1, 1 << 30), (200, 33), (0, 16), (2 ** 31 - 1, 1), (4, 311), (290, 5)]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_window_matches(case):
    cache, g = make_cache(3, **case)
    q = queries(cache, g)
    for s, w in RANGES:
        out = window(cache, q, s, w)
        torch.cuda.synchronize()

        def seen(T):
            t = torch.arange(T)
            return (t < s) | (t >= T - w)
        check(cache, q, out, seen)
    K.kvc_check_device(cache)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_weights_match(case):
    cache, g = make_cache(4, **case)
    D = cache.dims
    q = queries(cache, g, 1.5)
    n = max(slots_of(cache, i) for i in range(D.n_layers)) + 3
    before = torch.rand(D.n_layers, D.batch, D.n_kv_heads, n, generator=g, device="cuda")
    out, after = weights(cache, q, before)
    torch.cuda.synchronize()
    check(cache, q, out, lambda T: torch.ones(T, dtype=torch.bool))
    gq = D.n_q_heads // D.n_kv_heads
    for layer in range(D.n_layers):
        keys, *_ = contents(cache, layer)
        qd = q[layer].double().reshape(D.batch, D.n_kv_heads, gq, D.head_dim)
        x = qd @ keys.transpose(-1, -2) / math.sqrt(D.head_dim)
        p = torch.softmax(x, -1).sum(2)
        p = torch.nn.functional.pad(p, (0, n * 32 - p.shape[-1])).unflatten(-1, (n, 32)).sum(-1)
        size = (qd.abs() @ keys.abs().transpose(-1, -2)).amax((-1, -2)) / math.sqrt(D.head_dim)
        # logits as in check(), twice (a weight and the sum); exp2 to 2^-22; the addition to `before`
        e = 2 * sum_bound(size, D.head_dim, 2.0 ** -22)[..., None] + 2.0 ** -20
        lim = p * e + U32 * (before[layer].double() + p) + 1e-30
        got = after[layer].double() - before[layer].double()
        assert bool(((got - p).abs() <= lim).all()), ((got - p).abs() / lim).max()
        # slots past the last are handed on
        assert torch.equal(after[layer, ..., slots_of(cache, layer):], before[layer, ..., slots_of(cache, layer):])


def test_weights_in_place_and_again():
    cache, g = make_cache(5, q_heads=8, kv_heads=2, n=3000, bits=2)
    q = queries(cache, g)
    n = slots_of(cache, 0)
    before = torch.rand(1, 1, 2, n, generator=g, device="cuda")
    out, after = weights(cache, q, before)
    out2, after2 = weights(cache, q, before)
    assert torch.equal(out, out2) and torch.equal(after, after2)
    K.kvc_decode_weights(cache, 0, 1, q, n, before, before, out)
    assert torch.equal(before, after)


def test_hidden_values_do_not_reach_the_output():
    """Infinities and NaN in hidden values and window keys: the rows equal those of a cache without."""
    def made(bad):
        g = torch.Generator(device="cuda").manual_seed(9)
        dims = K.make_dims(1, 1, 4, 2, 128, 300, 16, 7, 4, 32, 64, 4)
        k = torch.randn(1, 2, 300, 128, generator=g, device="cuda").bfloat16()
        v = torch.randn(1, 2, 300, 128, generator=g, device="cuda").bfloat16()
        if bad:
            v[:, :, 5:200] = float("nan")
            v[:, :, 40:60] = float("inf")
            v[:, :, 200:206] = -float("inf")
            if bad > 1:
                v[:, :, 289] = float("nan")
        cache = K.kvc_prefill_compress(dims, [300], 0, None, k, v)
        return cache, queries(cache, g)
    for s, w, bad in ((5, 94, 1), (5, 10, 2), (3, 1, 2)):
        outs = []
        for b in (0, bad):
            cache, q = made(b)
            outs.append(window(cache, q, s, w))
        assert bool(torch.isfinite(outs[1]).all())
        assert torch.equal(*outs)
    assert bool(torch.isnan(window(made(2)[0], q, 5, 94)).all())    # token 289 is seen


def test_hidden_keys_of_an_exact_cache():
    g = torch.Generator(device="cuda").manual_seed(9)
    dims = K.make_dims(1, 1, 4, 2, 64, 100, 16, 7, 16, 32, 128, 4)
    k = torch.randn(1, 2, 100, 64, generator=g, device="cuda").bfloat16()
    v = torch.randn(1, 2, 100, 64, generator=g, device="cuda").bfloat16()
    outs = []
    for bad in (False, True):
        if bad:
            k[:, :, 7:81] = float("nan")
            v[:, :, 7:81] = float("inf")
        cache = K.kvc_prefill_compress(dims, [100], 0, None, k, v)
        q = (torch.ones(1, 1, 4, 64, device="cuda") / 8).bfloat16()
        outs.append(window(cache, q, 7, 19))
    assert bool(torch.isfinite(outs[1]).all()) and torch.equal(*outs)


def test_large_queries_and_far_scales():
    """Queries past fp16's range, and keys whose scale is (kWideScale): as 64 bits. Keys whose minimum
    itself passes 65,504 are stored with an infinite zero-point: what sees them is not finite."""
    for scale, spread in ((1.0, 3e5), (1e4, 1e-3), (3e4, 1e-3)):
        cache, g = make_cache(6, q_heads=8, kv_heads=2, d=128, n=400, alpha=16, bits=2, scale=scale)
        q = queries(cache, g, spread)
        n = slots_of(cache, 0)
        out, after = weights(cache, q, torch.zeros(1, 1, 2, n, device="cuda"))
        if scale == 3e4:
            assert bool(torch.isinf(K.kvc_export_layer(cache, 0)["k_zero"]).any((0, 2, 3)).all())
            assert not bool(torch.isfinite(out).any())
            continue
        assert bool(torch.isfinite(out).all() & torch.isfinite(after).all())
        check(cache, q, out, lambda T: torch.ones(T, dtype=torch.bool))
        check(cache, q, window(cache, q, 4, 90), lambda T: (torch.arange(T) < 4) | (torch.arange(T) >= T - 90))


def test_empty_layers():
    """A layer that holds no token: the output is 0 and the weights are handed on."""
    dims = K.make_dims(2, 1, 2, 2, 64, 8, 0, 7, 2, 32, 64, 4)
    cache = K.kvc_cache_create(dims, [8, 8])
    k = torch.randn(1, 2, 8, 64, device="cuda").bfloat16()
    kept = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvc_prefill_selected(cache, 0, kept, 0, k, k)
    K.kvc_prefill_compress(dims, [8, 8], 1, None, k, k, cache)
    q = torch.randn(2, 1, 2, 64, device="cuda").bfloat16()
    before = torch.rand(2, 1, 2, 2, device="cuda")
    out, after = weights(cache, q, before)
    assert bool((out[0] == 0).all()) and bool((out[1] != 0).any())
    assert torch.equal(after[0], before[0])
    assert abs(float((after[1] - before[1]).sum()) - 2) < 1e-5
    assert bool((window(cache, q, 1, 1)[0] == 0).all())
    one = torch.full((1, 1, 2, 64), 7.0, device="cuda")
    K.kvc_decode_weights(cache, 0, 1, q[:1].contiguous(), 2, before, after, one)   # nothing but the empty one
    assert bool((one == 0).all()) and torch.equal(after[0], before[0])


# ------------------------------------------------------------------------------------ eviction
def small_cache(cache, keep, max_new=4, n_extra=0):
    D = cache.dims
    n = 32 * (keep + 1) + 32 + n_extra
    window_len = D.window_len if D.bits != 16 else (n + max_new + 31) // 32 * 32
    dims = K.make_dims(D.n_layers, D.batch, D.n_q_heads, D.n_kv_heads, D.head_dim, n, 0, 1, D.bits,
                       32, window_len, max_new)
    bits = [K.kvc_layer_info_get(cache, i)["bits"] for i in range(D.n_layers)]
    return K.kvc_cache_create_layers(dims, [n] * D.n_layers, bits)


def evict(cache, small, keep, recent, w, stream=None):
    D = cache.dims
    stay = torch.full_like(w, -5.0)
    groups = torch.full((D.n_layers, D.batch, D.n_kv_heads, keep), -7, dtype=torch.int32, device="cuda")
    K.kvc_evict_groups(cache, small, 0, D.n_layers, keep, recent, w.shape[-1], w, stay, groups, stream)
    return stay, groups


def expected_groups(w, E, keep, recent):
    out = torch.full((*w.shape[:-1], keep), -1, dtype=torch.int32)
    for at in [(b, h) for b in range(w.shape[0]) for h in range(w.shape[1])]:
        row = w[at].tolist()
        rank = [(i < E - recent, math.isnan(x), 0.0 if math.isnan(x) else -x, i) for i, x in enumerate(row[:E])]
        ids = sorted(i for *_, i in sorted(rank)[:keep])
        out[at][:len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return out


def check_evicted(cache, small, keep, recent, w, stay, groups):
    D = cache.dims
    for layer in range(D.n_layers):
        info, after = K.kvc_layer_info_get(cache, layer), K.kvc_layer_info_get(small, layer)
        exact = info["bits"] == 16
        E = info["window_tokens"] // 32 if exact else info["packed_tokens"] // 32
        want = expected_groups(w[layer].cpu(), E, keep, recent)
        assert torch.equal(groups[layer].cpu(), want)
        m = min(keep, E)
        assert after["packed_tokens"] == (0 if exact else 32 * m)
        assert after["window_tokens"] == (32 * m + info["window_tokens"] % 32 if exact else info["window_tokens"])
        assert after["appended"] == 0 and after["n_kept"] == 0 and after["prefilled"] == 1
        k0, v0, *_ = contents(cache, layer)
        k1, v1, *_ = contents(small, layer)
        tail = torch.arange(32 * E, k0.shape[2])
        n_slots = E + -(-len(tail) // 32)
        for b in range(D.batch):
            for h in range(D.n_kv_heads):
                ids = want[b, h][:m].long()
                rows = torch.cat([(ids[:, None] * 32 + torch.arange(32)).reshape(-1), tail]).cuda()
                assert torch.equal(k0[b, h, rows], k1[b, h]) and torch.equal(v0[b, h, rows], v1[b, h])
                left = torch.cat([w[layer, b, h].cpu()[ids], w[layer, b, h].cpu()[E:n_slots]])
                got = stay[layer, b, h].cpu()
                assert torch.equal(torch.nan_to_num(got[:len(left)], nan=-9.0), torch.nan_to_num(left, nan=-9.0))
                assert bool((got[len(left):] == 0).all())


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("recent", [0, 2])
def test_evict_matches(case, recent):
    cache, g = make_cache(7, **case)
    D = cache.dims
    n = max(slots_of(cache, i) for i in range(D.n_layers)) + 2
    # few distinct weights (ties), zeros of both signs, infinities and NaN among them
    w = torch.randint(-2, 6, (D.n_layers, D.batch, D.n_kv_heads, n), generator=g, device="cuda").float() / 3
    r = torch.rand(w.shape, generator=g, device="cuda")
    w = torch.where(r < 0.1, -0.0, w).masked_fill(r > 0.97, float("nan")).masked_fill((r > 0.2) & (r < 0.23), float("inf"))
    w = w.masked_fill((r > 0.3) & (r < 0.33), -float("inf"))
    most = max(K.kvc_layer_info_get(cache, i)["packed_tokens"] // 32 for i in range(D.n_layers))
    for keep in sorted({max(recent, 1), max(recent, most // 2, 1), max(most, recent, 1) + 1}):
        small = small_cache(cache, keep)
        stay, groups = evict(cache, small, keep, recent, w)
        torch.cuda.synchronize()
        check_evicted(cache, small, keep, recent, w, stay, groups)
        # and again into the same cache, from weights of another order
        K.kvc_cache_reset(small)
        w2 = w.flip(-1).contiguous()
        stay, groups = evict(cache, small, keep, recent, w2)
        torch.cuda.synchronize()
        check_evicted(cache, small, keep, recent, w2, stay, groups)


@pytest.mark.parametrize("n", [32 * 4096 + 40, 32 * 4097 + 5, 32 * 9000])
def test_evict_many_groups(n):
    """At and past what a block holds of a unit's weights in registers."""
    cache, g = make_cache(8, q_heads=1, kv_heads=1, d=64, n=n, alpha=3, bits=2)
    E = slots_of(cache, 0)
    w = torch.rand(1, 1, 1, E, generator=g, device="cuda")
    w[..., 100:3000] = w[..., 50:51]
    for keep in (1, 517, 3001, E // 32 * 31):
        small = small_cache(cache, keep)
        stay, groups = evict(cache, small, keep, 1, w)
        torch.cuda.synchronize()
        check_evicted(cache, small, keep, 1, w, stay, groups)


def test_streams_and_graph():
    """Captured and replayed on another stream, the three calls as used together."""
    cache, g = make_cache(11, q_heads=8, kv_heads=2, d=128, n=1000, alpha=16, bits=2)
    q = queries(cache, g)
    n = slots_of(cache, 0)
    before = torch.rand(1, 1, 2, n, generator=g, device="cuda")
    small = small_cache(cache, 9)
    out, after = weights(cache, q, before)
    stay, groups = evict(cache, small, 9, 1, after)
    out2, after2 = weights(small, q, stay)
    out3 = window(small, q, 3, 200)
    torch.cuda.synchronize()
    bufs = [torch.empty_like(t) for t in (out, after, stay, groups, out2, after2, out3)]
    K.kvc_cache_reset(small)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        K.kvc_decode_weights(cache, 0, 1, q, n, before, bufs[1], bufs[0])
        K.kvc_evict_groups(cache, small, 0, 1, 9, 1, n, bufs[1], bufs[2], bufs[3])
        K.kvc_decode_weights(small, 0, 1, q, n, bufs[2], bufs[5], bufs[4])
        K.kvc_decode_window(small, 0, 1, 3, 200, q, bufs[6])
    for _ in range(3):
        for b in bufs:
            b.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        for b, want in zip(bufs, (out, after, stay, groups, out2, after2, out3)):
            assert torch.equal(b, want)


def test_generation_goes_on():
    """Decode steps with accumulated weights and flushes, an eviction, more steps in the smaller cache:
    slots keep their tokens, and the sums are those of the steps' weights."""
    cache, g = make_cache(12, q_heads=4, kv_heads=2, d=64, n=400, alpha=16, bits=4, window=64, max_new=200)
    n = 400 // 32 + 200 // 32 + 4
    w = torch.zeros(1, 1, 2, n, device="cuda")
    total = torch.zeros(1, 2, n, dtype=torch.float64, device="cuda")
    steps = 0

    def step(c, w, total):
        kn, vn = (torch.randn(1, 1, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
        q = queries(c, g)
        out = torch.empty(1, 1, 4, 64, device="cuda")
        K.kvc_append_layers(c, 0, 1, kn, vn)
        K.kvc_decode_weights(c, 0, 1, q, n, w, w, out)
        keys, *_ = contents(c, 0)
        x = q[0].double().reshape(1, 2, 2, 64) @ keys.transpose(-1, -2) / 8
        p = torch.softmax(x, -1).sum(2)
        total += torch.nn.functional.pad(p, (0, n * 32 - p.shape[-1])).unflatten(-1, (n, 32)).sum(-1)
        check(c, q, out, lambda T: torch.ones(T, dtype=torch.bool))
    for _ in range(75):
        step(cache, w, total)
        steps += 1
    # each step's weights are within 2^-16 of themselves (check()'s bounds at these sizes)
    assert bool(((w[0].double() - total).abs() <= 2.0 ** -16 * total + 1e-30).all())
    small = small_cache(cache, 6, max_new=100)
    stay, groups = evict(cache, small, 6, 1, w)
    torch.cuda.synchronize()
    check_evicted(cache, small, 6, 1, w, stay, groups)
    total = stay[0].double()
    for _ in range(100):
        step(small, stay, total)
    assert bool(((stay[0].double() - total).abs() <= 2.0 ** -16 * total + 1e-30).all())
    assert K.kvc_layer_info_get(small, 0)["appended"] == 100
    with pytest.raises(K.KvcError) as e:
        step(small, stay, total)
    assert e.value.status == 6


def test_more_layers_than_a_launch_takes():
    """70 layers of three precisions: two launches of each kind, one scratch."""
    bits = [2, 16, 4, 2, 4, 4, 2] * 10
    cache, g = make_cache(21, q_heads=4, kv_heads=2, d=64, n=200, alpha=5, bits=2, layers=70, layer_bits=bits)
    q = queries(cache, g)
    n = max(slots_of(cache, i) for i in range(70))
    before = torch.rand(70, 1, 2, n, generator=g, device="cuda")
    out, after = weights(cache, q, before)
    check(cache, q, out, lambda T: torch.ones(T, dtype=torch.bool))
    check(cache, q, window(cache, q, 3, 40), lambda T: (torch.arange(T) < 3) | (torch.arange(T) >= T - 40))
    for layer in (0, 1, 63, 64, 69):
        one, w = torch.empty(1, 1, 4, 64, device="cuda"), torch.empty(1, 1, 2, n, device="cuda")
        K.kvc_decode_weights(cache, layer, 1, q[layer:layer + 1].contiguous(), n, before[layer:layer + 1].contiguous(), w, one)
        # (another split of the work: other roundings, fp32 sums of a few hundred terms)
        assert bool(((w[0] - after[layer]).abs() <= 2.0 ** -16 * after[layer]).all())
    small = small_cache(cache, 3)
    stay, groups = evict(cache, small, 3, 1, after)
    torch.cuda.synchronize()
    check_evicted(cache, small, 3, 1, after, stay, groups)


def test_calls_on_part_of_the_layers():
    cache, g = make_cache(22, q_heads=4, kv_heads=2, d=64, n=300, alpha=5, bits=4, layers=3)
    q = queries(cache, g)
    n = slots_of(cache, 0)
    w = torch.rand(3, 1, 2, n, generator=g, device="cuda")
    small = small_cache(cache, 4)
    for layer in (2, 0):
        part = w[layer:layer + 1].contiguous()
        stay, groups = torch.empty_like(part), torch.empty(1, 1, 2, 4, dtype=torch.int32, device="cuda")
        K.kvc_evict_groups(cache, small, layer, 1, 4, 0, n, part, stay, groups)
        torch.cuda.synchronize()
        want = expected_groups(w[layer].cpu(), 9, 4, 0)
        assert torch.equal(groups[0].cpu(), want)
    assert [K.kvc_layer_info_get(small, i)["prefilled"] for i in range(3)] == [1, 0, 1]
    refused(5, K.kvc_decode_window, small, 0, 3, 1, 1, q, torch.empty(3, 1, 4, 64, device="cuda"))


def test_far_values_keep_their_marks():
    """Values past fp16's range once dequantized: the small cache's units carry the marks that the
    tree attention goes by."""
    g = torch.Generator(device="cuda").manual_seed(23)
    dims = K.make_dims(1, 1, 4, 2, 128, 300, 16, 7, 2, 32, 64, 4)
    k = torch.randn(1, 2, 300, 128, generator=g, device="cuda").bfloat16()
    v = torch.randn(1, 2, 300, 128, generator=g, device="cuda").bfloat16()
    # (not below -65,504: a zero-point is a group's least value, in fp16)
    v[:, 1, 70:90] = v[:, 1, 70:90].abs() * 30000
    cache = K.kvc_prefill_compress(dims, [300], 0, None, k, v)
    n = slots_of(cache, 0)
    w = torch.arange(n, 0, -1, device="cuda").float().expand(1, 1, 2, n).contiguous()
    small = small_cache(cache, 6)
    evict(cache, small, 6, 0, w)
    torch.cuda.synchronize()
    assert bool((contents(small, 0)[1] > 65504).any()) and bool(torch.isfinite(contents(small, 0)[1]).all())
    q = torch.randn(1, 1, 4, 3, 128, generator=g, device="cuda").bfloat16()
    kd = torch.randn(1, 1, 2, 3, 128, generator=g, device="cuda").bfloat16()
    parents = torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    K.kvc_tree_attn(small, 0, 1, 3, parents, q, kd, kd, out)
    keys, values, *_ = contents(small, 0)
    for i in range(3):
        qq = q[0, :, :, i].double().reshape(1, 2, 2, 128)
        kk, vv = torch.cat([keys, kd[0, :, :, :i + 1].double()], 2), torch.cat([values, kd[0, :, :, :i + 1].double()], 2)
        want, size, av = attend(qq, kk, vv)
        # roundings of keys, values and weights (2^-11 each, drafted ones 2^-8), of the output (2^-8)
        lim = av * (2 * size * 2.0 ** -10 + 2.0 ** -7) + 2.0 ** -8 * want.abs() + 2.0 ** -20 * values.abs().amax()
        assert bool(((out[0, :, :, i].double().reshape(want.shape) - want).abs() <= lim).all())


# ------------------------------------------------------------------------------------ refusals
def refused(status, call, *args):
    before = K.kvc_launch_count()
    with pytest.raises(K.KvcError) as e:
        call(*args)
    assert e.value.status == status and K.kvc_launch_count() == before


def test_refusals():
    cache, g = make_cache(13, q_heads=4, kv_heads=2, d=64, n=300, layers=2, bits=2, max_new=4)
    q = queries(cache, g)
    out = torch.empty(2, 1, 4, 64, device="cuda")
    n = slots_of(cache, 0)
    w, stay = torch.rand(2, 1, 2, n, device="cuda"), torch.empty(2, 1, 2, n, device="cuda")
    groups = torch.empty(2, 1, 2, 4, dtype=torch.int32, device="cuda")
    odd = torch.empty(4096, dtype=torch.bfloat16, device="cuda")[1:]
    byte = torch.empty(4096, dtype=torch.uint8, device="cuda")[1:]

    dw = K.kvc_decode_window
    for lb, lc in ((-1, 1), (0, 3), (2, 1), (0, 0), (1, 2 ** 31 - 1)):
        refused(1, dw, cache, lb, lc, 1, 1, q, out)
    for s, last in ((-1, 1), (0, 0), (0, -5)):
        refused(1, dw, cache, 0, 2, s, last, q, out)
    for a, b in ((None, out), (q, None), (odd, out), (q, odd)):
        refused(1, dw, cache, 0, 2, 1, 1, a, b)

    kw = K.kvc_decode_weights
    for args in ((-1, 1, q, n, w, stay, out), (0, 3, q, n, w, stay, out), (0, 2, q, n - 1, w, stay, out),
                 (0, 2, q, 0, w, stay, out), (0, 2, odd, n, w, stay, out), (0, 2, q, n, byte, stay, out),
                 (0, 2, q, n, w, byte, out), (0, 2, q, n, w, stay, odd), (0, 2, None, n, w, stay, out),
                 (0, 2, q, n, None, stay, out), (0, 2, q, n, w, None, out), (0, 2, q, n, w, stay, None)):
        refused(1, kw, cache, *args)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        refused(5, kw, cache, 0, 2, q, n, w, stay, out)     # its first call is not captured

    ev = K.kvc_evict_groups
    small = small_cache(cache, 4)
    for args in ((cache, 0, 2, 4, 0, n, w, stay, groups), (small, 0, 3, 4, 0, n, w, stay, groups),
                 (small, 0, 2, 0, 0, n, w, stay, groups), (small, 0, 2, 4, 5, n, w, stay, groups),
                 (small, 0, 2, 4, -1, n, w, stay, groups), (small, 0, 2, 4, 0, n - 1, w, stay, groups),
                 (small, 0, 2, (1 << 20) + 1, 0, n, w, stay, groups), (small, 0, 2, 4, 0, n, byte, stay, groups),
                 (small, 0, 2, 4, 0, n, w, byte, groups), (small, 0, 2, 4, 0, n, w, stay, byte),
                 (small, 0, 2, 4, 0, n, None, stay, groups), (small, 0, 2, 4, 0, n, w, None, groups),
                 (small, 0, 2, 4, 0, n, w, stay, None)):
        refused(1, ev, cache, *args)

    def like(**change):
        d = dict(n_layers=2, batch=1, n_q_heads=4, n_kv_heads=2, head_dim=64, prompt_len=256, obs_window=0,
                 pool_kernel=1, bits=2, group_size=32, window_len=64, max_new_tokens=4)
        d.update(change)
        dims = K.make_dims(*d.values())
        return K.kvc_cache_create(dims, [256] * d["n_layers"])
    for change in (dict(n_layers=3), dict(batch=2), dict(n_q_heads=8), dict(n_kv_heads=4), dict(head_dim=128),
                   dict(bits=4), dict(window_len=96)):
        refused(2, ev, cache, like(**change), 0, 2, 4, 0, n, w, stay, groups)
    groups8 = torch.empty(2, 1, 2, 8, dtype=torch.int32, device="cuda")
    refused(6, ev, cache, like(prompt_len=32), 0, 2, 8, 0, n, w, stay, groups8)
    fits = like()
    ev(cache, fits, 0, 2, 4, 0, n, w, stay, groups)
    refused(5, ev, cache, fits, 0, 2, 4, 0, n, w, stay, groups)     # not empty
    K.kvc_cache_reset(fits)
    refused(5, ev, fits, cache, 0, 2, 4, 0, n, w, stay, groups)     # nothing to evict from
    refused(5, dw, fits, 0, 2, 1, 1, q, out)
    refused(5, kw, fits, 0, 2, q, n, w, stay, out)
    # the capacity is exact: what the smallest cache takes, it holds after max_new_tokens appends
    tight, extra = 0, None
    for p in range(32, 320, 32):
        c = like(prompt_len=p, max_new_tokens=70)
        try:
            ev(cache, c, 0, 2, 8, 0, n, w, stay, groups8)
        except K.KvcError as e:
            assert e.status == 6
            tight += 1
            continue
        extra = c
        break
    assert tight > 0 and extra is not None
    for _ in range(70):
        K.kvc_append_layers(extra, 0, 2, q[:, :, :2].contiguous(), q[:, :, :2].contiguous())
    info = K.kvc_layer_info_get(extra, 0)
    assert info["packed_tokens"] <= info["capacity_tokens"]
    K.kvc_check_device(extra)


def test_wait_that_gives_up_is_reported():
    cache, g = make_cache(14, q_heads=4, kv_heads=2, d=64, n=3000, bits=2)
    q = queries(cache, g)
    out = torch.empty(1, 1, 4, 64, device="cuda")
    want = window(cache, q, 4, 2000)
    K.kvc_set_wait_limit(cache, 0)
    K.kvc_decode_window(cache, 0, 1, 4, 2000, q, out)
    with pytest.raises(K.KvcError) as e:
        K.kvc_check_device(cache)
    assert e.value.status == 7
    K.kvc_set_wait_limit(cache, -1)
    assert torch.equal(window(cache, q, 4, 2000), want)
