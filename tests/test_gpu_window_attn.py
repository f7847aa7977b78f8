"""Prompt attention over a sliding window with sinks, and the cache it leaves, against a plain 64-bit
form and kvc_prefill_sinks."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import U32, UB, attend  # noqa: E402


def make(seed, q_heads, kv_heads, d, n, batch=1, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(batch, kv_heads, n, d, generator=g, device="cuda").bfloat16()
    v = torch.randn(batch, kv_heads, n, d, generator=g, device="cuda").bfloat16()
    q = (spread * torch.randn(batch, q_heads, n, d, generator=g, device="cuda")).bfloat16()
    return q, k, v


def new_cache(q, k, budget, bits=2, alpha=1):
    B, Hq, n, d = q.shape
    window = 128 if bits != 16 else (n + 4 + 31) // 32 * 32
    alpha = min(alpha, n - 1)
    dims = K.make_dims(1, B, Hq, k.shape[1], d, n, alpha, 1, bits, 32, window, 4)
    return K.kvc_cache_create(dims, [budget if alpha else n])


def prompt(cache, q, k, v, s, w, stream=None):
    x = torch.full_like(q, float("nan"))
    K.kvc_prefill_window(cache, 0, s, w, q, k, v, x, stream)
    return x


def check(q, k, v, s, w, x, skip=None):
    B, Hq, n, d = q.shape
    H = k.shape[1]
    t = torch.arange(n, device="cuda")
    seen = (t <= t[:, None]) & ((t < s) | (t[:, None] - t < w))
    for b in range(B):
        for h in range(Hq):
            kk, vv = k[b, h // (Hq // H)].double(), v[b, h // (Hq // H)].double()
            want, size, av = attend(q[b, h].double(), kk, vv, seen)
            got = x[b, h].double()
            # logits: exact products, fp32 sums whose steps may be cut off (2 U32 a term); weights:
            # exp2 of a rounded argument (16 U32 of the largest logit), one bf16 rounding; output: one
            e = size * (2 * d + 16) * U32
            lim = av * (2 * e + UB + 2.0 ** -18) + UB * (1 + UB) * want.abs()
            ok = (got - want).abs() <= lim
            if skip is not None:
                ok = ok | skip[:, None]
            assert bool(ok.all()), (b, h, ((got - want).abs() / lim).nan_to_num(math.inf).max())


SHAPES = [
    dict(q_heads=2, kv_heads=2, d=64, n=528),
    dict(q_heads=2, kv_heads=1, d=128, n=700),
    dict(q_heads=8, kv_heads=2, d=128, n=389, batch=2),
    dict(q_heads=16, kv_heads=2, d=64, n=1001),
    dict(q_heads=8, kv_heads=1, d=128, n=33),
    dict(q_heads=1, kv_heads=1, d=64, n=2),
    dict(q_heads=4, kv_heads=4, d=128, n=256, batch=3),
]
RANGES = [(4, 100), (0, 1), (0, 129), (1, 1), (300, 17), (5, 1 << 30), (1 << 30, 3), (128, 128), (130, 257), (33, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_matches(shape):
    q, k, v = make(1, **shape)
    for s, w in RANGES:
        cache = new_cache(q, k, 64)
        x = prompt(cache, q, k, v, s, w)
        torch.cuda.synchronize()
        K.kvc_check_device(cache)
        check(q, k, v, s, w, x)


def test_one_token():
    q, k, v = make(2, 4, 2, 64, 1)
    dims = K.make_dims(1, 1, 4, 2, 64, 1, 0, 1, 4, 32, 64, 4)
    cache = K.kvc_cache_create(dims, [1])
    x = prompt(cache, q, k, v, 0, 1)
    assert torch.equal(x, v.repeat_interleave(2, 1))


def test_more_items_than_ctas():
    """Every CTA takes several items: ring, barriers and tensor memory are handed on."""
    q, k, v = make(3, 8, 8, 64, 6000, batch=2)
    for s, w in ((4, 128), (0, 1), (200, 300)):
        x = prompt(new_cache(q, k, 64), q, k, v, s, w)
        y = prompt(new_cache(q, k, 64), q, k, v, s, w)
        assert torch.equal(x, y)
        check(q[:, 5:6], k[:, 5:6], v[:, 5:6], s, w, x[:, 5:6])


@pytest.mark.parametrize("q_heads,kv_heads,d,n", [(2, 2, 128, 257), (8, 2, 128, 389), (8, 1, 128, 161), (2, 1, 64, 300),
                                                  (8, 1, 64, 47), (2, 2, 64, 1)])
def test_many_units(q_heads, kv_heads, d, n):
    """Units enough that an item takes two row tiles, the last item's second one with few rows or none."""
    B = 160 // kv_heads
    if n == 1:
        q, k, v = make(11, q_heads, kv_heads, d, 1, batch=B)
        dims = K.make_dims(1, B, q_heads, kv_heads, d, 1, 0, 1, 4, 32, 64, 4)
        x = prompt(K.kvc_cache_create(dims, [1]), q, k, v, 0, 1)
        assert torch.equal(x, v)
        return
    q, k, v = make(11, q_heads, kv_heads, d, n, batch=B)
    for s, w in ((4, 100), (0, 1), (130, 33), (0, 1 << 30)):
        x = prompt(new_cache(q, k, 32), q, k, v, s, w)
        for b in (0, B // 2, B - 1):
            check(q[b:b + 1], k[b:b + 1], v[b:b + 1], s, w, x[b:b + 1])


def test_places_that_are_not_seen_many_units():
    """As in test_places_that_are_not_seen, where an item's two row tiles share a key tile that only one of them sees."""
    q, k, v = make(12, 4, 2, 128, 400, batch=80)
    s, w = 4, 70
    k[0, 0, 150] = float("nan")
    v[79, 1, 200, 3] = float("inf")
    x = prompt(new_cache(q, k, 64), q, k, v, s, w)
    t = torch.arange(400, device="cuda")
    for b, h, a in ((0, 0, 150), (79, 1, 200)):
        hit = (t >= a) & (t < a + w)
        kk, vv = k[b:b + 1, h:h + 1].clone(), v[b:b + 1, h:h + 1].clone()
        kk[~torch.isfinite(kk)] = 0
        vv[~torch.isfinite(vv)] = 0
        rows = x[b:b + 1, 2 * h:2 * h + 2]
        assert bool(torch.isfinite(rows[:, :, ~hit]).all())
        check(q[b:b + 1, 2 * h:2 * h + 2], kk, vv, s, w, rows, skip=hit)
    assert bool(torch.isnan(x[0, :2, 150:150 + w]).all())
    assert bool(torch.isinf(x[79, 2:, 200, 3]).all())


def test_growing_and_large_logits():
    """Maxima that rise along the keys (references follow, outputs are rescaled) and logits far
    past 2^16, where one key takes all the weight."""
    q, k, v = make(4, 2, 1, 64, 900)
    ramp = torch.linspace(0.1, 40, 900, device="cuda")[:, None]
    u = torch.ones(64, device="cuda") / 8
    up = (k.float() * 0.2 + ramp * u).bfloat16()
    qq = (q.float() * 0.2 + 8 * u).bfloat16()
    check(qq, up, v, 3, 400, prompt(new_cache(qq, up, 64), qq, up, v, 3, 400))
    big_q, big_k = (q.float() * 2.0 ** 20).bfloat16(), (k.float() * 2.0 ** 12).bfloat16()
    x = prompt(new_cache(big_q, big_k, 64), big_q, big_k, v, 3, 400)
    assert bool(torch.isfinite(x).all())
    t = torch.arange(900, device="cuda")
    seen = (t <= t[:, None]) & ((t < 3) | (t[:, None] - t < 400))
    for h in range(2):
        logits = big_q[0, h].double() @ big_k[0, 0].double().T / 8
        best = logits.masked_fill(~seen, -math.inf).topk(2, -1)
        # rows whose first two logits are apart by more than the fp32 sums may be off
        sure = best.values[:, 0] - best.values[:, 1] > 2.0 ** 33 * 64 * 64 * U32
        assert int(sure.sum()) > 400
        assert torch.equal(x[0, h][sure], v[0, 0][best.indices[:, 0]][sure])


def test_places_that_are_not_seen():
    """Infinities and NaN in keys and values: rows that see none of them are as without; a NaN that
    is seen makes the row NaN."""
    q, k, v = make(5, 8, 2, 128, 1200)
    k[0, 0, 500] = float("nan")
    v[0, 0, 501] = float("inf")
    v[0, 1, 700, 3] = float("nan")
    k[0, 1, 701] = -float("inf")
    s, w = 4, 150
    x = prompt(new_cache(q, k, 64), q, k, v, s, w)
    torch.cuda.synchronize()
    t = torch.arange(1200, device="cuda")
    for h, (a, b) in ((0, (500, 501 + w)), (1, (700, 701 + w))):
        hit = (t >= a) & (t < b)
        kk, vv = k[:, h:h + 1].clone(), v[:, h:h + 1].clone()
        kk[~torch.isfinite(kk)] = 0
        vv[~torch.isfinite(vv)] = 0
        rows = x[:, 4 * h:4 * h + 4]
        assert bool(torch.isfinite(rows[:, :, ~hit]).all())
        check(q[:, 4 * h:4 * h + 4], kk, vv, s, w, rows, skip=hit)
    assert bool(torch.isnan(x[0, :4, 500:500 + w]).all())
    assert bool(torch.isnan(x[0, 4:, 700:700 + w, 3]).all())


@pytest.mark.parametrize("bits", [2, 4, 16])
def test_leaves_the_cache_of_the_sinks_call(bits):
    q, k, v = make(6, 8, 2, 64, 900, batch=2)
    for s, budget in ((4, 260), (0, 64), (1000, 96), (7, 900)):
        got, want = new_cache(q, k, budget, bits, 16), new_cache(q, k, budget, bits, 16)
        prompt(got, q, k, v, s, 260)
        K.kvc_prefill_sinks(want, 0, s, k, v)
        a, b = K.kvc_export_layer(got, 0), K.kvc_export_layer(want, 0)
        assert K.kvc_layer_info_get(got, 0) == K.kvc_layer_info_get(want, 0)
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_as_used():
    """A prompt through the window, then tokens: each sees what a window over all tokens would show
    it (a 16-bit cache, so that nothing but the roundings of the calls differs)."""
    s, w, n, steps = 4, 96, 700, 40
    q, k, v = make(7, 4, 2, 64, n + steps)
    first = [z[:, :, :n].contiguous() for z in (q, k, v)]
    dims = K.make_dims(1, 1, 4, 2, 64, n, 16, 1, 16, 32, 256, steps)
    cache = K.kvc_cache_create(dims, [s + w])
    x = prompt(cache, *first, s, w)
    check(*first, s, w, x)
    full = new_cache(q, k, 64)
    whole = prompt(full, q, k, v, s, w)
    assert torch.equal(whole[:, :, :512], x[:, :, :512])   # rows do not depend on what follows them
    for i in range(n, n + steps):
        K.kvc_append(cache, 0, k[:, :, i].contiguous(), v[:, :, i].contiguous())
        out = torch.empty(1, 1, 4, 64, device="cuda")
        K.kvc_decode_window(cache, 0, 1, s, w, q[:, :, i].contiguous(), out)
        want = whole[:, :, i].double()
        # the prompt's row: bf16 weights and output; the step: fp32
        lim = 2 * UB * v.double().abs().amax()
        assert bool(((out[0].double() - want).abs() <= lim).all())


def test_stream_and_graph():
    q, k, v = make(8, 8, 2, 128, 500)
    want = prompt(new_cache(q, k, 96), q, k, v, 4, 96)
    torch.cuda.synchronize()
    cache = new_cache(q, k, 96)
    s, graph, x = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph, stream=s):
        K.kvc_prefill_window(cache, 0, 4, 96, q, k, v, x)
    for _ in range(3):
        x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)


def test_refusals():
    q, k, v = make(9, 8, 2, 64, 300)
    x = torch.full_like(q, 3.0)
    cache = new_cache(q, k, 64)

    def refused(status, *args):
        before = K.kvc_launch_count()
        with pytest.raises(K.KvcError) as e:
            K.kvc_prefill_window(*args)
        assert e.value.status == status and K.kvc_launch_count() == before
    refused(1, cache, 0, -1, 5, q, k, v, x)
    refused(1, cache, 0, 1, 0, q, k, v, x)
    refused(1, cache, 1, 1, 5, q, k, v, x)
    refused(1, cache, -1, 1, 5, q, k, v, x)
    for i in range(4):
        for bad in (None, torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:]):
            args = [q, k, v, x]
            args[i] = bad
            refused(1, cache, 0, 1, 5, *args)
    K.kvc_prefill_window(cache, 0, 1, 5, q, k, v, x)
    refused(5, cache, 0, 1, 5, q, k, v, x)


def test_output_at_16_bytes():
    """x_out 16-byte aligned and no more: rows are written in halves of a sector."""
    q, k, v = make(10, 8, 2, 128, 300, batch=2)
    want = prompt(new_cache(q, k, 64), q, k, v, 4, 96)
    room = torch.full((q.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    x = room[8:8 + q.numel()].view(q.shape)
    assert x.data_ptr() % 32 == 16
    K.kvc_prefill_window(new_cache(q, k, 64), 0, 4, 96, q, k, v, x)
    assert torch.equal(x, want)
    assert bool((room[:8] == 7).all()) and bool((room[8 + q.numel():] == 7).all())


def test_waits_that_give_up_are_reported():
    q, k, v = make(11, 8, 2, 128, 3000)
    cache = new_cache(q, k, 64)
    want = prompt(cache, q, k, v, 4, 96)
    K.kvc_cache_reset(cache)
    K.kvc_set_wait_limit(cache, 0)
    try:
        prompt(cache, q, k, v, 4, 96)
    except K.KvcError as e:             # (the packing's call may see the error word already)
        assert e.status == 7
    else:
        with pytest.raises(K.KvcError) as e:
            K.kvc_check_device(cache)
        assert e.value.status == 7
    torch.cuda.synchronize()
    try:
        K.kvc_check_device(cache)
    except K.KvcError as e:
        assert e.status == 7
    K.kvc_set_wait_limit(cache, -1)
    K.kvc_cache_reset(cache)
    assert torch.equal(prompt(cache, q, k, v, 4, 96), want)
    K.kvc_check_device(cache)


def test_two_caches_on_two_streams():
    made = [make(12 + i, 8, 2, 128 if i else 64, 2500) for i in range(2)]
    caches = [new_cache(q, k, 200) for q, k, v in made]
    want = [prompt(c, q, k, v, 4, 200) for c, (q, k, v) in zip(caches, made)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(w) for w in want]
    for _ in range(5):
        for s, c, (q, k, v), x in zip(streams, caches, made, got):
            x.fill_(0)
        torch.cuda.synchronize()
        for s, c, (q, k, v), x in zip(streams, caches, made, got):
            K.kvc_cache_reset(c)
            K.kvc_prefill_window(c, 0, 4, 200, q, k, v, x, s)
        torch.cuda.synchronize()
        for x, w in zip(got, want):
            assert torch.equal(x, w)
