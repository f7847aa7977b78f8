"""Prompt attention over a sliding window where values or keys are not finite: every output against the
formula in 64 bits (NaN, infinities and finite values each in their places), and the time of such
calls, which stays within a small multiple of a call's without."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import U32, UB, attend  # noqa: E402
from test_gpu_window_attn import make, new_cache, prompt  # noqa: E402

INF, NAN = math.inf, math.nan


def expected(q, k, v, seen):
    """softmax(q k / sqrt d) v of one head over the keys seen. A channel in which a row sees a NaN, or
    infinities of both signs, is NaN, one with infinities of one sign infinite; an infinite value whose
    weight is exactly 0 (its logit is -inf) makes it NaN."""
    x = (q @ k.T / math.sqrt(q.shape[-1])).masked_fill(~seen, -INF)
    w = torch.softmax(x, -1)
    w = torch.where(torch.isnan(w).any(-1, keepdim=True), NAN, w)
    out = w @ torch.where(torch.isfinite(v), v, 0.0)

    def any_of(rows, values):
        return rows.double() @ values.double() > 0
    up, down = any_of(seen & (w > 0), v == INF), any_of(seen & (w > 0), v == -INF)
    bad = any_of(seen, torch.isnan(v)) | (up & down) | any_of(seen & (w == 0), torch.isinf(v))
    out = torch.where(up, INF, out)
    out = torch.where(down, -INF, out)
    return torch.where(bad | torch.isnan(w).any(-1, keepdim=True), NAN, out)


def check(q, k, v, s, w, x):
    B, Hq, n, d = q.shape
    H = k.shape[1]
    t = torch.arange(n, device="cuda")
    seen = (t <= t[:, None]) & ((t < s) | (t[:, None] - t < w))
    counts = [0, 0, 0]
    for b in range(B):
        for h in range(Hq):
            kk, vv, qq = k[b, h // (Hq // H)].double(), v[b, h // (Hq // H)].double(), q[b, h].double()
            want, got = expected(qq, kk, vv, seen), x[b, h].double()
            assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, h)
            assert torch.equal(got == INF, want == INF) and torch.equal(got == -INF, want == -INF), (b, h)
            fine = torch.isfinite(want)
            # as where everything is finite, over the finite elements (two weights' roundings where a row
            # is formed again): logits' sums, weights rounded to bf16, one rounding of the output
            k0, v0 = torch.where(torch.isfinite(kk), kk, 0.0), torch.where(torch.isfinite(vv), vv, 0.0)
            _, size, av = attend(qq, k0, v0, seen)
            if bool(torch.isinf(kk).any()):     # weights are not those of k0: the largest value bounds them
                av = (seen.double().unsqueeze(-1) * v0.abs()).amax(1)
            e = size * (2 * d + 16) * U32
            lim = av * (2 * e + UB + 2.0 ** -18) + UB * (1 + UB) * want.abs()
            assert bool(((got - want).abs() <= lim)[fine].all()), (b, h)
            for i, m in enumerate((torch.isnan(want), torch.isinf(want), fine)):
                counts[i] += int(m.sum())
    return counts


def sprinkle(z, g, share, values):
    at = torch.rand(z.shape, generator=g, device="cuda")
    for i, value in enumerate(values):
        z.masked_fill_((at >= i * share) & (at < (i + 1) * share), value)


def one_seen_by_all(k, v, g): v[:, :, 0, 3] = NAN
def one_late(k, v, g): v[:, :, 200, 5] = INF
def few(k, v, g): sprinkle(v, g, 1e-4, (NAN, INF, -INF))
def many(k, v, g): sprinkle(v, g, 3e-3, (NAN, INF, -INF))
def infinities(k, v, g): sprinkle(v, g, 1e-3, (INF,))
def every_other(k, v, g): v[:, :, 1::2] = INF
def all_values(k, v, g): v.fill_(NAN)


def channels(k, v, g):
    v[..., 1], v[..., 7], v[..., 40] = NAN, INF, -INF
    v[:, :, ::3, 9] = INF
    v[:, :, 1::3, 9] = -INF


def keys(k, v, g):
    sprinkle(k, g, 5e-5, (NAN, INF, -INF))
    sprinkle(v, g, 1e-4, (NAN, INF))


def key_and_value(k, v, g):
    """A key whose logits are infinite, beside an infinite value: a weight of exactly 0 where the logit is
    -inf (NaN), rows without a sum where it is +inf."""
    k[:, :, 30, 2] = INF
    v[:, :, 30, 6] = -INF
    v[:, :, 2::5, 6] = -INF


WHAT = [one_seen_by_all, one_late, few, many, infinities, every_other, all_values, channels, keys, key_and_value]
SHAPES = [
    dict(q_heads=2, kv_heads=2, d=64, n=528),
    dict(q_heads=8, kv_heads=2, d=128, n=389, batch=2),
    dict(q_heads=8, kv_heads=1, d=64, n=333),
    dict(q_heads=4, kv_heads=2, d=128, n=300, batch=80),     # items of two row tiles
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
@pytest.mark.parametrize("what", WHAT, ids=[f.__name__ for f in WHAT])
def test_each_element(shape, what):
    q, k, v = make(41, **shape)
    g = torch.Generator(device="cuda").manual_seed(42)
    what(k, v, g)
    some = 0
    for s, w in ((4, 100), (0, 1), (70, 33), (0, 1 << 30), (1 << 30, 5)):
        x = prompt(new_cache(q, k, 64), q, k, v, s, w)
        torch.cuda.synchronize()
        b = slice(0, 2) if shape.get("batch", 1) > 2 else slice(None)
        counts = check(q[b], k[b], v[b], s, w, x[b])
        some += counts[0] + counts[1]
    assert some > 0


@pytest.mark.parametrize("size", [3e38, 1e37])
@pytest.mark.parametrize("what", [None, one_late, channels])
def test_values_whose_sums_pass_fp32(size, what):
    """Finite values near the largest there is: their weighted mean is finite, and so is the output."""
    q, k, v = make(44, 4, 2, 64, 400)
    v = ((1 + 0.1 * v.float().clamp(-1, 1)) * size).bfloat16()
    assert bool(torch.isfinite(v).all())
    if what:
        what(k, v, None)
    for s, w in ((4, 100), (0, 1 << 30)):
        x = prompt(new_cache(q, k, 64), q, k, v, s, w)
        torch.cuda.synchronize()
        assert check(q, k, v, s, w, x)[2] > 0


def elapsed(call):
    best = math.inf
    for _ in range(4):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("d,n,w", [(128, 8192, 1 << 30), (64, 8192, 1 << 30), (128, 16384, 1024)])
def test_time_has_a_bound(d, n, w):
    """What rows see is read about once for 32 of them, not every key for each: a call takes a few times
    what it takes without (with every such row formed again: some hundred times). Values that rows see;
    the rows that a hidden one spoils, a few hundred, are formed again, by one CTA."""
    q, k, v = make(43, 8, 2, d, n)
    cache, x = new_cache(q, k, 64), torch.empty_like(q)

    def call(k, v):
        K.kvc_cache_reset(cache)
        K.kvc_prefill_window(cache, 0, 4, w, q, k, v, x)
    call(k, v)
    clean = elapsed(lambda: call(k, v))
    for what in (one_seen_by_all, all_values, channels):
        kk, vv = k.clone(), v.clone()
        what(kk, vv, None)
        t = elapsed(lambda: call(kk, vv))
        assert t <= 20 * clean, (what.__name__, t, clean)
    kk = k.clone()
    kk[:, :, 0, 3] = NAN
    t = elapsed(lambda: call(kk, v))
    assert t <= 3 * clean and bool(torch.isnan(x).all()), (t, clean)
