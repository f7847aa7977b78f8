"""Edges of the calls that read listed groups or many queries at a time: layers that hold nothing,
stored values and queries past fp16's range, dominant tokens, cancelling queries, and what an
earlier sequence left in the window. All against plain 64-bit forms over the exported cache."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import U16, U32, UB, attend, contents, sum_bound  # noqa: E402
from test_gpu_groups import check_decode, decode, expected_lists, queries, select  # noqa: E402
from test_gpu_tree import check, inputs, tree, trees  # noqa: E402


def cache_of(k, v, q_heads, bits, alpha=0, window=64, max_new=4):
    """A one-layer cache of the keys and values [B][H][n][d], kept whole."""
    B, H, n, d = k.shape
    dims = K.make_dims(1, B, q_heads, H, d, n, alpha, 7, bits, 32, window, max_new)
    return K.kvc_prefill_compress(dims, [n], 0, None, k.bfloat16().contiguous(),
                                  v.bfloat16().contiguous())


# ------------------------------------------------------------------ layers that hold nothing
def empty_between(d, bits, heads=(4, 2), batch=2, layers=5, empty=(1, 3)):
    """Layers of a prompt kept whole, but for those in `empty`, which keep no token and have no
    observation window."""
    n = 200
    dims = K.make_dims(layers, batch, heads[0], heads[1], d, n, 0, 7, bits, 32, 64, 4)
    cache = K.kvc_cache_create(dims, [n] * layers)
    g = torch.Generator(device="cuda").manual_seed(d + bits)
    for layer in range(layers):
        k = torch.randn(batch, heads[1], n, d, generator=g, device="cuda").bfloat16()
        v = torch.randn(batch, heads[1], n, d, generator=g, device="cuda").bfloat16()
        if layer in empty:
            K.kvc_prefill_selected(cache, layer, None, 0, k, v)
        else:
            K.kvc_prefill_compress(dims, [n] * layers, layer, None, k, v, cache)
    torch.cuda.synchronize()
    return cache, g


@pytest.mark.parametrize("d,bits", [(64, 2), (128, 4)])
@pytest.mark.parametrize("empty", [(1, 3), (0,), (4,), (0, 1, 2, 3, 4)])
def test_listed_decode_of_layers_that_hold_nothing(d, bits, empty):
    cache, g = empty_between(d, bits, empty=empty)
    q = queries(cache, g)
    lists = select(cache, q, 3)
    assert torch.equal(lists.cpu(), expected_lists(cache, q, 3))
    for layer in empty:
        assert (lists[layer] == -1).all()
    got = decode(cache, q, lists)
    check_decode(cache, q, lists, got)
    for layer in empty:                      # alone, and with entries that name no group
        out = torch.full_like(got[layer], float("nan"))
        K.kvc_decode_groups(cache, layer, 1, q[layer], 3, torch.zeros_like(lists[layer]), out)
        assert (out == 0).all()
        full = torch.full_like(out, float("nan"))
        K.kvc_decode_attn(cache, layer, 1, q[layer], full)
        assert (full == 0).all()


@pytest.mark.parametrize("d,bits", [(64, 2), (64, 4), (128, 2)])
@pytest.mark.parametrize("heads,batch,T", [((4, 2), 2, 5), ((8, 8), 40, 9), ((8, 2), 100, 6),
                                           ((8, 1), 60, 33)])
def test_tree_over_layers_that_hold_nothing(d, bits, heads, batch, T):
    """The drafted tokens alone, alone in a launch and between layers that hold tokens."""
    cache, g = empty_between(d, bits, heads, batch, layers=3, empty=(0, 2))
    q, k, v = inputs(cache, g, T)
    parents = trees("padding", batch, T, g)
    got = tree(cache, parents, q, k, v)
    check(cache, parents, q, k, v, got)
    for layer in (0, 2):
        out = torch.full_like(q[layer], float("nan"))
        for _ in range(10):
            K.kvc_tree_attn(cache, layer, 1, T, parents, q[layer], k[layer], v[layer], out)
        assert torch.equal(out, got[layer])


# ------------------------------------------- stored values and queries past fp16's range
def wide(shape, g, low, high, share):
    """Values of N(0, 1), a share of the 32-token groups spread over [low, high] instead."""
    B, H, n, d = shape
    x = torch.randn(shape, generator=g, device="cuda")
    far = low + (high - low) * torch.rand(shape, generator=g, device="cuda")
    on = torch.rand(B, H, n // 32, 1, 1, generator=g, device="cuda") < share
    return torch.where(on, far.reshape(B, H, n // 32, 32, d), x.reshape(B, H, n // 32, 32, d)).reshape(shape)


# zero-points and scales finite in fp16, the largest stored values up to twice fp16's range
WIDE = [dict(d=128, bits=4, heads=(8, 2)), dict(d=64, bits=2, heads=(2, 1)),
        dict(d=128, bits=2, heads=(4, 4)), dict(d=64, bits=4, heads=(8, 1))]


@pytest.mark.parametrize("case", WIDE, ids=[str(i) for i in range(len(WIDE))])
@pytest.mark.parametrize("part", ["keys", "values", "both"])
@pytest.mark.parametrize("T", [3, 40])
def test_tree_over_stored_values_past_fp16(case, part, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    shape = (2, case["heads"][1], 704, case["d"])
    k = wide(shape, g, -6e4, 1.2e5, 0.4 if part != "values" else 0.0)
    v = wide(shape, g, -2e4, 1.3e5, 0.4 if part != "keys" else 0.0)
    cache = cache_of(k, v, case["heads"][0], case["bits"])
    q, kd, vd = inputs(cache, g, T)
    if part != "values":                     # logits of a few units against the far keys
        q = (q.float() * 1e-5).bfloat16()
    parents = trees("random", 2, T, g)
    got = tree(cache, parents, q, kd, vd)
    assert torch.isfinite(got).all()
    check(cache, parents, q, kd, vd, got)


def test_tree_over_a_group_flushed_past_fp16():
    """The group becomes one of far values by appending: the window's flush."""
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn(1, 2, 64, 64, generator=g, device="cuda")
    v = torch.randn(1, 2, 64, 64, generator=g, device="cuda")
    cache = cache_of(k, v, 4, 4, window=64, max_new=96)
    far = wide((1, 2, 96, 64), g, -2e4, 1.3e5, 1.0)
    for i in range(96):
        vn = far[:, :, i].bfloat16()[None].contiguous()
        kn = torch.randn(1, 1, 2, 64, generator=g, device="cuda").bfloat16()
        K.kvc_append_layers(cache, 0, 1, kn, vn)
    assert K.kvc_layer_info_get(cache, 0)["packed_tokens"] > 64
    q, kd, vd = inputs(cache, g, 6)
    parents = trees("random", 1, 6, g)
    got = tree(cache, parents, q, kd, vd)
    assert torch.isfinite(got).all()
    check(cache, parents, q, kd, vd, got)


def test_marked_units_beside_others_and_waits_that_give_up():
    """Some sequences of a call store values past fp16's range, others do not: those others' rows
    are what they are without them. Waits that give up leave nothing behind."""
    g = torch.Generator(device="cuda").manual_seed(8)
    k = torch.randn(6, 2, 2000, 64, generator=g, device="cuda")
    v = torch.randn(6, 2, 2000, 64, generator=g, device="cuda")
    q, kd, vd = None, None, None
    outs = []
    for far in (False, True):
        if far:
            v[1, 0, 700:900] = v[1, 0, 700:900].abs() * 3e4
            k[4, 1, 32:64, 3] = 1e5 * torch.rand(32, generator=g, device="cuda")
        cache = cache_of(k, v, 8, 4)
        if q is None:
            q, kd, vd = inputs(cache, g, 7)
            q[:, :, :, :, 3] *= 2.0 ** -14
        parents = trees("chain", 6, 7, g)
        outs.append(tree(cache, parents, q, kd, vd))
        check(cache, parents, q, kd, vd, outs[-1])
    same = [b for b in range(6) if b not in (1, 4)]
    assert torch.equal(outs[0][:, same], outs[1][:, same])
    for polls in (0, 1, 2):
        K.kvc_set_wait_limit(cache, polls)
        tree(cache, parents, q, kd, vd)
        torch.cuda.synchronize()
        K.kvc_set_wait_limit(cache, -1)
        try:
            tree(cache, parents, q, kd, vd)
            K.kvc_check_device(cache)
        except K.KvcError as e:
            assert e.status == 7
        assert torch.equal(tree(cache, parents, q, kd, vd), outs[1])


def test_a_sequence_after_one_of_far_values():
    """What a sequence's far values were does not show in the next one's results: the same bits
    as on a cache that has stored nothing else."""
    g = torch.Generator(device="cuda").manual_seed(12)
    k = 1e-2 * torch.randn(1, 2, 640, 64, generator=g, device="cuda")
    v = 1e-5 * torch.randn(1, 2, 640, 64, generator=g, device="cuda")
    far = wide((1, 2, 640, 64), g, -2e4, 1.3e5, 0.5)
    fresh = cache_of(k, v, 4, 4)
    used = cache_of(far, far, 4, 4)
    torch.cuda.synchronize()
    K.kvc_cache_reset(used)
    dims = fresh.dims
    K.kvc_prefill_compress(dims, [640], 0, None, k.bfloat16(), v.bfloat16(), used)
    q, kd, vd = inputs(fresh, g, 5)
    parents = trees("random", 1, 5, g)
    want = tree(fresh, parents, q, kd, vd)
    check(fresh, parents, q, kd, vd, want)
    assert torch.equal(tree(used, parents, q, kd, vd), want)
    qd = queries(fresh, g)
    lists = select(fresh, qd, 6)
    assert torch.equal(decode(used, qd, lists), decode(fresh, qd, lists))


# ----------------------------------------------- queries and keys past fp16's range
@pytest.mark.parametrize("case", WIDE, ids=[str(i) for i in range(len(WIDE))])
@pytest.mark.parametrize("q_scale,k_scale", [(1e-5, None), (1e5, 2e-3), (2.0 ** 40, 2.0 ** -9),
                                             (2.0 ** -20, 2.0 ** 9), (300.0, 0.05)])
def test_listed_decode_of_queries_and_keys_past_fp16(case, q_scale, k_scale):
    g = torch.Generator(device="cuda").manual_seed(6)
    H = case["heads"][1]
    shape = (2, H, 700, case["d"])
    k = (wide((2, H, 704, case["d"]), g, -6e4, 1.2e5, 0.4)[:, :, :700] if k_scale is None
         else torch.randn(shape, generator=g, device="cuda") * k_scale)
    v = torch.randn(shape, generator=g, device="cuda")
    cache = cache_of(k, v, case["heads"][0], case["bits"])
    q = queries(cache, g, q_scale)
    lists = select(cache, q, 12)
    assert torch.equal(lists.cpu(), expected_lists(cache, q, 12))
    got = decode(cache, q, lists)
    assert torch.isfinite(got).all()
    check_decode(cache, q, lists, got)


def check_decode_of_far_keys(cache, q, lists, got):
    """check_decode with the terms that ordinary keys leave below its own. A key is formed as
    (code - mid) S + mid S + Z, mid = 2^(b-1): terms that add up to K_c = |Z| + 2^b S per channel
    whatever the key itself is, so the products' roundings and the sums' go with sum_c |q_c| K_c. A
    query element is fp16 after its row was scaled to a largest of 1/4 at least: off by at most half
    a subnormal step, 2^-25, which is 2^-23 of the row's largest, against K_c again."""
    D = cache.dims
    H, gq, d = D.n_kv_heads, D.n_q_heads // D.n_kv_heads, D.head_dim
    keys, values, G, _, _ = contents(cache, 0)
    x = K.kvc_export_layer(cache, 0)
    bits = K.kvc_layer_info_get(cache, 0)["bits"]
    parts = x["k_zero"].double().abs() + 2 ** bits * x["k_scale"].double()
    for h in range(H):
        ids = lists[0, 0, h].long()
        ids = ids[(ids >= 0) & (ids < G)]
        rows = (ids[:, None] * 32 + torch.arange(32, device="cuda")).reshape(-1)
        rows = torch.cat([rows, torch.arange(G * 32, keys.shape[2], device="cuda")])
        qd = q[0, 0, h * gq:(h + 1) * gq].double()
        o = got[0, 0, h * gq:(h + 1) * gq].double()
        want, size, wv = attend(qd, keys[0, h, rows], values[0, h, rows])
        big = parts[0, h, ids] if len(ids) else torch.zeros(1, d, device="cuda").double()
        terms = (qd.abs() @ big.T).amax(-1, keepdim=True) / math.sqrt(d)
        most = qd.abs().amax(-1, keepdim=True) * big.sum(-1).amax() / math.sqrt(d)
        dx = sum_bound(torch.maximum(size, terms), d, 2.0 ** -21) + 2.0 ** -23 * most
        vmax = values[0, h, rows].abs().amax()
        tol = 2 * dx * wv.amax(-1, keepdim=True) + vmax * (2.0 ** -18 + len(rows) * U32)
        err = (o - want).abs()
        assert torch.all(err <= tol), (err.max().item(), (err / tol).max().item())


@pytest.mark.parametrize("bits,d", [(4, 128), (2, 64)])
def test_listed_decode_of_far_groups_flushed_and_far_values(bits, d):
    """Far keys that the window's flush packs, queries of ordinary size but for the far channels,
    and values past fp16's range."""
    g = torch.Generator(device="cuda").manual_seed(14)
    H, n = 2, 320
    k = torch.randn(1, H, n, d, generator=g, device="cuda")
    v = wide((1, H, n, d), g, -2e4, 1.3e5, 0.4)
    cache = cache_of(k, v, 8, bits, window=64, max_new=160)
    for _ in range(160):
        kn = torch.randn(1, 1, H, d, generator=g, device="cuda")
        kn[..., 5:9] = 1.2e5 * torch.rand(1, 1, H, 4, generator=g, device="cuda") - 6e4
        vn = torch.randn(1, 1, H, d, generator=g, device="cuda")
        K.kvc_append_layers(cache, 0, 1, kn.bfloat16(), vn.bfloat16())
    for spread in (1.0, 30.0, 1e-4):
        q = queries(cache, g, spread)
        q[..., 5:9] = (q[..., 5:9].float() * 3e-6).bfloat16()
        q[..., 6] = (q[..., 6].float() * 30).bfloat16()
        lists = select(cache, q, 9)
        assert torch.equal(lists.cpu(), expected_lists(cache, q, 9))
        got = decode(cache, q, lists)
        assert torch.isfinite(got).all()
        check_decode_of_far_keys(cache, q, lists, got)
    q = queries(cache, g)                    # products past fp16's range: one token takes all
    lists = select(cache, q, 14)
    got = decode(cache, q, lists)
    assert torch.isfinite(got).all()
    check_decode_of_far_keys(cache, q, lists, got)


# ----------------------------------------------------------------------- a dominant token
@pytest.mark.parametrize("heads,T", [((1, 1), 5), ((8, 1), 4), ((8, 1), 9)])
@pytest.mark.parametrize("gap", [13.3, 20.0, 26.0, 28.7])
def test_tree_with_a_dominant_token_of_no_value(heads, T, gap):
    """One token of value 0 takes nearly all the weight, 2^gap times that of each of the others:
    the output is what the others contribute. A weight is within 2^-32 of the largest of a row
    (or its own rounding) in the products."""
    B, n, d = 200, 4096, 64
    k = torch.zeros(B, 1, n, d, device="cuda")
    k[:, :, 0, 0] = 3.0                      # stored exactly: zero-point 0, scale 1, code 3
    v = torch.ones(B, 1, n, d, device="cuda")
    v[:, :, 0] = 0.0
    v[:, :, :, 32:] *= -0.5
    cache = cache_of(k, v, heads[0], 2)
    keys, values, G, _, _ = contents(cache, 0)
    assert torch.equal(keys[..., 0, 0], torch.full((B, 1), 3.0, device="cuda").double()) and G == 128
    q = torch.zeros(1, B, heads[0], T, d, device="cuda")
    q[..., 0] = gap * math.log(2.0) * math.sqrt(d) / 3.0
    q = q.bfloat16()
    kd = torch.zeros(1, B, 1, T, d, device="cuda").bfloat16()
    parents = trees("star", B, T, None)
    got = tree(cache, parents, q, kd, kd)
    qd = q[0, 0, 0, 0].double()
    kk = torch.cat([keys[0, 0], torch.zeros(1, d, device="cuda").double()])
    vv = torch.cat([values[0, 0], torch.zeros(1, d, device="cuda").double()])
    want, size, _ = attend(qd[None], kk, vv)
    # the logit's product is exact (both factors are), its scale takes two roundings of fp32 and
    # the weights' exponential 2^-22
    tol = want.abs() * (UB + 2 * (float(size.max()) * 8 * U32 + 2.0 ** -22) + U16)
    tol = tol + n * 2.0 ** -32 * vv.abs().amax(0)
    err = (got[0].double() - want).abs()
    assert torch.all(err <= tol), (err / tol).max().item()


# ------------------------------------------------------------------- queries that cancel
@pytest.mark.parametrize("order", [(2.0 ** 30, 1.0, -2.0 ** 30, 0.0), (1.0, 2.0 ** 30, 0.0, -2.0 ** 30),
                                   (2.0 ** 30, 2.0 ** -6, -2.0 ** 30, 1.0)])
@pytest.mark.parametrize("G", [200, 5000])
def test_selection_where_the_heads_queries_cancel(order, G):
    """Large queries of two heads cancel in the score's sum and leave another head's, over keys
    that are constant in each group (their bounds are one value)."""
    d = 64
    g = torch.Generator(device="cuda").manual_seed(G)
    base = torch.randn(1, 1, G, 1, d, generator=g, device="cuda")
    base[..., 1:] *= 2.0 ** -5               # the cancelling channel decides the order
    k = base.expand(1, 1, G, 32, d).reshape(1, 1, G * 32, d)
    cache = cache_of(k, torch.zeros_like(k), 4, 4)
    q = torch.randn(1, 1, 4, d, generator=g, device="cuda") * 0.5
    q[0, 0, :, 0] = torch.tensor(order, device="cuda")
    q = q.bfloat16()
    for kk in (1, 17, 64, G // 2):
        assert torch.equal(select(cache, q, kk).cpu(), expected_lists(cache, q, kk)), kk


# --------------------------------------------------- what an earlier sequence left behind
@pytest.mark.parametrize("bits,d", [(2, 64), (4, 128), (16, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_old_window_slots_reach_no_output(bits, d, bad):
    """A sequence whose values are not finite is followed by an ordinary one with fewer tokens in
    the window: the slots behind its last token, which still hold the old values, do not count."""
    n, H = 300, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    dims = K.make_dims(1, 1, 4, H, d, n, 0, 7, bits, 32, 64 if bits != 16 else 320, 4)
    k = torch.randn(1, H, n, d, generator=g, device="cuda").bfloat16()
    v = torch.randn(1, H, n, d, generator=g, device="cuda").bfloat16()
    dirty = v.clone()
    dirty[:, :, 256:] = bad
    cache = K.kvc_prefill_compress(dims, [n], 0, None, k, dirty)
    for kept in (257, 265, 270):
        K.kvc_cache_reset(cache)
        index = torch.arange(kept, dtype=torch.int32, device="cuda").expand(1, H, kept).contiguous()
        K.kvc_prefill_selected(cache, 0, index, kept, k, v)
        q = queries(cache, g)
        lists = select(cache, q, 8)
        got = decode(cache, q, lists)
        assert torch.isfinite(got).all()
        check_decode(cache, q, lists, got)
        full = torch.empty_like(got)
        K.kvc_decode_attn(cache, 0, 1, q, full)
        assert torch.isfinite(full).all()
        qt, kd, vd = inputs(cache, g, 3)
        parents = trees("chain", 1, 3, g)
        check(cache, parents, qt, kd, vd, tree(cache, parents, qt, kd, vd))
        K.kvc_cache_reset(cache)
        K.kvc_prefill_compress(dims, [n], 0, None, k, dirty, cache)
