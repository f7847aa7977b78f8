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
