"""A compressed cache and its contents as 64-bit arrays, for the tests of the calls that read
listed groups or many queries at a time: plain forms in float64 and the error bounds that
follow from the kernels' roundings."""
from __future__ import annotations

import math

import torch

import kv_cache_compression_snapkv_gb300 as K

U16, UB, U32 = 2.0 ** -11, 2.0 ** -8, 2.0 ** -24     # half a step of fp16, bf16, fp32


def make_cache(seed, layers=1, batch=1, q_heads=4, kv_heads=2, d=128, n=300, alpha=16, bits=2,
               window=64, appended=0, max_new=None, layer_bits=None, scale=1.0):
    """A cache of a prompt kept whole (packed groups, then the window), with `appended` tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    max_new = max(appended, 1) if max_new is None else max_new
    if bits == 16:
        window = (n + max_new + 31) // 32 * 32
    dims = K.make_dims(layers, batch, q_heads, kv_heads, d, n, alpha, 7, bits, 32, window, max_new)
    budgets = [n] * layers
    cache = (K.kvc_cache_create_layers(dims, budgets, layer_bits) if layer_bits
             else K.kvc_cache_create(dims, budgets))
    for layer in range(layers):
        k = (scale * torch.randn(batch, kv_heads, n, d, generator=g, device="cuda")).bfloat16()
        v = torch.randn(batch, kv_heads, n, d, generator=g, device="cuda").bfloat16()
        K.kvc_prefill_compress(dims, budgets, layer, None, k, v, cache)
    for _ in range(appended):
        kn = (scale * torch.randn(layers, batch, kv_heads, d, generator=g, device="cuda")).bfloat16()
        vn = torch.randn(layers, batch, kv_heads, d, generator=g, device="cuda").bfloat16()
        K.kvc_append_layers(cache, 0, layers, kn, vn)
    torch.cuda.synchronize()
    return cache, g


def contents(cache, layer):
    """Keys and values [B][H][tokens][d] in float64 (packed ones dequantized, then the window,
    oldest first), the number of packed groups, and each group's lower and upper key bounds."""
    x = K.kvc_export_layer(cache, layer)
    torch.cuda.synchronize()
    bits = K.kvc_layer_info_get(cache, layer)["bits"]
    B, H, T, d = x["k_codes"].shape
    G = T // 32
    lo = x["k_zero"].double()
    hi = lo + (2 ** bits - 1) * x["k_scale"].double()
    kc = x["k_codes"].double().reshape(B, H, G, 32, d)
    kp = (kc * x["k_scale"].double()[:, :, :, None] + lo[:, :, :, None]).reshape(B, H, T, d)
    vc = x["v_codes"].double().reshape(B, H, T, d // 32, 32)
    vp = (vc * x["v_scale"].double()[..., None] + x["v_zero"].double()[..., None]).reshape(B, H, T, d)
    return (torch.cat([kp, x["win_k"].double()], 2), torch.cat([vp, x["win_v"].double()], 2),
            G, lo, hi)


def attend(q, keys, values, seen=None):
    """softmax(q k / sqrt d) v in float64 over the last two axes; rows that see nothing are 0.
    Also sum_c |q_c k_c| / sqrt(d) of the worst seen pair per row, and the largest |v|."""
    d = q.shape[-1]
    x = q @ keys.transpose(-1, -2) / math.sqrt(d)
    if seen is None:
        seen = torch.ones_like(x, dtype=torch.bool)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - top.masked_fill(top == -math.inf, 0.0)).masked_fill(~seen, 0.0)
    s = w.sum(-1, keepdim=True)
    w = w / s.masked_fill(s == 0, 1.0)
    size = (q.abs() @ keys.abs().transpose(-1, -2) / math.sqrt(d)).masked_fill(~seen, 0.0)
    return w @ values, size.amax(-1, keepdim=True), w @ values.abs()


def sum_bound(size, d, unit):
    """How far a logit may be off: a dot product of d terms whose operands carry one rounding
    of `unit` each, accumulated in fp32, for terms that add up to `size` in magnitude."""
    return size * (2 * unit + d * U32)
