"""Cases of the operators that bound what a long generation attends to.

Four operators stand beside the library's prefill and decode attention:

  prompt   attention of every prompt query over a sliding window and the first tokens (sinks), the
           layer's cache then made of the sinks and the most recent tokens (and read once, by the
           first generated token's query over the same window);
  window   the single-token form over a compressed cache: the first and the last cached tokens;
  weights  decode attention over the whole cache that also adds what attention every 32 cached
           tokens receive, summed over the query heads that share the kv head, to a running sum;
  evict    the groups of 32 tokens with the least accumulated weight leave: those that stay go, in
           order and with the window, to a smaller cache (which the next step then reads).

`run` computes them in elementary torch operations, or (own) by the library's calls, on a cache
made from the same keys and values.
"""
import math

import torch

own = False

GROUP = 32          # tokens of a packed group; channels of a value group
WINDOW = 128        # recent-window slots of a 2- or 4-bit cache
STEPS = 8           # decode steps that a cache is sized for


# ------------------------------------------------------------------------------------ the cases
def _case(name, op, layers, batch, q_heads, kv_heads, d, n, alpha, bits, **more):
    return dict(name=name, op=op, layers=layers, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
                d=d, n=n, alpha=alpha, bits=bits, **more)


def listed():
    return [
        # a short chat turn on a small model: what counts is the call's latency
        _case("prompt small", "prompt", 1, 1, 4, 4, 64, 528, 16, 2, sinks=4, window=128),
        # ragged length and window, eight query heads to a kv head, small heads, three sequences
        _case("prompt gqa8 odd", "prompt", 1, 3, 16, 2, 64, 20011, 31, 4, sinks=37, window=1000),
        # one layer of a 131,072-token prompt with the long-context heads (GQA 4)
        _case("prompt long", "prompt", 1, 1, 32, 8, 128, 131072, 32, 2, sinks=4, window=4096),
        _case("window small", "window", 1, 1, 4, 4, 64, 528, 16, 2, sinks=4, window=128),
        # a window layer over a 131,072-token prompt kept whole at 2 bits
        _case("window long 2-bit", "window", 1, 1, 32, 8, 128, 131072, 64, 2, sinks=4, window=4096),
        # the 4 x 32,768-token workload (40 heads, 4 bits); edges inside groups
        _case("window mha 4-bit", "window", 1, 4, 40, 40, 128, 32768, 0, 4, sinks=45, window=8005),
        # a 16-bit cache (every token exact) of a small batch: two layers, one call
        _case("weights 16-bit", "weights", 2, 2, 8, 2, 64, 777, 9, 16),
        _case("weights gqa8 odd", "weights", 2, 3, 16, 2, 64, 20011, 37, 4),
        _case("weights mha 4-bit", "weights", 1, 4, 40, 40, 128, 32768, 0, 4),
        # a short cache halved
        _case("evict small", "evict", 1, 1, 4, 4, 64, 528, 16, 2, keep=8, recent=1),
        # a 131,072-token prompt kept whole at 2 bits, a quarter of it stays
        _case("evict long 2-bit", "evict", 1, 1, 32, 8, 128, 131072, 64, 2, keep=1024, recent=32),
        # 160 units at 4 bits, half of every one stays
        _case("evict mha 4-bit", "evict", 1, 4, 40, 40, 128, 32768, 0, 4, keep=512, recent=4),
    ]


def draw(rng):
    """One more case: lengths, heads, windows and budgets over the listed ones' ranges."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prompt", "window", "weights", "evict"])
    g = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    kv_heads = log_int(1, 40 if g == 1 else 8)
    batch = log_int(1, 4)
    layers = 1 if op == "prompt" else rng.choice([1, 1, 2])
    bits = rng.choice([2, 4]) if op == "prompt" else rng.choice([2, 4, 4, 16])
    alpha = rng.choice([1, 16, 31, 32] if op == "prompt" else [0, 1, 16, 32, rng.randint(2, 90)])
    units = layers * batch * kv_heads
    if op == "prompt":
        # query rows and visible pairs of the call, at most what the largest listed case has
        n = max(alpha + 1, log_int(40, min(131072, 4_000_000 // (units * g))))
        window = log_int(1, max(1, min(2 * n, 16_000_000_000 // (units * g * n), 65536)))
        return dict(op=op, layers=layers, batch=batch, q_heads=g * kv_heads, kv_heads=kv_heads, d=d, n=n,
                    alpha=alpha, bits=bits, sinks=rng.choice([0, 1, 4, log_int(1, 100)]), window=window)
    # tokens of all units together, at most half of what the largest listed case holds
    most = min(131072 if bits != 16 else 32768, 2_600_000 // units)
    n = max(alpha + 1, log_int(40, most))
    case = dict(op=op, layers=layers, batch=batch, q_heads=g * kv_heads, kv_heads=kv_heads, d=d,
                n=n, alpha=alpha, bits=bits)
    if op == "window":
        case["sinks"] = rng.choice([0, 1, 4, log_int(1, 200)])
        case["window"] = log_int(1, 2 * n)
    elif op == "evict":
        case["keep"] = log_int(1, max(1, n // GROUP))
        case["recent"] = min(case["keep"], rng.choice([0, 1, log_int(1, 32)]))
    return case


def _spread(case):
    """Tokens of a prompt kept whole: packed groups, and tokens in the exact window."""
    groups = 0 if case["bits"] == 16 else (case["n"] - case["alpha"]) // GROUP
    return groups, case["n"] - groups * GROUP


def _evictable(case):
    groups, exact = _spread(case)
    return exact // GROUP if case["bits"] == 16 else groups


def _slots(case):
    """Groups of 32 cached tokens of a layer, the window's last one begun."""
    groups, exact = _spread(case)
    return groups + (exact + GROUP - 1) // GROUP


# ------------------------------------------------------------------------------------ the inputs
def _draws(case, seed):
    """Keys, values and queries of a case: key channels of different spreads (log-normal), queries
    with a direction of their head, standard normal values; rounded once to bf16. Accumulated
    weights are log-normal, about a step's worth, some of them equal (groups that received nothing)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    L, B, Hq, H, d, n = (case[x] for x in ("layers", "batch", "q_heads", "kv_heads", "d", "n"))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    sigma = torch.exp(0.5 * normal(L, 1, H, 1, d))
    k = torch.stack([(normal(B, H, n, d) * sigma[layer]).bfloat16() for layer in range(L)])
    v = torch.stack([normal(B, H, n, d).bfloat16() for layer in range(L)])
    u = normal(L, 1, H, 1, d)
    u = 2 * u / u.norm(dim=-1, keepdim=True)
    out = {"k": k, "v": v}
    out["q"] = (normal(L, B, H, Hq // H, d) + u).bfloat16().reshape(L, B, Hq, d)
    if case["op"] == "prompt":
        rows = [(normal(B, Hq // H, n, d) + u[0, :, h, :, None]).bfloat16() for h in range(H)]
        out["q_full"] = torch.stack(rows, 1).reshape(B, Hq, n, d)
    if case["op"] in ("weights", "evict"):
        a = torch.exp(1.5 * normal(L, B, H, _slots(case))) * (Hq // H) / _slots(case)
        out["before"] = torch.where(torch.rand(a.shape, generator=g, device="cuda") < 0.1, 0.0, a)
    return out


def _pack(x, groups_axis, bits):
    """Group quantization along an axis of length 32: codes (uint8), fp16 scale and zero-point."""
    x = x.float()
    lo, hi = x.amin(groups_axis, keepdim=True), x.amax(groups_axis, keepdim=True)
    scale = ((hi - lo) / float(2 ** bits - 1)).half()
    zero = lo.half()
    s = scale.float()
    codes = torch.where(s == 0, torch.zeros_like(x), torch.round((x - zero.float()) / s))
    codes = codes.clamp(0, 2 ** bits - 1).to(torch.uint8)
    return codes, scale.squeeze(groups_axis), zero.squeeze(groups_axis)


def _arrays(bits, packed, k, v):
    """A compressed cache of the tokens k, v as arrays: the first `packed` in groups (keys per
    channel over 32 tokens, values per token over 32 channels), the others exact."""
    L, B, H, n, d = k.shape
    G = packed // GROUP
    store = {"win_k": k[..., packed:, :].contiguous(), "win_v": v[..., packed:, :].contiguous()}
    ks, vs = [], []
    for layer in range(L):
        if G:
            ks.append(_pack(k[layer, :, :, :packed].reshape(B, H, G, GROUP, d), 3, bits))
            vs.append(_pack(v[layer, :, :, :packed].reshape(B, H, G, GROUP, d // GROUP, GROUP), 5, bits))
    if G:
        for name, parts in (("k", ks), ("v", vs)):
            for j, what in enumerate(("codes", "scale", "zero")):
                store[name + "_" + what] = torch.stack([p[j] for p in parts])
    store["n_groups"] = G
    return store


def _budget(case):
    """Prompt tokens kept beside the observation tokens: the sinks and a window's worth."""
    return min(case["n"] - case["alpha"], case["sinks"] + case["window"])


def _dims(case, n):
    """Dimensions of a cache of prompts of n tokens."""
    import kv_cache_compression_snapkv_gb300 as kvc
    bits = case["bits"]
    window = WINDOW if bits != 16 else (n + STEPS + 31) // 32 * 32
    return kvc.make_dims(case["layers"], case["batch"], case["q_heads"], case["kv_heads"],
                         case["d"], n, case["alpha"], 7, bits, GROUP, window, STEPS)


def _cache(case, k, v):
    """The prompt kept whole, as the library's handle."""
    import kv_cache_compression_snapkv_gb300 as kvc
    dims = _dims(case, case["n"])
    budgets = [case["n"]] * case["layers"]
    cache = kvc.kvc_cache_create(dims, budgets)
    for layer in range(case["layers"]):
        kvc.kvc_prefill_compress(dims, budgets, layer, None, k[layer], v[layer], cache)
    torch.cuda.current_stream().synchronize()   # k and v are dropped by the caller
    return cache


def prepare(case, seed):
    """What a program has before the call: a prompt's queries, keys and values and an empty cache; or
    the prompt's compressed cache (the library's handle, or the same contents as arrays: what each
    side's program keeps between steps), the step's queries and the accumulated weights."""
    state = _draws(case, seed)
    L, B, Hq, H, d = (case[x] for x in ("layers", "batch", "q_heads", "kv_heads", "d"))
    if case["op"] == "prompt":
        if own:
            import kv_cache_compression_snapkv_gb300 as kvc
            state["cache"] = kvc.kvc_cache_create(_dims(case, case["n"]), [_budget(case)])
    else:
        k, v = state.pop("k"), state.pop("v")
        if own:
            state["cache"] = _cache(case, k, v)
        else:
            state["store"] = _arrays(case["bits"], _spread(case)[0] * GROUP, k, v)
    if own:
        import kv_cache_compression_snapkv_gb300 as kvc
        state["out"] = torch.empty(L, B, Hq, d, dtype=torch.float32, device="cuda")
        if case["op"] == "prompt":
            state["x_out"] = torch.empty_like(state["q_full"])
        if "before" in state:
            state["after"] = torch.empty_like(state["before"])
        if case["op"] == "evict":
            # a cache for what stays: n_keep groups, the observation tokens or more of the window
            n = GROUP * (case["keep"] + 1) + case["alpha"]
            state["small"] = kvc.kvc_cache_create(_dims(case, n), [n] * L)
            state["groups"] = torch.empty(L, B, H, case["keep"], dtype=torch.int32, device="cuda")
            state["stay"] = torch.empty_like(state["before"])
    state["case"] = case
    return state


# ------------------------------------------------------------------------------------ one pass
def _keys(store):
    return store["k_codes"].float() * store["k_scale"].float().unsqueeze(4) + store["k_zero"].float().unsqueeze(4)


def _values(store):
    x = store["v_codes"].float() * store["v_scale"].float().unsqueeze(-1) + store["v_zero"].float().unsqueeze(-1)
    return x.flatten(-2)


def _tokens(store):
    keys, values = store["win_k"].float(), store["win_v"].float()
    if store["n_groups"]:
        keys = torch.cat([_keys(store).flatten(3, 4), keys], 3)
        values = torch.cat([_values(store).flatten(3, 4), values], 3)
    return keys, values


def _attend(q, keys, values):
    """One query per head over all the given tokens: outputs and softmax weights."""
    L, B, Hq, d = q.shape
    H = keys.shape[2]
    x = q.float().reshape(L, B, H, Hq // H, d) @ keys.transpose(-1, -2) / math.sqrt(d)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return (p @ values).reshape(L, B, Hq, d), p


def _decode_window(store, q, sinks, window):
    """The first `sinks` and the last `window` cached tokens: only the groups that hold one of them
    are unpacked."""
    G, exact = store["n_groups"], store["win_k"].shape[3]
    T = G * GROUP + exact
    first = max(0, T - window)
    group = torch.arange(G, device=q.device)
    read = (group * GROUP < sinks) | (group * GROUP + GROUP > first)
    at = torch.arange(T, device=q.device)
    held = torch.cat([read.repeat_interleave(GROUP), torch.ones(exact, dtype=torch.bool, device=q.device)])
    part = {x: y[:, :, :, read] for x, y in store.items() if x[:2] in ("k_", "v_")}
    part.update(win_k=store["win_k"], win_v=store["win_v"], n_groups=int(read.sum()))
    keys, values = _tokens(part)
    seen = ((at < sinks) | (at >= first))[held]
    return _attend(q, keys[:, :, :, seen], values[:, :, :, seen])[0]


def _decode_weights(store, q, before):
    """The whole cache; every 32 tokens' weights (of all the kv head's query heads) are added."""
    out, p = _attend(q, *_tokens(store))
    p = p.sum(3)
    p = torch.nn.functional.pad(p, (0, -p.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP)).sum(-1)
    return out, before + torch.nn.functional.pad(p, (0, before.shape[-1] - p.shape[-1]))


def _evict(store, bits, keep, recent, weights):
    """The `keep` groups of the largest weights (ties to the lower index, the `recent` newest in any
    case), in order; a 16-bit cache's groups are its window's whole ones."""
    exact = store["win_k"].shape[3]
    E = exact // GROUP if bits == 16 else store["n_groups"]
    rank = weights[..., :E].clone()
    rank[..., max(0, E - recent):] = math.inf
    m = min(keep, E)
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :m].sort(-1).values
    groups = torch.nn.functional.pad(ids, (0, keep - m), value=-1).to(torch.int32)
    stay = torch.cat([weights.gather(-1, ids), weights[..., E:]], -1)
    stay = torch.nn.functional.pad(stay, (0, weights.shape[-1] - stay.shape[-1]))

    def pick(x, rows):      # rows `ids` of axis 3, in pieces of `rows`
        x = x if rows == 1 else x[:, :, :, :E * rows].unflatten(3, (E, rows))
        index = ids.reshape(*ids.shape, *[1] * (x.dim() - 4)).expand(*ids.shape, *x.shape[4:])
        x = x.gather(3, index)
        return x if rows == 1 else x.flatten(3, 4)

    if bits == 16:
        small = {x: torch.cat([pick(store[x], GROUP), store[x][:, :, :, E * GROUP:]], 3) for x in ("win_k", "win_v")}
        small["n_groups"] = 0
    else:
        small = {x: pick(y, 1) for x, y in store.items() if x[:2] in ("k_", "v_")}
        small.update(win_k=store["win_k"], win_v=store["win_v"], n_groups=m)
    return groups, stay, small


def _prompt(q, k, v, sinks, window):
    """Sliding-window attention with sinks, one kv head at a time (the logits of all would not fit).
    Queries are taken in blocks of C >= window, which see their own and the previous block's keys."""
    B, Hq, n, d = q.shape
    H = k.shape[1]
    C = min(max(window, 256), n)
    nb = -(-n // C)
    s = min(sinks, n)
    i = torch.arange(nb * C, device=q.device).reshape(nb, C, 1)
    j = (torch.arange(nb, device=q.device) * C - C).reshape(nb, 1, 1) + torch.arange(2 * C, device=q.device)
    near = (j <= i) & (i - j < window) & (j >= s) & (j < n)
    far = torch.arange(s, device=q.device) <= i
    out = torch.empty_like(q)

    def blocks(x):          # [B, n, d] as [B, nb, 2 C, d]: the previous block's rows before its own
        x = torch.nn.functional.pad(x.float(), (0, 0, C, nb * C - n)).reshape(B, nb + 1, C, d)
        return torch.cat([x[:, :-1], x[:, 1:]], 2)

    g = Hq // H
    for h in range(H):
        kb, vb = blocks(k[:, h]).unsqueeze(2), blocks(v[:, h]).unsqueeze(2)
        qb = torch.nn.functional.pad(q[:, h * g:(h + 1) * g].float(), (0, 0, 0, nb * C - n))
        qb = qb.reshape(B, g, nb, C, d).transpose(1, 2) / math.sqrt(d)
        x = (qb @ kb.transpose(-1, -2)).masked_fill_(~near.unsqueeze(1), -math.inf)
        y = (qb @ k[:, h, :s].float().transpose(-1, -2)[:, None, None]).masked_fill_(~far.unsqueeze(1), -math.inf)
        top = torch.cat([x.amax(-1, keepdim=True), y], -1).amax(-1, keepdim=True).clamp_(min=-1e30)
        x, y = x.sub_(top).exp_(), y.sub_(top).exp_()
        o = x @ vb + y @ v[:, h, :s].float()[:, None, None]
        o = o / (x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True))
        out[:, h * g:(h + 1) * g] = o.transpose(1, 2).reshape(B, g, nb * C, d)[:, :, :n].bfloat16()
        del x, y, o
    return out


def _sinks_cache(case, k, v):
    """The cache of the sinks and the most recent tokens of a prompt."""
    n, alpha, b = case["n"], case["alpha"], _budget(case)
    s = min(case["sinks"], b)
    rest = n - alpha - (b - s)
    k, v = (torch.cat([x[:, :, :s], x[:, :, rest:]], 2).unsqueeze(0) for x in (k, v))
    return _arrays(case["bits"], b // GROUP * GROUP, k, v)


def run(state):
    case = state["case"]
    layers, op = case["layers"], case["op"]
    if own:
        import kv_cache_compression_snapkv_gb300 as kvc
        cache, q, out = state["cache"], state["q"], state["out"]
        if op == "prompt":
            kvc.kvc_cache_reset(cache)
            kvc.kvc_prefill_window(cache, 0, case["sinks"], case["window"], state["q_full"], state["k"][0],
                                   state["v"][0], state["x_out"])
            kvc.kvc_decode_window(cache, 0, 1, case["sinks"], case["window"], q, out)
            return {"x_out": state["x_out"], "first": out}
        if op == "window":
            kvc.kvc_decode_window(cache, 0, layers, case["sinks"], case["window"], q, out)
            return {"out": out}
        slots = state["before"].shape[-1]
        if op == "weights":
            kvc.kvc_decode_weights(cache, 0, layers, q, slots, state["before"], state["after"], out)
            return {"out": out, "weights": state["after"]}
        kvc.kvc_cache_reset(state["small"])
        kvc.kvc_evict_groups(cache, state["small"], 0, layers, case["keep"], case["recent"], slots,
                             state["before"], state["stay"], state["groups"])
        kvc.kvc_decode_weights(state["small"], 0, layers, q, slots, state["stay"], state["after"], out)
        return {"groups": state["groups"], "out": out, "weights": state["after"]}
    q = state["q"]
    if op == "prompt":
        x_out = _prompt(state["q_full"], state["k"][0], state["v"][0], case["sinks"], case["window"])
        store = _sinks_cache(case, state["k"][0], state["v"][0])
        return {"x_out": x_out, "first": _decode_window(store, q, case["sinks"], case["window"])}
    if op == "window":
        return {"out": _decode_window(state["store"], q, case["sinks"], case["window"])}
    if op == "weights":
        out, after = _decode_weights(state["store"], q, state["before"])
        return {"out": out, "weights": after}
    groups, stay, small = _evict(state["store"], case["bits"], case["keep"], case["recent"], state["before"])
    out, after = _decode_weights(small, q, stay)
    return {"groups": groups, "out": out, "weights": after}


# ------------------------------------------------------------------------------------ floors
def _seen(n, sinks, window):
    """Visible (query, key) pairs of a head: min(i + 1, window) in the window, and the sinks before it."""
    w = min(window, n)
    near = w * (w + 1) // 2 + (n - w) * w
    m = n - w                       # queries with m' = 1 .. m keys before their window
    s = min(sinks, m)
    return near + s * (s + 1) // 2 + (m - s) * s


def work(case):
    L, B, Hq, H, d, n = (case[x] for x in ("layers", "batch", "q_heads", "kv_heads", "d", "n"))
    bits, g, units = case["bits"], Hq // H, L * B * H
    block = 8 * d * (bits + 1)
    step = 6 * L * B * Hq * d       # a step's queries and outputs
    if case["op"] == "prompt":
        # prompt and outputs; what the cache keeps, written and read again by the first query
        kept = _budget(case)
        cache = units * (kept // GROUP * block + (kept % GROUP + case["alpha"]) * 4 * d)
        return {"bytes": 4 * B * (Hq + H) * n * d + 2 * cache + step,
                "flops": 4 * d * B * Hq * (_seen(n, case["sinks"], case["window"]) + min(n, case["sinks"] + case["window"]))}
    groups, exact = _spread(case)
    if case["op"] == "window":
        T = groups * GROUP + exact
        first = max(0, T - case["window"])
        s = min(case["sinks"], T)
        read = groups if first // GROUP <= (s + GROUP - 1) // GROUP else \
            min(groups, (s + GROUP - 1) // GROUP) + max(0, groups - first // GROUP)
        tail = exact - max(0, min(exact, first - groups * GROUP)) + max(0, min(s, first) - groups * GROUP)
        return {"bytes": units * (read * block + tail * 4 * d) + step,
                "flops": 4 * d * g * units * min(T, s + T - first)}
    if case["op"] == "weights":
        return {"bytes": units * (groups * block + exact * 4 * d + 8 * _slots(case)) + step,
                "flops": 4 * d * g * units * n}
    # what stays is read, written and read again by the step; the weights and lists
    m = min(case["keep"], _evictable(case))
    if bits == 16:
        stay = (exact - (_evictable(case) - m) * GROUP) * 4 * d
        tokens = exact - (_evictable(case) - m) * GROUP
    else:
        stay = m * block + exact * 4 * d
        tokens = m * GROUP + exact
    return {"bytes": units * (3 * stay + 16 * _slots(case) + 4 * case["keep"]) + step,
            "flops": 4 * d * g * units * tokens}


# ------------------------------------------------------------------------------------ 64 bits
def _exact_group(x, bits):
    """What a group of 32 values (last axis) stands for once stored, in 64 bits: the quantizer's
    own roundings (32-bit differences and quotients, 16-bit scale and zero-point) and no other."""
    x = x.to(torch.float64)
    levels = 2 ** bits - 1
    least, most = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    step = ((most - least).float().double() / levels).float().half().double()
    base = least.float().half().double()
    ratio = ((x - base).float().double() / step).float().double()
    code = torch.nan_to_num(torch.round(ratio), nan=0.0, posinf=0.0, neginf=0.0)
    code = torch.minimum(torch.maximum(code, torch.zeros_like(code)), torch.full_like(code, levels))
    return base + step * code


def _exact_unit(case, k, v, m):
    """Keys and values of one (layer, sequence, kv head) as stored, the first m tokens packed."""
    d = k.shape[-1]
    kt = _exact_group(k[:m].reshape(-1, GROUP, d).transpose(1, 2), case["bits"]) if m else k[:0].double()
    vt = _exact_group(v[:m].reshape(m, d // GROUP, GROUP), case["bits"]) if m else v[:0].double()
    kt = kt.transpose(1, 2).reshape(m, d) if m else kt
    return torch.cat([kt, k[m:].double()]), torch.cat([vt.reshape(m, d), v[m:].double()])


def _exact_prompt(case, x):
    """Rows in blocks of 1024 queries, each over the keys from its first row's window on and the sinks."""
    B, Hq, H, d, n = (case[c] for c in ("batch", "q_heads", "kv_heads", "d", "n"))
    s, W, g = case["sinks"], case["window"], Hq // H
    out = torch.empty(B, Hq, n, d, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            k, v = x["k"][0, b, h].double(), x["v"][0, b, h].double()
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                j0 = max(0, i0 - W + 1)
                j = torch.cat([torch.arange(min(s, j0)), torch.arange(j0, i1)]).cuda()
                i = torch.arange(i0, i1, device="cuda")[:, None]
                hide = (j > i) | ((i - j >= W) & (j >= s))
                q = x["q_full"][b, h * g:(h + 1) * g, i0:i1].double()
                x_ = (q @ k[j].T / math.sqrt(d)).masked_fill(hide, -math.inf)
                out[b, h * g:(h + 1) * g, i0:i1] = torch.softmax(x_, -1) @ v[j]
    return out


def exact(case, seed):
    x = _draws(case, seed)
    L, B, Hq, H, d, n = (case[c] for c in ("layers", "batch", "q_heads", "kv_heads", "d", "n"))
    g, op, bits = Hq // H, case["op"], case["bits"]
    if op == "prompt" and 4 * d * B * Hq * n * (min(n, case["window"]) + 1024 + case["sinks"]) > 1.2e13:
        return None
    outs, sums, lists = [], [], []
    for layer in range(L):
        for b in range(B):
            for h in range(H):
                k, v = x["k"][layer, b, h], x["v"][layer, b, h]
                q = x["q"][layer, b, h * g:(h + 1) * g].double()
                if op == "prompt":
                    m = min(n - case["alpha"], case["sinks"] + case["window"])
                    first = min(case["sinks"], m)
                    keep = torch.cat([torch.arange(first), torch.arange(n - case["alpha"] - m + first, n)]).cuda()
                    keys, values = _exact_unit(case, k[keep], v[keep], m // GROUP * GROUP)
                else:
                    packed = 0 if bits == 16 else (n - case["alpha"]) // GROUP * GROUP
                    keys, values = _exact_unit(case, k, v, packed)
                slot = torch.arange(len(keys), device="cuda") // GROUP
                if op in ("prompt", "window"):
                    at = torch.arange(len(keys), device="cuda")
                    seen = (at < case["sinks"]) | (at >= len(keys) - case["window"])
                    keys, values = keys[seen], values[seen]
                if op in ("weights", "evict"):
                    total = x["before"][layer, b, h].double()
                if op == "evict":
                    E = n // GROUP if bits == 16 else packed // GROUP
                    order = sorted(range(E), key=lambda i, w=total.tolist(): (i < E - case["recent"], -w[i], i))
                    stay = sorted(order[:case["keep"]])
                    lists.append(torch.tensor(stay + [-1] * (case["keep"] - len(stay)), dtype=torch.int32))
                    stay = stay + list(range(E, len(total)))
                    rows = torch.nonzero(torch.isin(slot, torch.tensor(stay, device="cuda"))).reshape(-1)
                    keys, values = keys[rows], values[rows]
                    # the groups that stay are full but the last one
                    slot = torch.arange(len(rows), device="cuda") // GROUP
                    left = total[stay]
                    total = torch.zeros_like(total)
                    total[:len(stay)] = left
                p = torch.softmax(q @ keys.T / math.sqrt(d), -1)
                outs.append(p @ values)
                if op in ("weights", "evict"):
                    sums.append(total.index_add(0, slot, p.sum(0)))
    first = torch.stack(outs).reshape(L, B, Hq, d)
    if op == "prompt":
        return {"x_out": _exact_prompt(case, x), "first": first}
    if op == "window":
        return {"out": first}
    found = {"out": first, "weights": torch.stack(sums).reshape(x["before"].shape)}
    if op == "evict":
        found["groups"] = torch.stack(lists).reshape(L, B, H, case["keep"])
    return found
