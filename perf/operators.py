"""Cases of the operators that read a compressed cache selectively or many queries at a time.

Three operators stand beside the library's decode attention:

  select_groups  per (sequence, kv head), the packed groups of 32 tokens that can matter most to
                 the step's queries, by an upper bound formed from the groups' stored key scales
                 and zero-points (a group's per-channel minimum and maximum);
  decode_groups  decode attention over the listed groups and the exact recent window;
  tree_attn      attention of a tree of drafted tokens over the cache, the window and each node's
                 own ancestors.

`run` computes them in elementary torch operations, or (own) by the library's calls, on a cache
made from the same keys and values.
"""
import math

import torch

own = False

GROUP = 32          # tokens of a packed group; channels of a value group
WINDOW = 128        # recent-window slots of a 2- or 4-bit cache


# ------------------------------------------------------------------------------------ the cases
def _case(name, op, layers, batch, q_heads, kv_heads, d, n, alpha, bits, **more):
    return dict(name=name, op=op, layers=layers, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
                d=d, n=n, alpha=alpha, bits=bits, **more)


def listed():
    return [
        # a short chat turn on a small model: what counts is the call's latency
        _case("select small", "select", 1, 1, 4, 4, 64, 528, 16, 2, k=4),
        # one layer of a 131,072-token prompt kept whole at 2 bits, GQA 4 (the long-context heads)
        _case("select long 2-bit", "select", 1, 1, 32, 8, 128, 131072, 64, 2, k=64),
        # one layer of the 4 x 32,768-token quantize-only workload (40 heads, 4 bits)
        _case("select mha 4-bit", "select", 1, 4, 40, 40, 128, 32768, 0, 4, k=64),
        # a ragged length, eight query heads to a kv head, small heads, two layers at once
        _case("select gqa8 odd", "select", 2, 3, 16, 2, 64, 20011, 37, 4, k=33),
        _case("decode small", "decode", 1, 1, 4, 4, 64, 528, 16, 2, k=4),
        _case("decode long 2-bit", "decode", 1, 1, 32, 8, 128, 131072, 64, 2, k=64),
        _case("decode mha 4-bit", "decode", 1, 4, 40, 40, 128, 32768, 0, 4, k=64),
        # lists with unused entries (-1) and in no order, a ragged length
        _case("decode gqa8 odd", "decode", 2, 3, 16, 2, 64, 20011, 37, 4, k=33),
        # a single drafted token over a 16-bit cache
        _case("tree one node 16-bit", "tree", 1, 1, 8, 2, 64, 777, 9, 16, t=1),
        # a drafted tree over the 512 + 32 kept tokens of a compressed 8-kv-head layer
        _case("tree kept 512", "tree", 1, 1, 32, 8, 128, 544, 32, 2, t=26),
        # the largest tree over a 131,072-token prompt kept whole at 2 bits
        _case("tree long 2-bit", "tree", 1, 1, 32, 8, 128, 131072, 64, 2, t=64),
        # four sequences with trees of different sizes over 32,768 tokens at 4 bits
        _case("tree mha 4-bit", "tree", 1, 4, 40, 40, 128, 32768, 0, 4, t=16),
    ]


def draw(rng):
    """One more case: lengths, heads and list or tree sizes over the listed ones' ranges."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["select", "decode", "tree", "tree"])
    g = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    kv_heads = log_int(1, 40 if g == 1 else 8)
    batch = log_int(1, 4)
    layers = rng.choice([1, 1, 2])
    bits = rng.choice([2, 4, 4, 16] if op == "tree" else [2, 4])
    alpha = rng.choice([0, 1, 16, 32, rng.randint(2, 90)])
    # tokens of all units together, at most half of what the largest listed case holds
    units = layers * batch * kv_heads
    most = min(131072 if bits != 16 else 32768, 2_600_000 // units)
    n = max(alpha + 1, log_int(40, most))
    case = dict(op=op, layers=layers, batch=batch, q_heads=g * kv_heads, kv_heads=kv_heads, d=d,
                n=n, alpha=alpha, bits=bits)
    if op == "tree":
        t = log_int(1, 64)
        # logits of the whole call, at most half of the largest listed case's
        t = max(1, min(t, 130_000_000 // (units * g * n)))
        case["t"] = t
    else:
        case["k"] = log_int(1, 96)
    return case


# ------------------------------------------------------------------------------------ the inputs
def _draws(case, seed):
    """Keys, values and queries of a case: key channels of different spreads (log-normal), queries
    with a direction of their head, standard normal values; rounded once to bf16."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    L, B, Hq, H, d, n = (case[x] for x in ("layers", "batch", "q_heads", "kv_heads", "d", "n"))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    sigma = torch.exp(0.5 * normal(L, 1, H, 1, d))
    k = torch.stack([(normal(B, H, n, d) * sigma[layer]).bfloat16() for layer in range(L)])
    v = torch.stack([normal(B, H, n, d).bfloat16() for layer in range(L)])
    u = normal(L, 1, H, 1, 1, d)
    u = 2 * u / u.norm(dim=-1, keepdim=True)
    rows = case.get("t", 1)
    q = (normal(L, B, H, Hq // H, rows, d) + u).bfloat16().reshape(L, B, Hq, rows, d)
    out = {"k": k, "v": v, "q": q if "t" in case else q[:, :, :, 0].contiguous()}
    if "t" in case:
        out["k_draft"] = (normal(L, B, H, rows, d) * sigma).bfloat16()
        out["v_draft"] = normal(L, B, H, rows, d).bfloat16()
        # node i hangs from a node before it or from the last cached token (-1); sequence b > 0
        # has fewer nodes, the rest is padding (-2)
        i = torch.arange(rows, device="cuda")
        r = torch.rand(B, rows, generator=g, device="cuda")
        parents = torch.floor(r * (i + 1)).to(torch.int32).clamp(max=rows - 1) - 1
        parents = torch.minimum(parents, (i - 1).to(torch.int32))
        size = torch.tensor([max(1, rows - (b * rows) // 5) for b in range(B)], device="cuda")
        out["parents"] = torch.where(i < size[:, None], parents, -2).to(torch.int32).contiguous()
    if case["op"] == "decode":
        # distinct groups in random order; one list in three ends with unused entries
        n_groups = (n - case["alpha"]) // GROUP
        kk = case["k"]
        order = torch.rand(L, B, H, max(n_groups, 1), generator=g, device="cuda").argsort(-1)
        ids = torch.full((L, B, H, kk), -1, dtype=torch.int32, device="cuda")
        m = min(kk, n_groups)
        ids[..., :m] = order[..., :m].to(torch.int32)
        unit = torch.arange(L * B * H, device="cuda").reshape(L, B, H, 1)
        drop = (unit % 3 == 2) & (torch.arange(kk, device="cuda") >= kk - kk // 4)
        out["groups"] = torch.where(drop, -1, ids).to(torch.int32).contiguous()
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


def _arrays(case, k, v):
    """The compressed cache of a prompt kept whole, as arrays: packed keys per channel over 32
    tokens, packed values per token over 32 channels, the remaining tokens exact."""
    L, B, H, n, d = k.shape
    bits = case["bits"]
    packed = 0 if bits == 16 else (n - case["alpha"]) // GROUP * GROUP
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


def _cache(case, k, v):
    """The same cache as the library's handle."""
    import kv_cache_compression_snapkv_gb300 as kvc
    n, bits = case["n"], case["bits"]
    window = WINDOW if bits != 16 else (n + 8 + 31) // 32 * 32
    dims = kvc.make_dims(case["layers"], case["batch"], case["q_heads"], case["kv_heads"],
                         case["d"], n, case["alpha"], 7, bits, GROUP, window, 8)
    budgets = [n] * case["layers"]
    cache = kvc.kvc_cache_create(dims, budgets)
    for layer in range(case["layers"]):
        kvc.kvc_prefill_compress(dims, budgets, layer, None, k[layer], v[layer], cache)
    torch.cuda.current_stream().synchronize()   # k and v are dropped by the caller
    return cache


def prepare(case, seed):
    """The prompt's compressed cache (the library's handle, or the same contents as arrays: what
    each side's program keeps between steps) and the step's inputs."""
    state = _draws(case, seed)
    k, v = state.pop("k"), state.pop("v")
    if own:
        state["cache"] = _cache(case, k, v)
    else:
        state["store"] = _arrays(case, k, v)
    L, B, Hq, d = case["layers"], case["batch"], case["q_heads"], case["d"]
    if case["op"] == "select":
        state["out"] = torch.empty(L, B, case["kv_heads"], case["k"], dtype=torch.int32, device="cuda")
    elif case["op"] == "decode":
        state["out"] = torch.empty(L, B, Hq, d, dtype=torch.float32, device="cuda")
    else:
        state["out"] = torch.empty(L, B, Hq, case["t"], d, dtype=torch.bfloat16, device="cuda")
    state["case"] = case
    return state


# ------------------------------------------------------------------------------------ one pass
def _select(store, q, kk, bits):
    """The kk groups of the largest sum over the group's query heads of the upper bound
    sum_c max(q_c lo_c, q_c hi_c) of q . k, ascending, -1 where there are fewer groups; in 64 bits,
    since the bounds next to the border decide. A bound that is not finite ranks last."""
    G = store["n_groups"]
    L, B, Hq, d = q.shape
    H = store["win_k"].shape[2]
    ids = torch.full((L, B, H, kk), -1, dtype=torch.int32, device=q.device)
    if G == 0:
        return ids
    qd = q.double().reshape(L, B, H, Hq // H, d)
    pos, neg = qd.clamp(min=0).sum(3), qd.clamp(max=0).sum(3)
    lo = store["k_zero"].double()
    hi = lo + (2 ** bits - 1) * store["k_scale"].double()
    score = (hi * pos[:, :, :, None] + lo * neg[:, :, :, None]).sum(-1)
    score = torch.where(torch.isfinite(score), score, -math.inf)
    m = min(kk, G)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :m]
    ids[..., :m] = torch.sort(best, dim=-1).values.to(torch.int32)
    return ids


def _keys(store):
    return store["k_codes"].float() * store["k_scale"].float().unsqueeze(4) + store["k_zero"].float().unsqueeze(4)


def _values(store):
    x = store["v_codes"].float() * store["v_scale"].float().unsqueeze(-1) + store["v_zero"].float().unsqueeze(-1)
    return x.flatten(-2)


def _decode(store, q, groups):
    """One query per head over the listed groups and the window: one softmax."""
    L, B, Hq, d = q.shape
    H = store["win_k"].shape[2]
    keys, values = store["win_k"].float(), store["win_v"].float()
    seen = torch.ones(keys.shape[:-1], dtype=torch.bool, device=q.device)
    if store["n_groups"]:
        ok = (groups >= 0) & (groups < store["n_groups"])
        at = torch.where(ok, groups, 0).long()
        index = [torch.arange(s, device=q.device).reshape(shape) for s, shape in
                 ((L, (L, 1, 1, 1)), (B, (1, B, 1, 1)), (H, (1, 1, H, 1)))]
        part = {x: store[x][index[0], index[1], index[2], at] for x in store if x[:2] in ("k_", "v_")}
        keys = torch.cat([_keys(part).flatten(3, 4), keys], 3)
        values = torch.cat([_values(part).flatten(3, 4), values], 3)
        seen = torch.cat([ok.unsqueeze(-1).expand(*ok.shape, GROUP).flatten(3, 4), seen], 3)
    if keys.shape[3] == 0:
        return torch.zeros(L, B, Hq, d, device=q.device)
    x = q.float().reshape(L, B, H, Hq // H, d) @ keys.transpose(-1, -2) / math.sqrt(d)
    x = torch.where(seen.unsqueeze(3), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.where(seen.unsqueeze(3), torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
    s = w.sum(-1, keepdim=True)
    return (w @ values / torch.where(s == 0, 1.0, s)).reshape(L, B, Hq, d)


def _tree(store, q, parents, k_draft, v_draft):
    """Every node over the cache, its ancestors and itself; a padding node's row is zero."""
    L, B, Hq, T, d = q.shape
    H = k_draft.shape[2]
    node = torch.arange(T, device=q.device)
    bad = (parents < -1) | (parents >= node)
    link = ((parents.unsqueeze(-1) == node) & ~bad.unsqueeze(-1)).float()
    sees = torch.eye(T, device=q.device) + link          # of itself and its parent
    for _ in range(6):                                    # 2, 4, ... 64 steps up the tree
        sees = ((sees @ sees) > 0).float()
    alive = (sees @ bad.float().unsqueeze(-1)).squeeze(-1) == 0
    mask = (sees > 0) & alive.unsqueeze(-1)
    keys, values = store["win_k"].float(), store["win_v"].float()
    if store["n_groups"]:
        keys = torch.cat([_keys(store).flatten(3, 4), keys], 3)
        values = torch.cat([_values(store).flatten(3, 4), values], 3)
    qf = q.float().reshape(L, B, H, Hq // H, T, d) / math.sqrt(d)
    old = qf.flatten(3, 4) @ keys.transpose(-1, -2)
    new = qf.flatten(3, 4) @ k_draft.float().transpose(-1, -2)
    hide = ~mask.reshape(1, B, 1, 1, T, T).expand(L, B, H, Hq // H, T, T).flatten(3, 4)
    new = new.masked_fill(hide, -math.inf)
    top = torch.maximum(old.amax(-1, keepdim=True) if old.shape[-1] else -math.inf, new.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, 0.0, top)
    old, new = torch.exp(old - top), torch.exp(new - top)
    s = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    o = (old @ values + new @ v_draft.float()) / torch.where(s == 0, 1.0, s)
    o = o.reshape(L, B, H, Hq // H, T, d).masked_fill(~alive.reshape(1, B, 1, 1, T, 1), 0.0)
    return o.reshape(L, B, Hq, T, d).bfloat16()


def run(state):
    case = state["case"]
    layers, op = case["layers"], case["op"]
    if own:
        import kv_cache_compression_snapkv_gb300 as kvc
        out = state["out"]
        if op == "select":
            kvc.kvc_select_groups(state["cache"], 0, layers, state["q"], case["k"], out)
        elif op == "decode":
            kvc.kvc_decode_groups(state["cache"], 0, layers, state["q"], case["k"], state["groups"], out)
        else:
            kvc.kvc_tree_attn(state["cache"], 0, layers, case["t"], state["parents"], state["q"],
                              state["k_draft"], state["v_draft"], out)
        return out
    store = state["store"]
    if op == "select":
        return _select(store, state["q"], case["k"], case["bits"])
    if op == "decode":
        return _decode(store, state["q"], state["groups"])
    return _tree(store, state["q"], state["parents"], state["k_draft"], state["v_draft"])


# ------------------------------------------------------------------------------------ floors
def work(case):
    L, B, Hq, H, d, n = (case[x] for x in ("layers", "batch", "q_heads", "kv_heads", "d", "n"))
    bits = case["bits"]
    groups = 0 if bits == 16 else (n - case["alpha"]) // GROUP
    window = n - groups * GROUP
    block = 8 * d * (bits + 1)
    units = L * B * H
    if case["op"] == "select":
        # every group's key scales and zero-points, the queries, the lists
        return {"bytes": units * groups * 4 * d + 2 * L * B * Hq * d + 4 * units * case["k"],
                "flops": 4 * units * groups * d}
    if case["op"] == "decode":
        lists = units * min(case["k"], groups)
        # one list in three leaves out a quarter of its entries
        used = lists - sum(max(0, min(case["k"], groups) - (case["k"] - case["k"] // 4))
                           for u in range(units) if u % 3 == 2)
        tokens = used * GROUP + units * window
        return {"bytes": used * block + units * window * 4 * d + 4 * units * case["k"] + 6 * L * B * Hq * d,
                "flops": 4 * (Hq // H) * tokens * d}
    t = case["t"]
    return {"bytes": units * (groups * block + window * 4 * d + 4 * t * d) + 4 * L * B * Hq * t * d + 4 * B * t,
            "flops": 4 * L * B * Hq * t * (n + t) * d}


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
    return base + step * code, base.squeeze(-1), (base + step * levels).squeeze(-1)


def _exact_unit(case, k, v):
    """Keys and values of one (layer, sequence, kv head) as stored, and each group's bounds."""
    n, d = k.shape
    if case["bits"] == 16:
        return k.double(), v.double(), None, None
    m = (n - case["alpha"]) // GROUP * GROUP
    kt, lo, hi = _exact_group(k[:m].reshape(-1, GROUP, d).transpose(1, 2), case["bits"])
    vt = _exact_group(v[:m].reshape(m, d // GROUP, GROUP), case["bits"])[0]
    return (torch.cat([kt.transpose(1, 2).reshape(m, d), k[m:].double()]),
            torch.cat([vt.reshape(m, d), v[m:].double()]), lo, hi)


def exact(case, seed):
    x = _draws(case, seed)
    L, B, Hq, H, d, n = (case[c] for c in ("layers", "batch", "q_heads", "kv_heads", "d", "n"))
    g = Hq // H
    made = {}
    for layer in range(L):
        for b in range(B):
            for h in range(H):
                keys, values, lo, hi = _exact_unit(case, x["k"][layer, b, h], x["v"][layer, b, h])
                q = x["q"][layer, b, h * g:(h + 1) * g].double()
                G = 0 if lo is None else lo.shape[0]
                if case["op"] == "select":
                    ids = torch.full((case["k"],), -1, dtype=torch.int32, device="cuda")
                    if G:
                        bound = sum(torch.maximum(q[j] * lo, q[j] * hi).sum(1) for j in range(g))
                        first = bound.argsort(descending=True, stable=True)[:case["k"]]
                        ids[:len(first)] = first.sort().values.to(torch.int32)
                    made[layer, b, h] = ids
                elif case["op"] == "decode":
                    m = G * GROUP
                    listed_ = x["groups"][layer, b, h].long()
                    listed_ = listed_[(listed_ >= 0) & (listed_ < G)]
                    rows = (listed_[:, None] * GROUP + torch.arange(GROUP, device="cuda")).reshape(-1)
                    rows = torch.cat([rows, torch.arange(m, n, device="cuda")])
                    if len(rows) == 0:
                        made[layer, b, h] = torch.zeros(g, d, dtype=torch.float64, device="cuda")
                    else:
                        p = torch.softmax(q @ keys[rows].T / math.sqrt(d), -1)
                        made[layer, b, h] = p @ values[rows]
                else:
                    t = case["t"]
                    parent = x["parents"][b].tolist()
                    kk = torch.cat([keys, x["k_draft"][layer, b, h].double()])
                    vv = torch.cat([values, x["v_draft"][layer, b, h].double()])
                    shut = torch.full((t, t), -math.inf, dtype=torch.float64)
                    real = torch.zeros(t, dtype=torch.bool)
                    for i in range(t):
                        path, j = [], i
                        while 0 <= j:
                            path.append(j)
                            j = parent[j] if parent[j] < j else -2
                        if j == -1:
                            real[i] = True
                            shut[i, path] = 0.0
                        else:
                            shut[i, i] = 0.0
                    logits = q.reshape(g, t, d) @ kk.T / math.sqrt(d)
                    logits[..., n:] += shut.cuda()
                    made[layer, b, h] = (torch.softmax(logits, -1) @ vv) * real.cuda().reshape(1, t, 1)
    def stack(last):
        return torch.stack([torch.stack([torch.stack([made[layer, b, h] for h in range(H)])
                                         for b in range(B)]) for layer in range(L)]).reshape(last)
    if case["op"] == "select":
        return stack((L, B, H, case["k"]))
    if case["op"] == "decode":
        return stack((L, B, Hq, d))
    return stack((L, B, Hq, case["t"], d))
