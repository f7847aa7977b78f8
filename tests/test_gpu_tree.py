"""Attention of a tree of drafted tokens over the cache, against a plain 64-bit form over the
exported cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu
K = pytest.importorskip("kv_cache_compression_snapkv_gb300")

from _selective import U16, U32, UB, attend, contents, make_cache, sum_bound  # noqa: E402

CACHES = [
    dict(q_heads=8, kv_heads=2, d=128, n=1000, alpha=32, bits=2),
    dict(q_heads=4, kv_heads=4, d=64, n=528, alpha=16, bits=2),
    dict(q_heads=8, kv_heads=1, d=128, n=2500, alpha=0, bits=4),
    dict(q_heads=4, kv_heads=2, d=64, n=777, alpha=9, bits=4, batch=3, layers=2),
    dict(q_heads=4, kv_heads=2, d=128, n=1, alpha=0, bits=4),                  # one token
    dict(q_heads=4, kv_heads=1, d=128, n=320, alpha=0, bits=2),                # an empty window
    dict(q_heads=4, kv_heads=2, d=128, n=300, alpha=16, bits=2, appended=90),  # a wrapped window
    dict(q_heads=4, kv_heads=2, d=64, n=300, alpha=16, bits=2, layers=3, layer_bits=[2, 16, 4]),
    dict(q_heads=2, kv_heads=1, d=128, n=777, alpha=5, bits=16, appended=7),
    dict(q_heads=8, kv_heads=1, d=64, n=333, alpha=5, bits=16),
    dict(q_heads=2, kv_heads=2, d=128, n=900, alpha=70, bits=4, window=1024, appended=700),
    dict(q_heads=1, kv_heads=1, d=128, n=20000, alpha=5, bits=2),
    dict(q_heads=2, kv_heads=1, d=128, n=30000, alpha=5, bits=16),             # many window tiles
    dict(q_heads=8, kv_heads=1, d=64, n=20000, alpha=5, bits=16),
    dict(q_heads=4, kv_heads=4, d=64, n=12001, alpha=50, bits=4, batch=4, window=256),
]
IDS = [f"{i}" for i in range(len(CACHES))]


def trees(kind, B, T, g):
    i = torch.arange(T)
    if kind == "chain":
        p = (i - 1).repeat(B, 1)
    elif kind == "star":
        p = torch.full((B, T), -1)
    elif kind == "random":
        p = torch.stack([torch.tensor([int(torch.randint(-1, max(j, 0), (1,))) if j else -1
                                       for j in range(T)]) for _ in range(B)])
    else:   # padding: bad links of every sort, and what hangs from them
        p = trees("random", B, T, g).clone()
        for b in range(B):
            for j, bad in ((T // 2, -2), (T - 1, T - 1), (T // 3, T + 5), (T // 4, -2 ** 31),
                           (T - 2, 2 ** 31 - 1)):
                if 0 <= j < T and (b + j) % 2 == 0:
                    p[b, j] = bad
        return p.int().cuda()
    return p.int().cuda()


def inputs(cache, g, T):
    D = cache.dims
    def normal(h):
        return torch.randn(D.n_layers, D.batch, h, T, D.head_dim, generator=g, device="cuda").bfloat16()
    return normal(D.n_q_heads), normal(D.n_kv_heads), normal(D.n_kv_heads)


def tree(cache, parents, q, k, v, stream=None):
    out = torch.full_like(q, float("nan"))
    K.kvc_tree_attn(cache, 0, cache.dims.n_layers, q.shape[3], parents, q, k, v, out, stream)
    return out


def masks(parents):
    """[B][T][T] visible drafted tokens; [B][T] nodes that are not padding."""
    B, T = parents.shape
    see, real = torch.zeros(B, T, T, dtype=torch.bool), torch.zeros(B, T, dtype=torch.bool)
    for b, p in enumerate(parents.tolist()):
        for i in range(T):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = p[j] if p[j] < j else -2
            if j == -1:
                real[b, i] = True
                see[b, i, path] = True
    return see.cuda(), real.cuda()


def check(cache, parents, q, k, v, got):
    D = cache.dims
    H, gq, d = D.n_kv_heads, D.n_q_heads // D.n_kv_heads, D.head_dim
    see, real = masks(parents)
    T = parents.shape[1]
    for layer in range(D.n_layers):
        keys, values, G, _, _ = contents(cache, layer)
        old = torch.ones(keys.shape[2], dtype=torch.bool, device="cuda")
        for b in range(D.batch):
            row = see[b]
            kd, vd = k[layer, b].double(), v[layer, b].double()
            live = real[b]
            if not bool(live.any()):
                assert torch.all(got[layer, b] == 0)
                continue
            at = live.nonzero()[:, 0]
            for h in range(H):
                seen = torch.cat([old.expand(len(at), -1), row[at][:, at]], 1)
                kk, vv = torch.cat([keys[b, h], kd[h, at]]), torch.cat([values[b, h], vd[h, at]])
                for j in range(gq):
                    o = got[layer, b, h * gq + j].double()
                    assert torch.all(o[~live] == 0)
                    qd = q[layer, b, h * gq + j, at].double()
                    want, size, wv = attend(qd, kk, vv, seen)
                    # stored keys and values as fp16 (packed) or as they are, queries exact up
                    # to 2^-25 of their row's largest; weights rounded to fp16 or bf16 for the
                    # product; fp32 sums; the output rounded to bf16
                    dx = sum_bound(size, d, U16)
                    tol = wv.amax(-1, keepdim=True) * (2 * dx + UB + 2 * U16 + len(kk) * U32)
                    tol = tol + UB * want.abs()
                    err = (o[at] - want).abs()
                    assert torch.all(err <= tol), (err.max().item(), (err / tol).max().item())
                    # the roundings are independent: the whole row is far nearer
                    rel = (o[at] - want).norm() / want.norm().clamp(min=1e-30)
                    assert rel <= 2 * UB, rel.item()


@pytest.mark.parametrize("case", CACHES, ids=IDS)
@pytest.mark.parametrize("T,kind", [(1, "chain"), (5, "random"), (26, "random"), (64, "random"),
                                    (33, "chain"), (17, "padding"), (64, "padding")])
def test_tree(case, T, kind):
    cache, g = make_cache(300 + T, **case)
    q, k, v = inputs(cache, g, T)
    parents = trees(kind, cache.dims.batch, T, g)
    check(cache, parents, q, k, v, tree(cache, parents, q, k, v))


@pytest.mark.parametrize("case", [CACHES[0], CACHES[3], CACHES[8]], ids=["0", "3", "8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_padding_and_masked_nodes_reach_no_other_row(case, bad):
    cache, g = make_cache(11, **case)
    T = 20
    B = cache.dims.batch
    q, k, v = inputs(cache, g, T)
    parents = trees("star", B, T, g)
    parents[:, 3], parents[:, 9], parents[:, 10] = -2, 9, 3      # padding, and a child of it
    want = tree(cache, parents, q, k, v)
    check(cache, parents, q, k, v, want)
    dirty = [x.clone() for x in (q, k, v)]
    for x in dirty:
        x[:, :, :, [3, 9, 10]] = bad
    assert torch.equal(tree(cache, parents, *dirty), want)
    # a real node's own values reach itself and its descendants only
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    v2[:, :, :, 5, 1] = bad
    k2[:, :, :, 6, 2] = bad
    got = tree(cache, parents, q2, k2, v2)
    others = [i for i in range(T) if i not in (5, 6)]
    assert torch.equal(got[:, :, :, others], want[:, :, :, others])
    assert not torch.isfinite(got[:, :, :, 5, 1]).any()
    assert torch.isfinite(got[:, :, :, 5, 2:]).all()
    v2[:, :, :, 5, 1] = 0
    parents[:, 7] = 5
    v2[:, :, :, 5, 1] = bad
    got = tree(cache, parents, q, k, v2)
    assert not torch.isfinite(got[:, :, :, [5, 7], 1]).any()
    assert torch.isfinite(got[:, :, :, [5, 7], 2:]).all()


def test_extreme_magnitudes():
    """Queries over bf16's range, and drafted keys and values beyond fp16's."""
    cache, g = make_cache(12, q_heads=4, kv_heads=2, d=128, n=500, alpha=16, bits=4, scale=0.01)
    q, k, v = inputs(cache, g, 9)
    parents = trees("random", 1, 9, g)
    for s in (2.0 ** -100, 2.0 ** -20):
        qs = (q.float() * s).bfloat16()
        check(cache, parents, qs, k, v, tree(cache, parents, qs, k, v))
    ks, vs = (k.float() * 2.0 ** 20).bfloat16(), (v.float() * 2.0 ** 90).bfloat16()
    qs = (q.float() * 2.0 ** -20).bfloat16()
    check(cache, parents, qs, ks, vs, tree(cache, parents, qs, ks, vs))
    # logits so large that their own rounding passes any slack: one token takes all the weight,
    # the one of the largest logit up to what the stored keys' rounding moves logits by
    keys, values, _, _, _ = contents(cache, 0)
    see, _ = masks(parents)
    for s in (2.0 ** 32, 2.0 ** 60, 2.0 ** 100):
        qs = (q.float() * s).bfloat16()
        got = tree(cache, parents, qs, k, v)
        for h in range(4):
            kk = torch.cat([keys[0, h // 2], k[0, 0, h // 2].double()])
            vv = torch.cat([values[0, h // 2], v[0, 0, h // 2].double()])
            qd = qs[0, 0, h].double()
            x = qd @ kk.T / 128 ** 0.5
            x[:, keys.shape[2]:].masked_fill_(~see[0], -torch.inf)
            dx = sum_bound((qd.abs() @ kk.abs().T / 128 ** 0.5).amax(-1), 128, U16)
            for i in range(9):
                off = (vv - got[0, 0, h, i].double()).abs().amax(-1)
                j = int(off.argmin())
                assert off[j] <= 2 * (UB + U16) * vv[j].abs().max()
                assert x[i, j] >= x[i].max() - 2 * dx[i]
    # sharp rows: one token takes nearly all the weight
    qs = (q.float() * 30).bfloat16()
    got = tree(cache, parents, qs, k, v)
    check(cache, parents, qs, k, v, got)


def test_chain_matches_appending_one_by_one():
    """A drafted chain verified at once, and the same tokens appended and decoded in turn (no
    group is flushed in between): the run of a speculative step and of its acceptance."""
    T = 12
    cache, g = make_cache(13, layers=2, q_heads=8, kv_heads=2, d=128, n=700, alpha=16, bits=2,
                          window=128, max_new=T)
    q, k, v = inputs(cache, g, T)
    parents = trees("chain", 1, T, g)
    got = tree(cache, parents, q, k, v)
    check(cache, parents, q, k, v, got)
    for i in range(T):
        out = torch.empty(2, 1, 8, 128, device="cuda")
        K.kvc_decode_step(cache, 0, 2, q[:, :, :, i].contiguous(), k[:, :, :, i].contiguous(),
                          v[:, :, :, i].contiguous(), out)
        # both within their own error of the same value; the outputs here are below 2
        assert torch.allclose(got[:, :, :, i].float(), out, atol=2 * UB, rtol=2 * UB)
        # the accepted prefix continues as a cache: selection and listed decode read it
        lists = torch.empty(2, 1, 2, 4, dtype=torch.int32, device="cuda")
        K.kvc_select_groups(cache, 0, 2, q[:, :, :, i].contiguous(), 4, lists)
    assert (lists >= 0).all()


def test_tree_does_not_change_the_cache():
    cache, g = make_cache(14, **CACHES[6])
    before = [t.clone() for t in contents(cache, 0)[:2]]
    info = K.kvc_layer_info_get(cache, 0)
    q, k, v = inputs(cache, g, 31)
    parents = trees("random", 1, 31, g)
    a = tree(cache, parents, q, k, v)
    b = tree(cache, parents, q, k, v)
    assert torch.equal(a, b)                       # the same bits on every run
    assert info == K.kvc_layer_info_get(cache, 0)
    assert all(torch.equal(x, y) for x, y in zip(before, contents(cache, 0)[:2]))


def test_streams_graphs_and_many_layers():
    cache, g = make_cache(15, layers=66, q_heads=2, kv_heads=1, d=64, n=200, alpha=3, bits=2)
    q, k, v = inputs(cache, g, 6)
    parents = trees("random", 1, 6, g)
    want = tree(cache, parents, q, k, v)
    check(cache, parents, q, k, v, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(q)
        with torch.cuda.graph(graph, stream=side):
            K.kvc_tree_attn(cache, 0, 66, 6, parents, q, k, v, out, side)
        graph.replay()
        first = out.clone()
        out.zero_()
        graph.replay()
    side.synchronize()
    assert torch.equal(first, want) and torch.equal(out, want)
    parents.copy_(trees("star", 1, 6, g))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(cache, parents, q, k, v, out)


@pytest.mark.parametrize("heads,T", [((2, 2), 5), ((8, 2), 8), ((8, 2), 9), ((8, 2), 30)])
def test_short_segments_of_many_sequences(heads, T):
    """No window and one tile of packed groups, a tree per sequence, many of them to a block."""
    cache, g = make_cache(30, layers=2, batch=300, q_heads=heads[0], kv_heads=heads[1], d=64, n=96,
                          alpha=0, bits=2)
    q, k, v = inputs(cache, g, T)
    parents = trees("padding", 300, T, g)
    got = tree(cache, parents, q, k, v)
    check(cache, parents, q, k, v, got)
    # against the call in which every sequence holds this one's tree: the same bits
    for b in range(0, 300, 37):
        same = tree(cache, parents[b:b + 1].repeat(300, 1), q, k, v)
        assert torch.equal(same[:, b], got[:, b])


def test_rows_do_not_depend_on_one_another():
    """A row's bits are the same whatever the queries of the other rows are."""
    cache, g = make_cache(31, q_heads=2, kv_heads=1, d=128, n=700, alpha=16, bits=4)
    for T in (7, 20):
        q, k, v = inputs(cache, g, T)
        q = (q.float() * 4).bfloat16()
        parents = trees("star", 1, T, g)
        want = tree(cache, parents, q, k, v)
        for s in (0.0, 3.0, 1e4, 1e30, float("inf"), float("nan")):
            q2 = q.clone()
            q2[:, :, 0, ::2] *= s
            got = tree(cache, parents, q2, k, v)
            assert torch.equal(got[:, :, :, 1::2], want[:, :, :, 1::2])
            assert torch.equal(got[:, :, 1], want[:, :, 1])


def test_a_captured_first_call_is_refused():
    cache, g = make_cache(32, q_heads=4, kv_heads=2, d=64, n=100, alpha=4, bits=2)
    q, k, v = inputs(cache, g, 3)
    p, out = trees("chain", 1, 3, g), torch.zeros_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(K.KvcError) as e:
            K.kvc_tree_attn(cache, 0, 1, 3, p, q, k, v, out, side)
        out.add_(1)
    assert e.value.status == 5
    check(cache, p, q, k, v, tree(cache, p, q, k, v))


@pytest.mark.parametrize("case,T", [(CACHES[0], 5), (CACHES[0], 26), (CACHES[3], 16), (CACHES[8], 40)])
def test_waits_that_give_up_are_reported_and_leave_nothing_behind(case, T):
    """With no polls allowed every wait of the launch gives up at once: the call after it (or
    the device check) says so, and later calls give what a fresh cache gives."""
    cache, g = make_cache(17, **case)
    q, k, v = inputs(cache, g, T)
    parents = trees("random", cache.dims.batch, T, g)
    want = tree(cache, parents, q, k, v)
    torch.cuda.synchronize()
    K.kvc_set_wait_limit(cache, 0)
    tree(cache, parents, q, k, v)
    torch.cuda.synchronize()
    K.kvc_set_wait_limit(cache, -1)
    with pytest.raises(K.KvcError) as e:
        tree(cache, parents, q, k, v)
        K.kvc_check_device(cache)
    assert e.value.status == 7
    assert torch.equal(tree(cache, parents, q, k, v), want)
    torch.cuda.synchronize()
    K.kvc_check_device(cache)


def test_two_caches_at_once():
    """Calls on different caches from different streams may overlap."""
    made = [make_cache(20 + i, **CACHES[c]) for i, c in enumerate((0, 2))]
    sets = []
    for (cache, g), T in zip(made, (40, 16)):
        sets.append((cache, trees("random", 1, T, g), *inputs(cache, g, T)))
    want = [tree(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [torch.full_like(s[2], float("nan")) for s in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, st in zip(sets, outs, streams):
            K.kvc_tree_attn(s[0], 0, 1, s[2].shape[3], s[1], s[2], s[3], s[4], o, st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    cache, g = make_cache(16, layers=2, q_heads=4, kv_heads=2, d=64, n=100, alpha=4, bits=2)
    q, k, v = inputs(cache, g, 3)
    p = trees("chain", 1, 3, g)
    out = torch.empty_like(q)
    off = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:]

    def status(*a):
        with pytest.raises(K.KvcError) as e:
            K.kvc_tree_attn(cache, *a)
        return e.value.status
    for i in range(5):
        a = [p, q, k, v, out]
        a[i] = None
        assert status(0, 2, 3, *a) == 1
    for i in range(1, 5):
        a = [p, q, k, v, out]
        a[i] = off
        assert status(0, 2, 3, *a) == 1
    assert status(0, 2, 0, p, q, k, v, out) == 1
    assert status(0, 2, 65, p, q, k, v, out) == 1
    assert status(1, 2, 3, p, q, k, v, out) == 1
    assert status(0, 0, 3, p, q, k, v, out) == 1
    K.kvc_cache_reset(cache)
    assert status(0, 2, 3, p, q, k, v, out) == 5
