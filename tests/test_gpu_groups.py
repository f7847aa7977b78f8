"""Group selection by the stored key bounds and decode attention over listed groups, against
plain 64-bit forms over the exported cache."""
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
    dict(q_heads=2, kv_heads=2, d=128, n=1, alpha=0, bits=4),                  # no group
    dict(q_heads=4, kv_heads=1, d=128, n=320, alpha=0, bits=2),                # an empty window
    dict(q_heads=4, kv_heads=2, d=128, n=300, alpha=16, bits=2, appended=90),  # flushed groups
    dict(q_heads=4, kv_heads=2, d=64, n=300, alpha=16, bits=2, layers=3, layer_bits=[2, 16, 4]),
    dict(q_heads=1, kv_heads=1, d=64, n=40000, alpha=5, bits=2),               # many groups
]
IDS = [f"{i}" for i in range(len(CASES))]


def queries(cache, g, spread=1.0):
    D = cache.dims
    return (spread * torch.randn(D.n_layers, D.batch, D.n_q_heads, D.head_dim, generator=g,
                                 device="cuda")).bfloat16()


def expected_lists(cache, q, k):
    D = cache.dims
    H, gq = D.n_kv_heads, D.n_q_heads // D.n_kv_heads
    out = torch.full((D.n_layers, D.batch, H, k), -1, dtype=torch.int32)
    for layer in range(D.n_layers):
        _, _, G, lo, hi = contents(cache, layer)
        if G == 0:
            continue
        qd = q[layer].double().reshape(D.batch, H, gq, 1, D.head_dim)
        s = torch.maximum(qd * lo[:, :, None], qd * hi[:, :, None]).sum((2, 4))
        s = torch.where(torch.isfinite(s), s, -torch.inf).cpu()
        best = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :k].sort(-1).values
        out[layer, ..., :best.shape[-1]] = best.int()
    return out


def select(cache, q, k, stream=None):
    D = cache.dims
    out = torch.full((D.n_layers, D.batch, D.n_kv_heads, k), -7, dtype=torch.int32, device="cuda")
    K.kvc_select_groups(cache, 0, D.n_layers, q, k, out, stream)
    return out


def decode(cache, q, lists, stream=None):
    D = cache.dims
    out = torch.full((D.n_layers, D.batch, D.n_q_heads, D.head_dim), float("nan"), device="cuda")
    K.kvc_decode_groups(cache, 0, D.n_layers, q, lists.shape[-1], lists, out, stream)
    return out


def check_decode(cache, q, lists, got):
    """Against softmax over the listed groups (each as often as it is listed) and the window."""
    D = cache.dims
    H, gq, d = D.n_kv_heads, D.n_q_heads // D.n_kv_heads, D.head_dim
    for layer in range(D.n_layers):
        keys, values, G, _, _ = contents(cache, layer)
        for b in range(D.batch):
            for h in range(H):
                ids = lists[layer, b, h].long().cpu()
                ids = ids[(ids >= 0) & (ids < G)]
                rows = (ids[:, None] * 32 + torch.arange(32)).reshape(-1)
                rows = torch.cat([rows, torch.arange(G * 32, keys.shape[2])]).cuda()
                qd = q[layer, b, h * gq:(h + 1) * gq].double()
                o = got[layer, b, h * gq:(h + 1) * gq].double()
                if len(rows) == 0:
                    assert torch.all(o == 0)
                    continue
                want, size, wv = attend(qd, keys[b, h, rows], values[b, h, rows])
                # q S and p S as fp16 pairs (hi + lo: 2^-21 of the product), fp32 sums; the
                # code and zero-point terms of a value are each up to 2^b times the value, the
                # weights go through exp2 (2^-22)
                vmax = values[b, h, rows].abs().amax()
                dx = sum_bound(size, d, 2.0 ** -21)
                tol = 2 * dx * wv.amax(-1, keepdim=True) + vmax * (2.0 ** -18 + len(rows) * U32)
                assert torch.all((o - want).abs() <= tol), (o - want).abs().max().item()


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("k", [1, 7, 64])
def test_selection_is_exact(case, k):
    cache, g = make_cache(100 + k, **case)
    for spread in (1.0, 40.0):
        q = queries(cache, g, spread)
        got = select(cache, q, k).cpu()
        assert torch.equal(got, expected_lists(cache, q, k))


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("k", [1, 6, 33])
def test_decode_over_listed_groups(case, k):
    cache, g = make_cache(200 + k, **case)
    q = queries(cache, g)
    lists = select(cache, q, k)
    check_decode(cache, q, lists, decode(cache, q, lists))
    # any order, skipped entries (negative, past the last group, the extreme integers) and
    # groups listed twice
    lists = lists[..., torch.randperm(k, device="cuda", generator=g)].contiguous()
    lists[..., 0::5] = torch.tensor(-1, dtype=torch.int32)
    lists[..., 1::5] = torch.tensor(2 ** 31 - 1, dtype=torch.int32)
    lists[..., 2::5] = 0
    if k > 3:
        lists[..., 3] = -2 ** 31
    check_decode(cache, q, lists, decode(cache, q, lists))


@pytest.mark.parametrize("case", [CASES[1], CASES[3], CASES[7], CASES[8]], ids=["1", "3", "7", "8"])
def test_all_groups_listed_is_the_full_decode(case):
    cache, g = make_cache(7, **case)
    q = queries(cache, g)
    D = cache.dims
    k = max(K.kvc_layer_info_get(cache, layer)["packed_tokens"] // 32 for layer in range(D.n_layers))
    lists = select(cache, q, k)
    got = decode(cache, q, lists)
    full = torch.empty_like(got)
    K.kvc_decode_attn(cache, 0, D.n_layers, q, full)
    check_decode(cache, q, lists, got)
    check_decode(cache, q, lists, full)   # to the same bound


@pytest.mark.parametrize("d,n,alpha", [(64, 60, 40), (128, 40, 20), (128, 200, 90)])
def test_listed_decode_of_a_window_is_accurate(d, n, alpha):
    """Few packed tokens, or none: weights, sums and outputs to fp32's accuracy. A logit is off by
    the exponential's and the scale's roundings and its fp32 sum's, a weight by 2^-26 of
    itself, the sums by their roundings: 16 half steps of fp32 cover the norm of a row's error."""
    cache, g = make_cache(40, q_heads=8, kv_heads=2, d=d, n=n, alpha=alpha, bits=4, window=128)
    q = queries(cache, g)
    lists = select(cache, q, 3)
    got = decode(cache, q, lists).double()
    keys, values, G, _, _ = contents(cache, 0)
    assert G <= 3                          # every packed group is listed
    qd = q[0, 0].double().reshape(2, 4, d)
    want = attend(qd, keys[0], values[0])[0].reshape(8, d)
    err = (got[0, 0] - want).norm(dim=-1) / want.norm(dim=-1)
    assert err.max() <= 16 * U32, err.max().item()


def test_ties_and_values_that_are_not_finite():
    """Equal groups: the lower index. A group whose scale or zero-point overflowed ranks last."""
    d, G = 64, 40
    dims = K.make_dims(1, 1, 2, 1, d, G * 32, 0, 7, 4, 32, 64, 4)
    k = torch.zeros(1, 1, G, 32, d, device="cuda")
    k[:, :, :, 0] = 1.0
    k[:, :, 5] = 2.0                     # scores higher with positive queries
    k[:, :, 9, 3, 7] = 1e30              # overflows the fp16 scale
    k[:, :, 11, 4, 8] = float("inf")
    v = torch.randn(1, 1, G * 32, d, device="cuda").bfloat16()
    cache = K.kvc_prefill_compress(dims, [G * 32], 0, None, k.reshape(1, 1, -1, d).bfloat16(), v)
    q = torch.ones(1, 1, 2, d, device="cuda").bfloat16()
    ordinary = [i for i in range(G) if i not in (5, 9, 11)]
    for kk in (1, 3, 20, 37, 39, 40, 45):
        want = sorted(([5] + ordinary + [9, 11])[:kk])
        got = select(cache, q, kk)[0, 0, 0].tolist()
        assert got == want + [-1] * (kk - len(want)), kk
    # nothing to choose by: the lowest indices
    for fill in (0.0, float("nan"), float("inf")):
        assert select(cache, torch.full_like(q, fill), 4)[0, 0, 0].tolist() == [0, 1, 2, 3]
    # queries at both ends of bf16's range rank alike
    for s in (2.0 ** 120, 2.0 ** -120):
        assert select(cache, q * s, 1)[0, 0, 0].tolist() == [5]


@pytest.mark.parametrize("n,same", [(9000, 300), (200000, 4000), (260000, 8000)])
def test_many_equal_scores_at_the_border(n, same):
    """More groups of the border's score than the selecting block ranks at once, among scores
    that differ in their last bits only; rows longer than it keeps in shared memory."""
    d, G = 64, n // 32
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn(1, 1, G, 32, d, generator=g, device="cuda").bfloat16()
    twins = torch.randperm(G, generator=g, device="cuda")[:same]
    k[:, :, twins] = k[:, :, twins[:1]]                       # equal groups
    near = torch.randperm(G, generator=g, device="cuda")[:same // 2]
    k[:, :, near] = k[:, :, twins[:1]]
    k[:, :, near, 31, d - 1] = (k[:, :, twins[:1], 31, d - 1] * 1.004).bfloat16()
    v = torch.zeros(1, 1, G * 32, d, device="cuda").bfloat16()
    dims = K.make_dims(1, 1, 1, 1, d, G * 32, 0, 7, 4, 32, 64, 4)
    cache = K.kvc_prefill_compress(dims, [G * 32], 0, None, k.reshape(1, 1, -1, d), v)
    q = torch.randn(1, 1, 1, d, generator=g, device="cuda").bfloat16()
    _, _, _, lo, hi = contents(cache, 0)
    qd = q[0, 0].double()
    s = torch.maximum(qd * lo[0, 0], qd * hi[0, 0]).sum(-1)
    at = int((s > s[twins[0]]).sum())                          # the twins' rank
    for kk in {max(1, at), at + 1, at + same // 3, min(G, at + same + same // 2 + 3)}:
        assert torch.equal(select(cache, q, kk).cpu(), expected_lists(cache, q, kk)), kk


def test_many_layers_streams_and_graphs():
    """More layers than one launch takes; a side stream; a captured and replayed pair of calls."""
    cache, g = make_cache(3, layers=66, q_heads=2, kv_heads=1, d=64, n=330, alpha=3, bits=2)
    q = queries(cache, g)
    want = select(cache, q, 3)
    assert torch.equal(want.cpu(), expected_lists(cache, q, 3))
    base = decode(cache, q, want)
    check_decode(cache, q, want, base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lists = select(cache, q, 3, side)
        out = decode(cache, q, lists, side)
        graph = torch.cuda.CUDAGraph()
        lists2, out2 = torch.empty_like(lists), torch.empty_like(out)
        with torch.cuda.graph(graph, stream=side):
            K.kvc_select_groups(cache, 0, 66, q, 3, lists2, side)
            K.kvc_decode_groups(cache, 0, 66, q, 3, lists2, out2, side)
        lists2.fill_(-5)
        graph.replay()
        graph.replay()
    side.synchronize()
    assert torch.equal(lists, want) and torch.equal(out, base)
    assert torch.equal(lists2, want) and torch.equal(out2, base)
    q.copy_(queries(cache, g))            # new queries in the captured buffers
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lists2.cpu(), expected_lists(cache, q, 3))
    assert torch.equal(out2, decode(cache, q, lists2))


def test_two_caches_at_once_and_calls_in_turn():
    """Calls on different caches from different streams may overlap; on one cache the calls
    share a workspace and follow each other."""
    made = [make_cache(30 + i, **CASES[c]) for i, c in enumerate((2, 3))]
    qs = [queries(c, g) for c, g in made]
    want = [(select(c, q, 9), decode(c, q, select(c, q, 9))) for (c, _), q in zip(made, qs)]
    full = []
    for (c, _), q in zip(made, qs):
        full.append(torch.empty_like(decode(c, q, select(c, q, 9))))
        K.kvc_decode_attn(c, 0, c.dims.n_layers, q, full[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(10):
        for (c, _), q, w, f, st in zip(made, qs, want, full, streams):
            with torch.cuda.stream(st):
                lists = select(c, q, 9, st)
                out = decode(c, q, lists, st)
                all_ = torch.empty_like(f)
                K.kvc_decode_attn(c, 0, c.dims.n_layers, q, all_, st)
                ok = torch.equal(lists, w[0]) and torch.equal(out, w[1]) and torch.equal(all_, f)
            assert ok


def test_listed_decode_reports_waits_that_give_up():
    cache, g = make_cache(33, **CASES[2])
    q = queries(cache, g)
    lists = select(cache, q, 20)
    want = decode(cache, q, lists)
    torch.cuda.synchronize()
    K.kvc_set_wait_limit(cache, 0)
    decode(cache, q, lists)
    torch.cuda.synchronize()
    K.kvc_set_wait_limit(cache, -1)
    with pytest.raises(K.KvcError) as e:
        decode(cache, q, lists)
        K.kvc_check_device(cache)
    assert e.value.status == 7
    assert torch.equal(decode(cache, q, lists), want)
    torch.cuda.synchronize()
    K.kvc_check_device(cache)


def test_layer_ranges():
    cache, g = make_cache(5, layers=4, q_heads=4, kv_heads=2, d=128, n=700, alpha=8, bits=4)
    q = queries(cache, g)
    lists = select(cache, q, 5)
    out = decode(cache, q, lists)
    part, o = torch.empty_like(lists[1:3]), torch.empty_like(out[1:3])
    K.kvc_select_groups(cache, 1, 2, q[1:3].contiguous(), 5, part)
    K.kvc_decode_groups(cache, 1, 2, q[1:3].contiguous(), 5, part, o)
    assert torch.equal(part, lists[1:3])
    # other ranges split over the warps elsewhere: equal up to the sums' order
    assert torch.allclose(o, out[1:3], rtol=1e-5, atol=1e-5)


def test_a_captured_first_call_is_refused():
    cache, g = make_cache(8, q_heads=4, kv_heads=2, d=64, n=100, alpha=4, bits=2)
    q = queries(cache, g)
    lists = torch.zeros(1, 1, 2, 2, dtype=torch.int32, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(K.KvcError) as e:
            K.kvc_select_groups(cache, 0, 1, q, 2, lists, side)
        lists.add_(1)
    assert e.value.status == 5
    assert torch.equal(select(cache, q, 2).cpu(), expected_lists(cache, q, 2))


def test_refusals():
    cache, g = make_cache(6, layers=2, q_heads=4, kv_heads=2, d=64, n=100, alpha=4, bits=2)
    q = queries(cache, g)
    lists = torch.zeros(2, 1, 2, 4, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 1, 4, 64, device="cuda")
    off = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:]

    def status(f, *a):
        with pytest.raises(K.KvcError) as e:
            f(cache, *a)
        return e.value.status
    assert status(K.kvc_select_groups, 0, 2, q, 0, lists) == 1
    assert status(K.kvc_select_groups, 0, 2, q, (1 << 20) + 1, lists) == 1
    assert status(K.kvc_select_groups, 0, 2, None, 4, lists) == 1
    assert status(K.kvc_select_groups, 0, 2, q, 4, None) == 1
    assert status(K.kvc_select_groups, 0, 2, off, 4, lists) == 1
    assert status(K.kvc_select_groups, 1, 2, q, 4, lists) == 1
    assert status(K.kvc_select_groups, -1, 1, q, 4, lists) == 1
    assert status(K.kvc_select_groups, 0, 2 ** 31 - 1, q, 4, lists) == 1
    assert status(K.kvc_decode_groups, 0, 0, q, 4, lists, out) == 1
    assert status(K.kvc_decode_groups, 0, 2, q, 4, lists, None) == 1
    assert status(K.kvc_decode_groups, 0, 2, q, -1, lists, out) == 1
    assert status(K.kvc_decode_groups, 0, 2, off, 4, lists, out) == 1
    K.kvc_cache_reset(cache)
    assert status(K.kvc_select_groups, 0, 2, q, 4, lists) == 5
    assert status(K.kvc_decode_groups, 0, 2, q, 4, lists, out) == 5
