"""route, experts and moe on the GPU against plain 64-bit forms."""
import pytest
import torch

import bit_quantized_gemv_amd as q
from ops_util import DEV, TORCH, check_rows, dequantize, gen, matrix

pytestmark = pytest.mark.gpu


def problem(T, E, k, D, F, bits=4, gs=64, x="bf16", sb="bf16", seed=1):
    g = gen(seed)
    p = dict(bits=bits, gs=gs, k=k)
    p["x"] = torch.randn(T, D, generator=g).to(TORCH[x])
    p["router"] = (torch.randn(E, D, generator=g) / D ** 0.5).to(TORCH[x])
    p["w13"], p["s13"], p["b13"] = matrix(g, (E, 2 * F), D, bits, gs, sb)
    p["w2"], p["s2"], p["b2"] = matrix(g, (E, D), F, bits, gs, sb)
    return p


def want_route(p, renorm):
    logits = p["x"].double() @ p["router"].double().T
    rows = [sorted(range(len(r)), key=lambda e: (-r[e], e))[:p["k"]] for r in logits.tolist()]
    ids = torch.tensor(rows)
    top = torch.exp(logits.gather(1, ids) - logits.amax(1, keepdim=True))
    total = top.sum(1, keepdim=True) if renorm else torch.exp(logits - logits.amax(1, keepdim=True)).sum(1, keepdim=True)
    return top / total, ids


def want_experts(p, weights, ids):
    E, F = p["w13"].shape[0], p["w13"].shape[1] // 2
    y = torch.zeros(p["x"].shape, dtype=torch.float64)
    w13 = dequantize(p["w13"], p["s13"], p["b13"], p["bits"], p["gs"])
    w2 = dequantize(p["w2"], p["s2"], p["b2"], p["bits"], p["gs"])
    for t, row in enumerate(ids.tolist()):
        for j, e in enumerate(row):
            if 0 <= e < E:
                gu = w13[e] @ p["x"][t].double()
                h = gu[:F] * torch.sigmoid(gu[:F]) * gu[F:]
                y[t] += weights[t, j].double() * (w2[e] @ h)
    return y


def dev(p):
    return {k: v.to(DEV) for k, v in p.items() if isinstance(v, torch.Tensor)}


def call_experts(p, weights, ids, out_dtype=torch.float32, rows=None, **kw):
    d = dev(p)
    x, weights, ids = d["x"], weights.to(DEV), ids.to(DEV).to(torch.int32)
    if rows is not None:
        x, weights, ids = x[rows].contiguous(), weights[rows].contiguous(), ids[rows].contiguous()
    return q.experts(x, weights, ids, (d["w13"], d["s13"], d["b13"]), (d["w2"], d["s2"], d["b2"]),
                     bits=p["bits"], group_size=p["gs"], out_dtype=out_dtype, **kw)


def call_moe(p, renorm=True, out_dtype=torch.float32, **kw):
    d = dev(p)
    return q.moe(d["x"], d["router"], (d["w13"], d["s13"], d["b13"]), (d["w2"], d["s2"], d["b2"]), top_k=p["k"],
                 bits=p["bits"], group_size=p["gs"], renormalize=renorm, out_dtype=out_dtype, return_routing=True, **kw)


def some_ids(T, E, k, seed=3):
    g = gen(seed)
    return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32), torch.rand(T, k, generator=g)


def close32(a, b):
    """fp32 values of a 64-bit result: half a step (2^-24) and the same again for the result's own error."""
    assert ((a.cpu().double() - b).abs() <= 2.0 ** -23 * b.abs()).all()


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,D", [(1, 1, 1, 8), (1, 8, 8, 64), (5, 7, 2, 520), (17, 65, 5, 1024), (40, 130, 8, 2056),
                                     (300, 33, 3, 264), (3, 1024, 32, 128)])
def test_route(x, renorm, T, E, k, D):
    g = gen(T + E)
    p = dict(x=torch.randn(T, D, generator=g).to(TORCH[x]), router=torch.randn(E, D, generator=g).to(TORCH[x]) / D ** 0.5, k=k)
    p["router"] = p["router"].to(TORCH[x])
    weights, ids = q.route(p["x"].to(DEV), p["router"].to(DEV), top_k=k, renormalize=renorm)
    want_w, want_i = want_route(p, renorm)
    assert torch.equal(ids.cpu().long(), want_i)
    close32(weights, want_w)


def test_route_mixed_types_and_ties():
    g = gen(9)
    x = torch.randn(6, 64, generator=g)
    router = torch.randn(20, 64, generator=g).to(torch.bfloat16)
    router[7] = router[3]
    router[19] = router[3]
    router[12] = router[0]
    p = dict(x=x, router=router, k=20)
    weights, ids = q.route(x.to(DEV), router.to(DEV), top_k=20)
    want_w, want_i = want_route(p, True)
    assert torch.equal(ids.cpu().long(), want_i)
    close32(weights, want_w)
    z = q.route(torch.zeros(3, 64, device=DEV), router.to(DEV), top_k=4)
    assert torch.equal(z[1].cpu(), torch.tensor([[0, 1, 2, 3]] * 3, dtype=torch.int32))
    assert torch.equal(z[0].cpu(), torch.full((3, 4), 0.25))


def test_route_near_ties():
    """Logits that differ by less than fp32 resolves: the 64-bit order decides."""
    x = torch.zeros(1, 64)
    x[0, 0], x[0, 1] = 1.0, 2.0 ** -30
    router = torch.zeros(5, 64)
    router[:, 0] = 1.0
    router[:, 1] = torch.tensor([0.0, 1.0, -1.0, 3.0, 2.0])
    _, ids = q.route(x.to(DEV), router.to(DEV), top_k=5)
    assert ids.cpu().tolist() == [[3, 4, 1, 0, 2]]


def test_route_nan_counts_as_smallest():
    x = torch.ones(2, 64)
    router = torch.zeros(6, 64)
    router[:, 0] = torch.arange(6.0)
    router[4, 1] = float("nan")
    _, ids = q.route(x.to(DEV), router.to(DEV), top_k=6)
    assert ids.cpu().tolist() == [[5, 3, 2, 1, 0, 4]] * 2


@pytest.mark.parametrize("bits,gs", [(4, 64), (4, 128), (2, 64), (2, 128)])
@pytest.mark.parametrize("x,sb", [("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("T,E,k,D,F", [(1, 5, 2, 128, 128), (4, 3, 3, 384, 256), (19, 4, 2, 256, 640), (70, 2, 1, 128, 128)])
def test_experts(bits, gs, x, sb, T, E, k, D, F):
    p = problem(T, E, k, D, F, bits, gs, x=x, sb=sb)
    ids, weights = some_ids(T, E, k)
    want = want_experts(p, weights, ids)
    check_rows(call_experts(p, weights, ids), want, "fp32", "f32")
    check_rows(call_experts(p, weights, ids, out_dtype=torch.bfloat16), want, "bf16", "bf16")


@pytest.mark.parametrize("D,F", [(64, 64), (192, 64), (64, 192), (320, 448), (2112, 64)])
def test_odd_groups(D, F):
    for bits in (4, 2):
        p = problem(3, 4, 2, D, F, bits, 64)
        ids, weights = some_ids(3, 4, 2)
        check_rows(call_experts(p, weights, ids), want_experts(p, weights, ids), f"{bits}-bit", "f32")


@pytest.mark.parametrize("bits,gs,T,D,F", [(4, 64, 2, 65536, 64), (2, 128, 20, 64 * 1024, 128), (4, 64, 3, 64, 40000 // 64 * 64), (2, 64, 40, 128, 81920)])
def test_long_rows(bits, gs, T, D, F):
    """Rows whose scales go to the shared memory in windows, by pairs and sorted."""
    p = problem(T, 2, 2, D, F, bits, gs)
    ids, weights = some_ids(T, 2, 2)
    check_rows(call_experts(p, weights, ids), want_experts(p, weights, ids), "windows", "f32")


@pytest.mark.parametrize("T,E,k", [(64, 16, 2), (65, 16, 2), (16, 16, 8), (128, 3, 1), (256, 8, 2), (300, 2, 1)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_sorted_pairs(T, E, k, x):
    """Both sides of the rule by which pairs are sorted; experts that nothing chooses; empty slots among them."""
    p = problem(T, E, k, 192, 128, x=x, seed=T)
    ids, weights = some_ids(T, E, k)
    ids[ids == E - 1] = 0                       # the last expert meets nothing
    ids[::5, 0] = -1
    for dtype in (torch.float32, torch.bfloat16):
        want = want_experts(p, weights, ids)
        y = call_experts(p, weights, ids, out_dtype=dtype)
        keep = (want != 0).any(-1)
        assert (y[~keep] == 0).all()
        check_rows(y[keep], want[keep], str(dtype), "f32" if dtype == torch.float32 else "bf16")
    rows = [0, 1, T // 2, T - 1]
    assert torch.equal(call_experts(p, weights, ids, rows=rows), call_experts(p, weights, ids)[rows])


@pytest.mark.parametrize("T,E,k,D,F", [(63, 16, 2, 1024, 512), (64, 16, 2, 1024, 512), (40, 5, 3, 576, 448), (44, 5, 3, 576, 448),
                                       (20, 17, 9, 192, 128)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_sorted_pairs_of_larger_experts(T, E, k, D, F, x):
    """Both sides of the rule, by the pairs of an expert, by the products' size and by the slots of a token."""
    p = problem(T, E, k, D, F, x=x, seed=T)
    ids, weights = some_ids(T, E, k)
    ids[ids == E - 1] = 0
    ids[::5, 0] = -1
    want = want_experts(p, weights, ids)
    y = call_experts(p, weights, ids)
    keep = (want != 0).any(-1)
    assert (y[~keep] == 0).all()
    check_rows(y[keep], want[keep], "sorted", "f32")
    rows = [0, 1, T // 2, T - 1]
    assert torch.equal(call_experts(p, weights, ids, rows=rows), y[rows])


@pytest.mark.parametrize("bits,gs,T,E,k,D,F", [(4, 64, 150, 3, 1, 512, 5760), (2, 64, 90, 2, 2, 512, 5824), (4, 128, 254, 6, 1, 5888, 128),
                                              (4, 64, 200, 2, 1, 576, 320)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_many_tokens_per_expert(bits, gs, T, E, k, D, F, x):
    """One and two token tiles per wave, an expert's pairs shared by workgroups or gone through by each; uneven counts."""
    p = problem(T, E, k, D, F, bits, gs, x=x, seed=T)
    ids, weights = some_ids(T, E, k)
    ids[T // 4:T // 2, 0] = 0
    for dtype in (torch.float32, torch.bfloat16):
        want = want_experts(p, weights, ids)
        check_rows(call_experts(p, weights, ids, out_dtype=dtype), want, str(dtype), "f32" if dtype == torch.float32 else "bf16")
    rows = [0, T // 3, T - 1]
    assert torch.equal(call_experts(p, weights, ids, rows=rows), call_experts(p, weights, ids)[rows])


def test_empty_slots_and_repeats():
    p = problem(5, 4, 3, 128, 128)
    ids = torch.tensor([[-1, -1, -1], [2, -1, 4], [1, 1, 1], [3, 0, -7], [2 ** 31 - 1, 3, 3]], dtype=torch.int32)
    weights = torch.rand(5, 3, generator=gen(2))
    weights[0] = float("nan")        # never read: those slots are empty
    weights[1, 1] = float("inf")
    want = want_experts(p, weights, ids)
    y = call_experts(p, weights, ids)
    assert torch.equal(y[0].cpu(), torch.zeros(128))
    check_rows(y[1:], want[1:], "slots", "f32")


def test_all_tokens_on_one_expert():
    p = problem(150, 9, 1, 128, 64)
    ids, weights = torch.full((150, 1), 5, dtype=torch.int32), torch.ones(150, 1)
    check_rows(call_experts(p, weights, ids), want_experts(p, weights, ids), "one expert", "f32")


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_tokens_do_not_depend_on_the_call(x):
    p = problem(60, 6, 2, 512, 256, x=x)
    ids, weights = some_ids(60, 6, 2)
    whole = call_experts(p, weights, ids)
    assert torch.equal(whole, call_experts(p, weights, ids))
    for t in (0, 7, 31, 59):
        assert torch.equal(call_experts(p, weights, ids, rows=[t])[0], whole[t]), t
    assert torch.equal(call_experts(p, weights, ids, rows=list(range(59, -1, -1))), whole.flip(0))


@pytest.mark.parametrize("bits,E,k,D,F", [(4, 16, 8, 1088, 960), (2, 40, 9, 256, 320), (4, 12, 1, 64, 2944), (2, 9, 8, 128, 5888)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_whole_tokens_and_pairs_agree(bits, E, k, D, F, dtype):
    """Few tokens, whose experts' outputs are added up at once; more slots than waves; more tokens, by expert."""
    T = 9
    p = problem(T, E, k, D, F, bits, 64, seed=k)
    ids, weights = some_ids(T, E, k)
    ids[1] = -1
    ids[2, 0] = E
    want = want_experts(p, weights, ids)
    whole = call_experts(p, weights, ids, out_dtype=dtype)
    keep = [t for t in range(T) if t != 1 and bool((want[t] != 0).any())]
    check_rows(whole[keep], want[keep], "tokens", "f32" if dtype == torch.float32 else "bf16")
    assert (whole[1] == 0).all()
    for t in (0, 1, 2, 8):
        assert torch.equal(call_experts(p, weights, ids, out_dtype=dtype, rows=[t])[0], whole[t]), t


@pytest.mark.parametrize("T", [1, 2, 13, 40, 257, 520])
@pytest.mark.parametrize("renorm", [True, False])
def test_moe(T, renorm):
    p = problem(T, 16, 4, 192, 128, seed=T)
    y, weights, ids = call_moe(p, renorm)
    want_w, want_i = want_route(p, renorm)
    assert torch.equal(ids.cpu().long(), want_i)
    close32(weights, want_w)
    check_rows(y, want_experts(p, want_w, want_i), "moe", "f32")
    d = dev(p)
    w2, i2 = q.route(d["x"], d["router"], top_k=4, renormalize=renorm)
    assert torch.equal(w2, weights) and torch.equal(i2, ids)
    assert torch.equal(call_experts(p, w2.cpu(), i2.cpu()), y)


def test_no_tokens():
    p = problem(1, 4, 2, 128, 128)
    p["x"] = p["x"][:0]
    y, weights, ids = call_moe(p)
    assert y.shape == (0, 128) and weights.shape == (0, 2) and ids.shape == (0, 2)


def test_a_bad_token_stays_alone():
    p = problem(12, 4, 2, 128, 128)
    ids, weights = some_ids(12, 4, 2)
    clean = call_experts(p, weights, ids)
    p["x"][3, 5] = float("nan")
    y = call_experts(p, weights, ids)
    keep = [t for t in range(12) if t != 3]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[3]).all()


def test_stream_and_graph():
    p = problem(5, 8, 2, 256, 128)
    want = call_moe(p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call_moe(p, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = dev(p)
    out = torch.empty(5, 256, device=DEV)
    args = ((d["w13"], d["s13"], d["b13"]), (d["w2"], d["s2"], d["b2"]))
    kw = dict(top_k=2, bits=4, group_size=64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.moe(d["x"], d["router"], *args, out=out, **kw)
    for i in range(3):
        out.zero_()
        d["x"].copy_(p["x"] * (1 + i) + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.moe(d["x"], d["router"], *args, out_dtype=torch.float32, **kw)), i
