"""affine_lora on the GPU against a plain 64-bit form, and its invariants."""
import pytest
import torch

import bit_quantized_gemv_amd as q
from ops_util import DEV, TORCH, check_rows, dequantize, gen, matrix

pytestmark = pytest.mark.gpu


def problem(M, N, K, bits, gs, x="bf16", sb="bf16", R=16, L=3, ad="bf16", ids=None, seed=1):
    g = gen(seed)
    p = dict(bits=bits, gs=gs)
    p["w"], p["s"], p["b"] = matrix(g, (N,), K, bits, gs, sb)
    p["x"] = torch.randn(M, K, generator=g).to(TORCH[x])
    p["la"] = (torch.randn(L, R, K, generator=g) / K ** 0.5).to(TORCH[ad])
    p["lb"] = (torch.randn(L, N, R, generator=g) / R ** 0.5).to(TORCH[ad])
    p["scaling"] = 0.5 + torch.rand(L, generator=g)
    p["ids"] = torch.tensor([(5 * m + 1) % (L + 2) - 1 for m in range(M)] if ids is None else ids, dtype=torch.int32)
    return p


def want(p):
    y = p["x"].double() @ dequantize(p["w"], p["s"], p["b"], p["bits"], p["gs"]).T
    for m, a in enumerate(p["ids"].tolist()):
        if 0 <= a < p["la"].shape[0]:
            h = p["la"][a].double() @ p["x"][m].double()
            y[m] += p["scaling"][a].double() * (p["lb"][a].double() @ h)
    return y


def call(p, rows=None, out_dtype=torch.float32, **kw):
    d = {k: v.to(DEV) for k, v in p.items() if isinstance(v, torch.Tensor)}
    x, ids = d["x"], d["ids"]
    if rows is not None:
        x, ids = x[rows].contiguous(), ids[rows].contiguous()
    return q.affine_lora(d["w"], d["s"], d["b"], x, d["la"], d["lb"], ids, bits=p["bits"], group_size=p["gs"],
                         scaling=d["scaling"], out_dtype=out_dtype, **kw)


@pytest.mark.parametrize("bits,gs", [(4, 64), (4, 128), (2, 64), (2, 128)])
@pytest.mark.parametrize("x,sb,ad", [("bf16", "bf16", "bf16"), ("f32", "f16", "f16")])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (3, 50, 384), (17, 33, 640), (40, 130, 1280)])
def test_types_and_sizes(bits, gs, x, sb, ad, M, N, K):
    p = problem(M, N, K, bits, gs, x=x, sb=sb, ad=ad)
    check_rows(call(p), want(p), "fp32", "f32")
    check_rows(call(p, out_dtype=torch.bfloat16), want(p), "bf16", "bf16")


@pytest.mark.parametrize("K", [64, 192, 320, 2048, 2112, 4160])
def test_odd_groups(K):
    """Row lengths that end inside a slab, and odd group counts (unaligned scale rows)."""
    for bits in (4, 2):
        p = problem(5, 37, K, bits, 64)
        check_rows(call(p), want(p), f"{bits}-bit", "f32")


@pytest.mark.parametrize("R", [1, 5, 8, 31, 32, 33, 64, 100])
@pytest.mark.parametrize("ad", ["bf16", "f16"])
def test_ranks(R, ad):
    p = problem(9, 70, 256, 4, 64, R=R, ad=ad)
    check_rows(call(p), want(p), f"rank {R}", "f32")


@pytest.mark.parametrize("M,N,K,R", [(70, 100, 5120, 512), (64, 8200, 1024, 200), (64, 70, 16384, 96), (20, 9000, 640, 300)])
def test_many_ranks_of_many_tokens(M, N, K, R):
    """Hidden values that fill the shared memory."""
    p = problem(M, N, K, 4, 64, R=R, L=5)
    check_rows(call(p), want(p), f"rank {R}", "f32")


@pytest.mark.parametrize("bits,gs,M,N,K", [(4, 64, 3, 40, 65536), (2, 64, 20, 33, 65536 + 64), (4, 128, 2, 20, 131072),
                                           (2, 128, 1, 8200, 98304), (4, 64, 40, 8192, 32768)])
def test_long_rows(bits, gs, M, N, K):
    """Rows whose scales go to the shared memory in windows."""
    if N > 1000:
        p = problem(M, 64, K, bits, gs, R=8)
        reps = N // 64 + 1            # the same rows over and over: only the first 64 are compared in 64 bits
        for n in ("w", "s", "b"):
            p[n] = p[n].repeat(reps, 1)[:N].contiguous()
        p["lb"] = p["lb"].repeat(1, reps, 1)[:, :N].contiguous()
        y = call(p)
        first = {**p, "w": p["w"][:64], "s": p["s"][:64], "b": p["b"][:64], "lb": p["lb"][:, :64]}
        check_rows(y[:, :64], want(first), "first rows", "f32")
        assert torch.equal(y, y[:, :64].repeat(1, reps)[:, :N])
    else:
        p = problem(M, N, K, bits, gs, R=8)
        check_rows(call(p), want(p), "windows", "f32")


@pytest.mark.parametrize("ids", [[-1] * 20, [0] * 20, list(range(20)), [7, -1, 99, 3, -5] * 4])
def test_ids(ids):
    """No adapter, one for all, one each, and ids outside the range."""
    p = problem(20, 48, 256, 4, 64, L=20, ids=ids)
    check_rows(call(p), want(p), "ids", "f32")


@pytest.mark.parametrize("N", [15360 // 4, 7001, 12800 + 7])
def test_row_tiles(N):
    """Launches of one, two and four row tiles per workgroup (row counts on both sides of the rule)."""
    for M in (1, 20, 70):
        p = problem(M, N, 512, 4, 64, seed=M)
        check_rows(call(p), want(p), f"M {M}", "f32")


@pytest.mark.parametrize("bits,gs,N,K", [(4, 64, 16385, 512), (4, 128, 8215, 3200), (2, 64, 16417, 1024), (4, 64, 4129, 8256),
                                         (2, 128, 8200, 6272)])
@pytest.mark.parametrize("x,sb", [("bf16", "bf16"), ("f32", "f16")])
def test_two_row_tiles(bits, gs, N, K, x, sb):
    """More waves of one row tile than fit at once: two tiles each, the last one part empty."""
    p = problem(3, N, K, bits, gs, x=x, sb=sb, R=8, seed=N)
    y = call(p)
    check_rows(y, want(p), "two tiles", "f32")
    assert torch.equal(call(p, rows=[1])[0], y[1])


@pytest.mark.parametrize("bits,gs,M,N,K", [(4, 64, 61, 17003, 512), (4, 128, 70, 8209, 1280), (4, 64, 23, 16390, 576),
                                           (2, 64, 64, 17000, 1088), (4, 64, 47, 4500, 8192)])
@pytest.mark.parametrize("x,sb,ad", [("bf16", "bf16", "f16"), ("f32", "f16", "bf16")])
def test_token_tiles(bits, gs, M, N, K, x, sb, ad):
    """More waves of one token tile than fit at once: two and four tiles each, the last one part empty."""
    p = problem(M, N, K, bits, gs, x=x, sb=sb, ad=ad, R=24, L=5, seed=N)
    y = call(p)
    check_rows(y, want(p), "tiles", "f32")
    rows = [0, 17, M - 1]
    assert torch.equal(call(p, rows=rows), y[rows])


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_rows_do_not_depend_on_the_call(x):
    p = problem(70, 90, 1024, 4, 64, x=x, L=4)
    whole = call(p)
    assert torch.equal(whole, call(p)), "not repeatable"
    for m in (0, 1, 15, 16, 33, 69):
        assert torch.equal(call(p, rows=[m])[0], whole[m]), m
    assert torch.equal(call(p, rows=list(range(69, -1, -1))), whole.flip(0))


def test_many_tokens():
    """More tokens than one pair of launches takes."""
    p = problem(1030, 20, 128, 4, 64, L=5)
    check_rows(call(p), want(p), "M 1030", "f32")


def test_default_scaling_vector_and_empty():
    p = problem(4, 32, 128, 4, 64)
    p["scaling"] = torch.ones(3)
    d = {k: v.to(DEV) for k, v in p.items() if isinstance(v, torch.Tensor)}
    kw = dict(bits=4, group_size=64, out_dtype=torch.float32)
    y = q.affine_lora(d["w"], d["s"], d["b"], d["x"], d["la"], d["lb"], d["ids"], **kw)
    assert torch.equal(y, call(p))
    one = q.affine_lora(d["w"], d["s"], d["b"], d["x"][1], d["la"], d["lb"], d["ids"][1:2], **kw)
    assert one.shape == (32,) and torch.equal(one, y[1])
    none = q.affine_lora(d["w"], d["s"], d["b"], d["x"][:0], d["la"], d["lb"], d["ids"][:0], **kw)
    assert none.shape == (0, 32)


def test_a_bad_token_stays_alone():
    p = problem(20, 64, 256, 4, 64, ids=[m % 3 for m in range(20)])
    clean = call(p)
    p["x"][4, 7], p["x"][9, 100] = float("nan"), float("inf")
    y = call(p)
    keep = [m for m in range(20) if m not in (4, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[[4, 9]]).any()


def test_stream_and_graph():
    p = problem(6, 100, 512, 4, 64)
    d = {k: v.to(DEV) for k, v in p.items() if isinstance(v, torch.Tensor)}
    args = (d["w"], d["s"], d["b"], d["x"], d["la"], d["lb"], d["ids"])
    kw = dict(bits=4, group_size=64, scaling=d["scaling"], out_dtype=torch.float32)
    want_y = q.affine_lora(*args, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = q.affine_lora(*args, stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, want_y)
    out = torch.zeros_like(want_y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.affine_lora(*args, out=out, **kw)
    for i in range(3):
        out.zero_()
        d["x"].copy_(p["x"] * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.affine_lora(*args, **kw)), i
