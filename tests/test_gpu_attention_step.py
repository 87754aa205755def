"""append and attend together, as a serving program calls them: prompts in chunks,
verify blocks, rejected tokens, single tokens; against a plain 64-bit form of whole
sequences, in a graph, and through the quantized projections (examples/attention_step.py)."""
import math
import os
import sys

import pytest
import torch

import bit_quantized_gemv_amd as q
from attn_util import DEV, HALF, gen, rotate64

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

pytestmark = pytest.mark.gpu


class Sequence:
    """What a sequence's tokens are before append, on the CPU."""

    def __init__(self):
        self.q, self.k, self.v = [], [], []

    def add(self, q, k, v):
        for a, t in zip((self.q, self.k, self.v), (q, k, v)):
            a.extend(t.unbind(0))

    def cut(self, n):
        for a in (self.q, self.k, self.v):
            del a[len(a) - n:]


def plain(s, last, wq, wk, freqs, window, sinks):
    """Outputs of the last tokens of a sequence, from all of it, in 64 bits; queries, keys and values rounded as the cache holds them."""
    T = len(s.q)
    ang = torch.arange(T).double().unsqueeze(1) * freqs.double()
    qs = rotate64(torch.stack(s.q), wq, 1e-6, ang, False)[0].bfloat16().double()
    ks = rotate64(torch.stack(s.k), wk, 1e-6, ang, False)[0].bfloat16().double()
    vs = torch.stack(s.v).double()
    Hq, Hkv, D = qs.shape[1], ks.shape[1], ks.shape[2]
    out, reach = [], []
    j = torch.arange(T)
    for p in range(T - last, T):
        sees = j <= p
        if window:
            sees &= (j > p - window) | (j < sinks)
        k, v = ks[sees], vs[sees]
        g = qs[p].reshape(Hkv, Hq // Hkv, D)
        w = torch.softmax(torch.einsum("hgd,jhd->hgj", g, k) / math.sqrt(D), -1)
        out.append(torch.einsum("hgj,jhd->hgd", w, v).reshape(Hq, D))
        reach.append(torch.einsum("hgj,jhd->hgd", w, v.abs()).reshape(Hq, D))
    return torch.stack(out), torch.stack(reach)


def near(got, want, reach, what):
    """As attend's own bound, with what queries and keys that are rounded the other way do: a key's score moves by a step of bf16 in one
    value of it and of the query, 2 * 2^-8 * |q_d k_d| / sqrt(D), below 2^-4 for the values here, and its weight by as much of itself."""
    lim = 2.0 ** -4 * reach + HALF["bf16"] * (reach + want.abs()) + 2e-5 * reach.amax(-1, keepdim=True)
    over = (got.cpu().double() - want).abs() - lim
    assert (over <= 0).all(), (what, float(over.max()))
    # and nearly all of them as if none were
    off = (got.cpu().double() - want).norm() / want.norm()
    assert off < 4e-3, (what, float(off))


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 4, 128), (6, 1, 80)])
def test_serving(window, sinks, Hq, Hkv, D):
    g = gen(Hq + D)
    P, pages_n = 8, 80
    kc, vc = (torch.full((pages_n, P, Hkv, D), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    order = torch.randperm(pages_n, generator=g).int()
    table = order[:60].reshape(3, 20).contiguous().to(DEV)          # 160 places each
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    freqs = 10000.0 ** (-torch.arange(D // 2).float() / (D // 2))
    seqs = [Sequence() for _ in range(3)]
    # new tokens of the three sequences in a call, and how many leave them after it
    for new, leave in (((70, 0, 1), (0, 0, 0)), ((1, 40, 5), (0, 0, 3)), ((13, 17, 1), (9, 0, 0)), ((1, 1, 1), (0, 0, 0)), ((4, 0, 20), (3, 0, 0))):
        T = sum(new)
        x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).bfloat16()
        parts = [t.unflatten(1, (-1, D)) for t in x.split((Hq * D, Hkv * D, Hkv * D), 1)]
        at = 0
        for s, n in zip(seqs, new):
            s.add(*(t[at:at + n] for t in parts))
            at += n
        starts = torch.tensor([0, *new]).cumsum(0).int().to(DEV)
        lengths = torch.tensor([len(s.q) for s in seqs], dtype=torch.int32, device=DEV)
        dev = [t.unflatten(1, (-1, D)) for t in x.to(DEV).split((Hq * D, Hkv * D, Hkv * D), 1)]
        qs = q.append(*dev, freqs.to(DEV), kc, vc, table, starts, lengths, q_weight=wq.to(DEV), k_weight=wk.to(DEV))
        got = q.attend(qs, kc, vc, table, starts, lengths, window=window, sinks=sinks, out_dtype=torch.float32)
        at = 0
        for i, (s, n) in enumerate(zip(seqs, new)):
            if n:
                near(got[at:at + n], *plain(s, n, wq, wk, freqs, window, sinks), (new, i))
            at += n
            s.cut(leave[i])


def test_graph_of_a_step():
    """append and attend of one token a sequence, captured once and replayed as the sequences grow: the eager calls' bits."""
    g = gen(3)
    B, Hq, Hkv, D, P = 5, 8, 2, 128, 16
    pools = [[torch.zeros(60, P, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(2)]
    table = torch.randperm(60, generator=g)[:50].int().reshape(B, 10).to(DEV)
    starts = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    lengths = torch.tensor([1, 40, 97, 15, 120], dtype=torch.int32, device=DEV)
    x = torch.randn(B, (Hq + 2 * Hkv) * D, generator=g).bfloat16().to(DEV)
    freqs = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).float().to(DEV)

    def step(kc, vc):
        parts = [t.unflatten(1, (-1, D)) for t in x.split((Hq * D, Hkv * D, Hkv * D), 1)]
        qs = q.append(*parts, freqs, kc, vc, table, starts, lengths)
        return q.attend(qs, kc, vc, table, starts, lengths, window=64, sinks=2, max_new=1)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*pools[1])
    for i in range(6):
        want = step(*pools[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1]), i
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        lengths += 1


def test_example():
    """The layer's outputs against the same calls on whole sequences in one chunk."""
    from examples import attention_step as ex
    layer, pool = ex.Attention(width=256, window=20, sinks=2, device=DEV), ex.Pool(40, 8, 2, 64, 16, DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn(90, 256, generator=g, device=DEV).bfloat16()
    whole = ex.step(layer, pool, ["whole"], [x])[0]
    at, parts = 0, []
    for n in (33, 1, 13, 40, 3):
        other = torch.randn(3, 256, generator=g, device=DEV).bfloat16()
        parts.append(ex.step(layer, pool, ["other", "parts"], [other, x[at:at + n]])[1])
        at += n
    a, b = whole.float(), torch.cat(parts).float()
    # the same sums in another order, weights rounded against other maxima: two roundings of weights and two of results
    assert ((a - b).norm() / a.norm()) < 4 * HALF["bf16"]
    assert torch.isfinite(a).all() and torch.isfinite(b).all()
