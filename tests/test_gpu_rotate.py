"""qmv_rotate and qmv_append against plain 64-bit forms."""
import math

import pytest
import torch

import bit_quantized_gemv_amd as q
from attn_util import DEV, TORCH, Batch, check_rounded, gen, rotate64

pytestmark = pytest.mark.gpu


def inputs(g, T, Hq, Hk, D, x, w, R, A, top=5000, stuck=False):
    """Queries, keys, values (views of one projection's output if `stuck`), weights, freqs, axes, positions."""
    if stuck:
        qkv = (torch.randn(T, (Hq + 2 * Hk) * D, generator=g) * 3).to(TORCH[x]).to(DEV)
        parts = [t.unflatten(1, (-1, D)) for t in qkv.split((Hq * D, Hk * D, Hk * D), 1)]
    else:
        parts = [(torch.randn(T, h, D, generator=g) * 3).to(TORCH[x]).to(DEV) for h in (Hq, Hk, Hk)]
    weights = [None if w is None else (1 + 0.3 * torch.randn(D, generator=g)).to(TORCH[w]).to(DEV) for _ in range(2)]
    freqs = (10000.0 ** (-torch.arange(R // 2) / max(R // 2, 1))).float().to(DEV) if R else None
    pos = torch.randint(-top, top, (A, T), generator=g).int().to(DEV)
    axes = None if A == 1 else torch.randint(0, A, (R // 2,), generator=g).int().to(DEV)
    return (*parts, *weights, freqs, axes, pos[0] if A == 1 else pos)


def angles_of(pos, axes, freqs, T):
    if freqs is None:
        return torch.zeros(T, 0, dtype=torch.float64)
    p = pos.cpu().double().reshape(-1, T)
    a = torch.zeros(len(freqs), dtype=torch.long) if axes is None else axes.cpu().long()
    known = (a >= 0) & (a < p.shape[0])
    return torch.where(known, p[a.clamp(0, p.shape[0] - 1)].T * freqs.cpu().double(), 0.0)


SHAPES = [
    # T, Hq, Hk, D, R, x, w, out, axes, interleaved, stuck
    (1, 32, 8, 128, 128, "bf16", "bf16", "bf16", 1, False, True),
    (13, 16, 8, 256, 256, "bf16", "bf16", "bf16", 1, False, True),
    (5, 10, 2, 80, 40, "f32", "f32", "f16", 1, True, True),
    (3, 1, 1, 8, 8, "f32", None, "bf16", 1, False, False),
    (1, 1, 1, 256, 8, "bf16", "f32", "f16", 2, True, False),
    (17, 5, 5, 64, 64, "bf16", None, "bf16", 3, False, True),
    (7, 3, 1, 104, 56, "f32", "bf16", "f16", 3, False, False),
    (4, 6, 2, 128, 0, "bf16", "bf16", "bf16", 1, False, True),
    (2000, 4, 2, 64, 32, "bf16", "bf16", "bf16", 1, True, True),
    (700, 33, 7, 96, 96, "f32", "f32", "f16", 2, False, True),
    (257, 1, 1, 16, 16, "bf16", "bf16", "f16", 1, True, False),
    (50, 128, 16, 128, 64, "bf16", "f32", "bf16", 1, False, True),
    (4200, 2, 1, 48, 32, "bf16", "bf16", "bf16", 1, False, True),
    (300, 9, 3, 112, 96, "f32", "f32", "f16", 2, True, False),
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,x,w,out,A,inter,stuck", SHAPES)
def test_rotate(T, Hq, Hk, D, R, x, w, out, A, inter, stuck):
    qi, ki, _, qw, kw, freqs, axes, pos = inputs(gen(T * 7 + D), T, Hq, Hk, D, x, w, R, A, stuck=stuck)
    got = q.rotate(qi, ki, freqs, pos, axes=axes, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter, out_dtype=TORCH[out])
    ang = angles_of(pos, axes, freqs, T)
    for name, g, xi, wi in (("q", got[0], qi, qw), ("k", got[1], ki, kw)):
        want, size = rotate64(xi.cpu(), None if wi is None else wi.cpu(), 1e-5, ang, inter)
        assert g.dtype == TORCH[out] and g.is_contiguous()
        check_rounded(g, want, size, out, name)


@pytest.mark.parametrize("T,Hq,Hk,D,R,x,w,out,A,inter,stuck", SHAPES)
@pytest.mark.parametrize("P,order", [(16, "page"), (7, "head"), (1, "one")])
def test_append(T, Hq, Hk, D, R, x, w, out, A, inter, stuck, P, order):
    if Hq % Hk:
        Hq = Hk * (Hq // Hk)
    g = gen(T * 3 + D + P)
    new = [T] if T < 4 else [T // 2, 0, T - T // 2 - 1, 1]
    lengths = [n + o for n, o in zip(new, (0, 3, 40, 15))]
    c = Batch(new, lengths, Hk, D, P, out, seed=T, order=order, fill=9.0)
    qi, ki, vi, qw, kw, freqs, axes, pos = inputs(g, T, Hq, Hk, D, x, w, R, A, stuck=stuck)
    use = pos if A > 1 or T % 2 else None
    k, v, pages, starts, lens = c.on()
    got = q.append(qi, ki, vi, freqs, k, v, pages, starts, lens, positions=use, axes=axes, q_weight=qw, k_weight=kw, eps=1e-6,
                   interleaved=inter)
    if use is None:
        use = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lengths)]).int()
    ang = angles_of(use, axes, freqs, T)
    want, size = rotate64(qi.cpu(), None if qw is None else qw.cpu(), 1e-6, ang, inter)
    check_rounded(got, want, size, out, "q")
    want, size = rotate64(ki.cpu(), None if kw is None else kw.cpu(), 1e-6, ang, inter)
    wk, wv = c.k.clone(), c.v.clone()
    kc, vc = k.cpu(), v.cpu()
    t = 0
    for b, (m, n) in enumerate(zip(new, lengths)):
        for j in range(n - m, n):
            page, slot = c.row(b, j)
            check_rounded(kc[page, slot], want[t], size[t], out, f"k of token {t}")
            assert torch.equal(vc[page, slot], vi[t].cpu().to(TORCH[out]))
            wk[page, slot], wv[page, slot] = kc[page, slot], vc[page, slot]
            t += 1
    assert torch.equal(kc, wk) and torch.equal(vc, wv), "a slot that is no new token's was written"


def test_far_positions():
    """Angles of positions up to 2^31 as 64 bits give them."""
    g = gen(5)
    T = 40
    qi, ki, _, qw, kw, freqs, _, _ = inputs(g, T, 2, 2, 64, "f32", "f32", 64, 1)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=g).int().to(DEV)
    pos[0], pos[1] = 2 ** 31 - 1, -2 ** 31
    got, _ = q.rotate(qi, ki, freqs, pos, q_weight=qw, out_dtype=torch.float16)
    want, size = rotate64(qi.cpu(), qw.cpu(), 1e-6, angles_of(pos, None, freqs, T), False)
    check_rounded(got, want, size, "f16")


def test_one_weight_and_axes_outside():
    g = gen(6)
    T, D = 9, 64
    qi, ki, _, qw, _, freqs, _, pos = inputs(g, T, 4, 2, D, "bf16", "bf16", D, 2)
    axes = torch.tensor(([0, 1, -1, 2, 5, 1, 0, -7] * 4), dtype=torch.int32, device=DEV)
    got = q.rotate(qi, ki, freqs, pos, axes=axes, q_weight=qw)
    ang = angles_of(pos, axes, freqs, T)
    for y, x, w in ((got[0], qi, qw.cpu()), (got[1], ki, None)):
        check_rounded(y, *rotate64(x.cpu(), w, 1e-6, ang, False), "bf16")


def test_heads_stand_alone():
    """A head's outputs are the same bits in any call; NaN and infinities stay in theirs."""
    g = gen(7)
    T, Hq, Hk, D = 33, 12, 4, 128
    qi, ki, _, qw, kw, freqs, _, pos = inputs(g, T, Hq, Hk, D, "bf16", "bf16", D, 1, stuck=True)
    kwargs = dict(q_weight=qw, k_weight=kw)
    yq, yk = q.rotate(qi, ki, freqs, pos, **kwargs)
    for t in (0, 20, 32):
        a, b = q.rotate(qi[t:t + 1], ki[t:t + 1, :2], freqs, pos[t:t + 1], **kwargs)
        assert torch.equal(a[0], yq[t]) and torch.equal(b[0], yk[t, :2])
    qi[3, 5, 7], qi[4, 2, 100], ki[3, 1, 0] = math.nan, math.inf, -math.inf
    zq, zk = q.rotate(qi, ki, freqs, pos, **kwargs)
    bad = torch.zeros(T, Hq, dtype=torch.bool, device=DEV)
    bad[3, 5] = bad[4, 2] = True
    assert torch.equal(zq[~bad], yq[~bad]) and not torch.isfinite(zq[bad].float()).all(-1).any()
    assert torch.equal(zk[4:], yk[4:]) and torch.equal(zk[3, 2:], yk[3, 2:])
    # a head of zeros is zeros
    qi.zero_()
    assert not q.rotate(qi, ki, freqs, pos, **kwargs)[0].any()


def test_append_leaves_out():
    """Tokens in no sequence, places below 0, above the table or on pages that hold nothing: nothing of theirs is written, and all else is."""
    g = gen(8)
    H, D, P = 2, 64, 4
    c = Batch([3, 5, 2], [2, 13, 6], H, D, P, seed=3, fill=7.0)     # the first has a token at place -1
    c.pages[1, 2] = 1000                                            # places 8 .. 11 hold nothing
    T = c.T + 4                                                     # four tokens behind the last sequence
    qi, ki, vi, qw, kw, freqs, _, pos = inputs(g, T, 4, H, D, "bf16", "bf16", D, 1)
    k, v, pages, starts, lens = c.on()
    lens[2] = 100                                                   # the table holds 16 places: the last two of them are new
    c.lengths[2] = pages.shape[1] * P
    out = torch.full((T, 4, D), 5.0, device=DEV, dtype=torch.bfloat16)
    q.append(qi, ki, vi, freqs, k, v, pages, starts, lens, q_weight=qw, k_weight=kw, positions=pos, out=out)
    want, size = rotate64(qi.cpu(), qw.cpu(), 1e-6, angles_of(pos, None, freqs, T), False)
    check_rounded(out[:c.T], want[:c.T], size[:c.T], "bf16")
    assert (out[c.T:] == 5).all()
    wk, wv, t = c.k.clone(), c.v.clone(), 0
    for b, (m, n) in enumerate(zip(c.new, c.lengths)):
        for j in range(n - m, n):
            at = c.row(b, j)
            if at:
                wv[at] = vi[t].cpu()
                wk[at] = k.cpu()[at]
            t += 1
    assert torch.equal(v.cpu(), wv) and torch.equal(k.cpu(), wk)


def test_streams_and_graph():
    g = gen(9)
    T, H, D, P = 6, 2, 64, 16
    c = Batch([4, 2], [20, 37], H, D, P, seed=4)
    qi, ki, vi, qw, kw, freqs, _, _ = inputs(g, T, 4, H, D, "bf16", "bf16", D, 1)
    k, v, pages, starts, lens = c.on()
    call = lambda kk, vv, out=None, stream=None: q.append(qi, ki, vi, freqs, kk, vv, pages, starts, lens, q_weight=qw, k_weight=kw, out=out,
                                                          stream=stream)
    want = call(k, v)
    k2, v2, *_ = c.on()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(k2, v2, stream=s)
    s.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))       # what was never written is NaN
    assert torch.equal(got, want) and same(k2, k) and same(v2, v)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(k2, v2, out)
    for i in range(3):
        qi.copy_(torch.randn(qi.shape, generator=g).to(qi.dtype))
        lens.copy_(c.lens - i)
        k.fill_(1.0), k2.fill_(1.0)
        want = call(k, v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(k2, k)


def test_no_tokens():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    a, b = q.rotate(z(0, 4, 64), z(0, 2, 64), None, None)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    i = lambda *s: z(*s, dt=torch.int32)
    assert q.append(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), None, z(3, 4, 2, 64), z(3, 4, 2, 64), i(1, 2), i(2), i(1)).shape == (0, 4, 64)


@pytest.mark.parametrize("B", [64, 65, 200, 4096, 4097, 9000])
def test_many_sequences(B):
    """Places of tokens among thousands of sequences, some of them empty, some of several tokens."""
    new = torch.arange(B) % 3
    new[5], new[-1] = 0, 2
    starts = torch.cat([torch.zeros(1), new.cumsum(0)]).int()
    T, H, D, P = int(starts[-1]), 1, 16, 4
    lengths = (new + torch.arange(B) % 5).int()
    pages = torch.arange(2 * B).int().reshape(B, 2)
    g = gen(B)
    k, v = (torch.randn(T, H, D, generator=g).bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(2 * B, P, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q.append(k.to(DEV), k.to(DEV), v.to(DEV), None, kc, vc, pages.to(DEV), starts.to(DEV), lengths.to(DEV))
    seq = torch.repeat_interleave(torch.arange(B), new)
    place = torch.arange(T) - starts[seq] + (lengths - new)[seq]
    for cache, x in ((kc, k), (vc, v)):
        want = torch.zeros(2 * B * P, H, D, dtype=torch.bfloat16)
        want[seq * 2 * P + place] = x
        assert torch.equal(cache.cpu().reshape(-1, H, D), want)


@pytest.mark.parametrize("eps", [0.0, 1e-45, 2.0 ** -130, 1e-6])
@pytest.mark.parametrize("x,out", [("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("D,R", [(64, 32), (24, 24), (256, 0)])
def test_norms_of_any_size(D, R, x, out, eps):
    """Heads from the smallest numbers to the largest, whose squares fp32 does not hold, and others beside them."""
    g = gen(D)
    sizes = [-148, -140, -126, -110, -75, -70, -64, -60, -50, -40, 0, 40, 60, 63, 64, 70, 100, 125]
    T, H = len(sizes), 3
    xs = torch.rand(T, H, D, generator=g).double() * (1 - 2 * torch.randint(0, 2, (T, H, D), generator=g)) * 2.0 ** torch.tensor(sizes).double().reshape(T, 1, 1)
    xs[:, 1] = torch.randn(T, D, generator=g).double()             # an ordinary head beside each
    xs[5, 2, 0] = 2.0 ** 90                                        # one value above all others of its head
    xs = xs.float().to(TORCH[x])
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(TORCH[x])
    freqs = (10000.0 ** (-torch.arange(R // 2) / max(R // 2, 1))).float() if R else None
    pos = torch.randint(0, 500, (T,), generator=g).int()
    dev = lambda t: None if t is None else t.to(DEV)
    got, _ = q.rotate(dev(xs), dev(xs), dev(freqs), dev(pos), q_weight=dev(w), k_weight=dev(w), eps=eps, out_dtype=TORCH[out])
    held = float(torch.tensor(eps, dtype=torch.float32))           # eps as the call holds it
    want, size = rotate64(xs, w, held, angles_of(pos, None, freqs, T), False)
    there = xs.double().abs().amax(-1) > 0                         # bf16 holds nothing of the smallest: 0 / 0 without eps
    there |= torch.tensor(held > 0)
    assert there.any(-1).all()
    check_rounded(got.cpu()[there], want[there], size[there], out)


@pytest.mark.parametrize("T,Hq,Hk,D", [(2 ** 22, 1, 1, 8), (70001, 16, 2, 16), (3, 1024, 1024, 256)])
def test_as_many_tokens_and_heads_as_there_may_be(T, Hq, Hk, D):
    g = torch.Generator(device=DEV).manual_seed(T)
    x, y = (torch.randn(T, h, D, generator=g, device=DEV).bfloat16() for h in (Hq, Hk))
    w = torch.rand(D, generator=g, device=DEV) + 0.5
    freqs = torch.rand(D // 2, generator=g, device=DEV)
    pos = torch.randint(0, 1000, (T,), generator=g, device=DEV).int()
    got = q.rotate(x, y, freqs, pos, q_weight=w, k_weight=w)
    some = torch.cat([torch.arange(min(T, 5)), torch.arange(max(0, T - 5), T), torch.randint(0, T, (200,), generator=gen(1))])
    on = some.to(DEV)
    for out, x in zip(got, (x, y)):
        want, size = rotate64(x[on].cpu(), w.cpu(), 1e-6, angles_of(pos[on], None, freqs, len(some)), False)
        check_rounded(out[on], want, size, "bf16")
