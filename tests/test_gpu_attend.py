"""qmv_attend against a plain 64-bit form."""
import math

import pytest
import torch

import bit_quantized_gemv_amd as q
from attn_util import DEV, TORCH, Batch, attend64, check_attend, gen

pytestmark = pytest.mark.gpu


def queries(c, Hq, seed=1, more=0, size=2.0):
    return (size * torch.randn(c.T + more, Hq, c.D, generator=gen(seed))).to(TORCH[c.dt])


def run(c, qs, **kw):
    return q.attend(qs.to(DEV), *c.on(), **kw)


def check(c, Hq, out="bf16", seed=1, window=0, sinks=0, scale=None, **kw):
    qs = queries(c, Hq, seed)
    got = run(c, qs, window=window, sinks=sinks, scale=scale, out_dtype=TORCH[out], **kw)
    check_attend(got, *attend64(qs, c, window, sinks, scale), c.dt, out, f"{c.new} {c.lengths}")
    return qs, got


# head sizes, groups of heads, page sizes, orders, types
SHAPES = [(64, 2, 1, 16, "page", "bf16", "bf16"), (128, 2, 4, 16, "page", "bf16", "f32"), (256, 1, 2, 32, "head", "f16", "f32"),
          (80, 2, 5, 17, "one", "f16", "bf16"), (8, 1, 1, 1, "page", "bf16", "f32"), (96, 3, 3, 5, "head", "bf16", "bf16"),
          (200, 1, 16, 64, "page", "bf16", "bf16"), (136, 2, 7, 100, "one", "f16", "f32"), (24, 4, 8, 3, "page", "f16", "bf16")]
# new tokens and lengths: one token; verify blocks; blocks that begin a sequence; chunks; all of them
BATCHES = [([1], [1]), ([1], [300]), ([13], [13]), ([5, 1, 16], [700, 2, 40]), ([33], [33]), ([70, 1, 0, 17], [331, 129, 9, 530])]


@pytest.mark.parametrize("new,lengths", BATCHES)
@pytest.mark.parametrize("D,H,G,P,order,dt,out", SHAPES)
def test_shapes(D, H, G, P, order, dt, out, new, lengths):
    check(Batch(new, lengths, H, D, P, dt, seed=D + P, order=order), H * G, out)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1025, 2048, 2049, 4100])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths(length, D):
    n = min(length, 3)
    check(Batch([n], [length], 1, D, 16, seed=length), 2, "f32")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_new_tokens(n, G):
    check(Batch([n, 1], [n + 90, 5], 1, 64, 16, seed=n), G)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (64, 4), (100, 70), (300, 300), (5000, 3), (7, 600)])
@pytest.mark.parametrize("new,lengths", [([1], [900]), ([13, 1], [1300, 20]), ([150, 40], [700, 40])])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(window, sinks, new, lengths, D):
    check(Batch(new, lengths, 2, D, 16, seed=window), 4, "f32", window=window, sinks=sinks)


def test_long_window():
    """Blocks far apart: the first tokens and the last of a long sequence."""
    check(Batch([4], [9000], 1, 64, 16, seed=1), 2, "f32", window=700, sinks=5)
    check(Batch([40], [9000], 1, 128, 64, seed=2), 2, "bf16", window=500, sinks=300)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3])
def test_scale(scale):
    check(Batch([3, 20], [100, 60], 2, 64, 16), 4, "f32", scale=scale)


def test_large_logits():
    """Weights that all but one key have lost, in every block of keys."""
    c = Batch([3, 30], [600, 333], 1, 128, 16, seed=3)
    qs = queries(c, 2, size=60.0)
    out, reach = attend64(qs, c)
    got = run(c, qs, out_dtype=torch.float32).cpu().double()
    # logits of several hundred: an fp32 sum of 128 products is off by up to 2^-17 of their size
    assert ((got - out).abs() <= 2.0 ** -17 * 128 * 60 * 3 / 128 ** 0.5 * reach.amax(-1, keepdim=True) + 2.0 ** -15 * reach).all()


def test_nothing_to_see():
    """Tokens at places below 0, sequences of no places, pages that hold nothing: zeros."""
    c = Batch([5, 2, 20], [3, 0, 11], 2, 64, 4, seed=4)
    qs, got = check(c, 4)
    assert not got[:2].any() and not got[5:7].any() and not got[7:16].any()
    c = Batch([2, 30], [7, 40], 2, 64, 4, seed=5)
    c.pages[:] = -1
    assert not run(c, queries(c, 4)).any()


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_bad_pages(bad):
    """A page outside the cache holds nothing."""
    for new in (2, 50):
        c = Batch([new, 1], [333, 90], 2, 64, 8, seed=6)
        for b, i in ((0, 0), (0, 7), (0, 20), (0, 41), (1, 3)):
            c.pages[b, i] = bad
        check(c, 4, "f32")


def test_lengths_beyond_the_table():
    c = Batch([2, 40], [64, 64], 2, 64, 16, seed=7)
    qs = queries(c, 2)
    k, v, pages, starts, lens = c.on()
    lens.fill_(2 ** 30)
    check_attend(q.attend(qs.to(DEV), k, v, pages, starts, lens), *attend64(qs, c), "bf16", "bf16")
    # max_length below them: the same as sequences of that length
    c.lengths = [50, 50]
    check_attend(q.attend(qs.to(DEV), k, v, pages, starts, lens, max_length=50), *attend64(qs, c), "bf16", "bf16")


def test_starts_out_of_order():
    """Starts outside the tokens and going back: what lies in a sequence is computed, nothing else is touched."""
    c = Batch([4, 3], [30, 30], 1, 64, 16, seed=8)
    qs = queries(c, 2).to(DEV)
    k, v, pages, _, lens = c.on()
    for s in ([0, 7, 3], [-5, 4, 100], [7, 7, 7], [2 ** 31 - 1, -2 ** 31, 5]):
        out = torch.full((7, 2, 64), 3.0, device=DEV)
        q.attend(qs, k, v, pages, torch.tensor(s, dtype=torch.int32, device=DEV), lens, out=out)
        torch.cuda.synchronize()
        if s == [7, 7, 7]:
            assert (out == 3).all()


def test_rows_behind_and_above():
    """Tokens behind the last sequence, and above max_new, are left as they were."""
    c = Batch([3, 9], [50, 70], 2, 64, 16, seed=9)
    qs = queries(c, 4, more=5)
    want, reach = attend64(qs, c)
    out = torch.full((17, 4, 64), 8.0, device=DEV)
    q.attend(qs.to(DEV), *c.on(), out=out)
    check_attend(out[:12], want[:12], reach[:12], "bf16", "f32")
    assert (out[12:] == 8).all()
    out.fill_(8.0)
    q.attend(qs.to(DEV), *c.on(), out=out, max_new=4)
    check_attend(out[:7], want[:7], reach[:7], "bf16", "f32")
    assert (out[7:] == 8).all()


@pytest.mark.parametrize("new", [3, 13, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 5)])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_hidden_values(new, window, sinks, junk):
    """What a token does not see does not touch its output: the same bits with NaN or infinities there."""
    c = Batch([new], [400], 2, 128, 16, seed=10, fill=0.0)
    qs = queries(c, 4)
    clean = run(c, qs, window=window, sinks=sinks, out_dtype=torch.float32)
    places = [400 - new // 2 - 1]                      # the second half of the new tokens sees it
    if window:
        places += [400 - new - 30, 9]                  # the first tokens see it, or none
    for j in places:
        c.k[c.row(0, j)] = junk
        c.v[c.row(0, j)] = junk
    got = run(c, qs, window=window, sinks=sinks, out_dtype=torch.float32)
    for i in range(new):
        p = 400 - new + i
        sees = any(j <= p and (not window or j > p - window or j < sinks) for j in places)
        if not sees:
            assert torch.equal(got[i], clean[i]), i
        elif junk != -math.inf:
            assert not torch.isfinite(got[i]).any(), i


@pytest.mark.parametrize("D,dt", [(64, "bf16"), (128, "f16"), (256, "bf16"), (80, "f16")])
@pytest.mark.parametrize("window", [0, 200])
def test_blocks_as_single_tokens(D, dt, window):
    """Up to 16 new tokens of a sequence get the bits that calls of one token get, whatever else is in the call."""
    length, n = 2700, 13
    c = Batch([n, 16], [length, 300], 2, D, 16, dt, seed=11)
    qs = queries(c, 6).to(DEV)
    k, v, pages, starts, lens = c.on()
    kw = dict(window=window, sinks=3 if window else 0)
    whole = q.attend(qs, k, v, pages, starts, lens, out_dtype=torch.float32, **kw)
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for i in range(n):
        got = q.attend(qs[i:i + 1], k, v, pages[:1], one, lens[:1] - (n - 1 - i), out_dtype=torch.float32, **kw)
        assert torch.equal(got[0], whole[i]), i
    many = 40                                         # many sequences: other launch shapes
    rep = q.attend(qs[:n].repeat(many, 1, 1), k, v, pages[:1].repeat(many, 1), torch.arange(many + 1, dtype=torch.int32, device=DEV) * n,
                   lens[:1].repeat(many), max_new=n, out_dtype=torch.float32, **kw)
    assert torch.equal(rep.reshape(many, n, 6, D), whole[:n].expand(many, n, 6, D))
    again = q.attend(qs, k, v, pages, starts, lens, out_dtype=torch.float32, max_new=16, max_length=length, **kw)
    assert torch.equal(again, whole)


@pytest.mark.parametrize("D,Hq,Hkv,n", [(64, 32, 2, 13), (128, 64, 8, 13), (128, 20, 4, 16), (256, 16, 8, 13), (256, 32, 4, 16), (96, 9, 3, 5)])
@pytest.mark.parametrize("window", [0, 333])
def test_row_tiles(D, Hq, Hkv, n, window):
    """Blocks of one to many tiles of rows, in calls that are cut up in different ways: the same bits."""
    length = 1900
    c = Batch([n], [length], Hkv, D, 16, seed=D + n)
    qs = queries(c, Hq).to(DEV)
    k, v, pages, starts, lens = c.on()
    kw = dict(window=window, sinks=5 if window else 0)
    whole = q.attend(qs, k, v, pages, starts, lens, **kw)
    check_attend(whole, *attend64(qs.cpu(), c, **kw), "bf16", "bf16")
    many = 70
    rep = q.attend(qs.repeat(many, 1, 1), k, v, pages.repeat(many, 1), torch.arange(many + 1, dtype=torch.int32, device=DEV) * n, lens.repeat(many),
                   max_new=n, max_length=length, **kw)
    assert torch.equal(rep.reshape(many, n, Hq, D), whole.expand(many, n, Hq, D))
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for i in (0, n - 1):
        got = q.attend(qs[i:i + 1], k, v, pages, one, lens - (n - 1 - i), **kw)
        assert torch.equal(got[0], whole[i]), i
    # beside a chunk, and with loose bounds
    c2 = Batch([n, 40], [length, 100], Hkv, D, 16, seed=D + n)
    k2, v2, pages2, starts2, lens2 = c2.on()
    q2 = torch.cat([qs, queries(c2, Hq)[n:].to(DEV)])
    again = q.attend(q2, k2, v2, pages2, starts2, lens2, **kw)
    alone = q.attend(qs, k2, v2, pages2[:1], starts2[:2], lens2[:1], **kw)
    assert torch.equal(again[:n], alone)


def of(c, qs, order, pages=None):
    """The call of a batch's sequences in another order, some of them more than once: q, then the rest."""
    k, v, table, _, lens = c.on()
    starts = c.starts.tolist()
    at = torch.tensor(order, device=DEV)
    new = torch.cat([qs[starts[b]:starts[b + 1]] for b in order]).to(DEV)
    begin = torch.tensor([0] + [c.new[b] for b in order]).cumsum(0).int().to(DEV)
    return new, k, v, (table if pages is None else pages)[at], begin, lens[at]


@pytest.mark.parametrize("D,Hq,Hkv,n,out", [(128, 8, 8, 1, "bf16"), (64, 12, 4, 13, "f32"), (256, 6, 2, 5, "bf16"), (128, 24, 2, 7, "f32"), (64, 8, 4, 3, "bf16")])
def test_wide_bounds(D, Hq, Hkv, n, out):
    """Bounds far above the lengths: workgroups that take many units each, most of them without work; the same bits."""
    P, lengths = 64, [9000, n, 1025, 33000, 1024, 6200, 2 * 8192]
    c = Batch([n] * 7, lengths, Hkv, D, P, seed=D + n)
    qs = queries(c, Hq)
    order = [i % 7 for i in range(70)]
    new, k, v, pages, begin, lens = of(c, qs, order)
    kw = dict(max_new=n, out_dtype=TORCH[out])
    tight = torch.cat([q.attend(qs[n * b:n * b + n].to(DEV), k, v, pages[b:b + 1], begin[:2], lens[b:b + 1], max_length=lengths[b], **kw) for b in range(7)])
    wide = torch.full((70, (1 << 22) // P), -1, dtype=torch.int32, device=DEV)
    wide[:, :pages.shape[1]] = pages
    got = q.attend(new, k, v, wide, begin, lens, **kw)
    assert torch.equal(got.reshape(10, 7 * n, Hq, D), tight.expand(10, 7 * n, Hq, D))
    ref = Batch([n], [lengths[5]], Hkv, D, P)
    ref.k, ref.v, ref.pages = c.k, c.v, c.pages[5:6]
    check_attend(tight[5 * n:6 * n], *attend64(qs[5 * n:6 * n], ref), "bf16", out)


@pytest.mark.parametrize("window,H,G,D", [(0, 2, 4, 64), (200, 2, 4, 64), (0, 4, 6, 64), (300, 1, 16, 128), (0, 4, 5, 40)])
def test_chunks_among_many(window, H, G, D):
    """Chunks here and there among hundreds of sequences, blocks of one and of many tokens beside them."""
    c = Batch([1, 16, 40, 0, 17, 3], [1300, 2100, 40, 77, 1500, 3], H, D, 16, seed=window)
    qs = queries(c, H * G)
    kw = dict(window=window, sinks=3 if window else 0)
    want, reach = attend64(qs, c, **kw)
    order = [0, 3, 0, 5] * 50 + [2, 1, 0, 4] + [0, 5, 3] * 40 + [1, 2, 2, 4, 0]
    new, k, v, pages, begin, lens = of(c, qs, order)
    got = q.attend(new, k, v, pages, begin, lens, **kw)
    alone = {}
    for i, b in enumerate(order):
        a, z, s = int(begin[i]), int(begin[i + 1]), c.starts.tolist()
        if c.new[b] > 16:
            check_attend(got[a:z], want[s[b]:s[b + 1]], reach[s[b]:s[b + 1]], "bf16", "bf16", (i, b))
        elif c.new[b]:
            if b not in alone:
                alone[b] = q.attend(new[a:z], k, v, pages[i:i + 1], begin[i:i + 2] - a, lens[i:i + 1], **kw)
                check_attend(alone[b], want[s[b]:s[b + 1]], reach[s[b]:s[b + 1]], "bf16", "bf16", b)
            assert torch.equal(got[a:z], alone[b]), (i, b)


@pytest.mark.parametrize("B", [1, 16, 40, 41])
@pytest.mark.parametrize("G,D", [(16, 64), (7, 200)])
def test_shares_among_many(B, G, D):
    """A chunk whose keys several workgroups share, first and last of sequences of single tokens."""
    c = Batch([300, 1, 11, 130], [1500, 1100, 700, 2000], 1, D, 32, seed=B)
    qs = queries(c, G)
    want, reach = attend64(qs, c)
    order = [0] + [1, 2, 1] * (B // 3) + [3]
    new, k, v, pages, begin, lens = of(c, qs, order)
    got = q.attend(new, k, v, pages, begin, lens, out_dtype=torch.float32)
    s = c.starts.tolist()
    for i, b in enumerate(order):
        a, z = int(begin[i]), int(begin[i + 1])
        check_attend(got[a:z], want[s[b]:s[b + 1]], reach[s[b]:s[b + 1]], "bf16", "f32", (i, b))
    assert torch.equal(q.attend(new, k, v, pages, begin, lens, out_dtype=torch.float32), got)


@pytest.mark.parametrize("bound", [1, 5, 16, 17, 30])
def test_more_new_than_bound(bound):
    """The first max_new tokens of a sequence, at their places; the rows of the others as they were."""
    c = Batch([40, 3], [700, 500], 2, 128, 16)
    qs = queries(c, 4)
    want, reach = attend64(qs, c)
    out = torch.full((43, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    run(c, qs, max_new=bound, out=out)
    for a, n in ((0, min(bound, 40)), (40, min(bound, 3))):
        check_attend(out[a:a + n], want[a:a + n], reach[a:a + n], "bf16", "bf16")
    assert (out[min(bound, 40):40] == 7).all() and (out[40 + min(bound, 3):] == 7).all()


@pytest.mark.parametrize("H", [1, 2])
def test_very_long(H):
    """More leaves and supers than a join takes in one round."""
    c = Batch([2], [70001], H, 256, 64, seed=H)
    qs = queries(c, H)
    kw = dict(out_dtype=torch.float32)
    got = run(c, qs, **kw)
    check_attend(got, *attend64(qs, c), "bf16", "f32")
    k, v, pages, starts, lens = c.on()
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for i in range(2):
        assert torch.equal(q.attend(qs[i:i + 1].to(DEV), k, v, pages, one, lens - 1 + i, **kw)[0], got[i])
    three = q.attend(qs.repeat(3, 1, 1).to(DEV), k, v, pages.repeat(3, 1), torch.arange(4, dtype=torch.int32, device=DEV) * 2, lens.repeat(3), **kw)
    assert torch.equal(three.reshape(3, 2, H, 256), got.expand(3, 2, H, 256))


@pytest.mark.parametrize("n,length,D", [(17, 20000, 64), (50, 9000, 256), (130, 5000, 192)])
def test_shared_keys(n, length, D):
    """Few rows over many keys: workgroups share the keys, and their parts are joined."""
    check(Batch([n], [length], 1, D, 32, seed=n), 1, "f32")


def test_chunks_repeat():
    """The same call again gives the same bits."""
    c = Batch([300, 2, 77], [900, 50, 77], 2, 128, 16, seed=12)
    qs = queries(c, 8)
    a, b = run(c, qs), run(c, qs)
    assert torch.equal(a, b)


def test_strided_queries():
    c = Batch([4, 30], [60, 90], 2, 64, 16, seed=13)
    qs = queries(c, 4)
    big = torch.randn(c.T, 10, 64).bfloat16().to(DEV)
    big[:, 3:7] = qs.to(DEV)
    assert torch.equal(q.attend(big[:, 3:7], *c.on()), run(c, qs))
    turned = qs.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(q.attend(turned, *c.on()), run(c, qs))


def test_shared_pages():
    """Sequences of a common beginning may hold it once, and a page may be in one's table twice."""
    c = Batch([2, 2], [64, 64], 2, 64, 16, seed=14)
    c.pages[1, :2] = c.pages[0, :2]
    c.pages[0, 3] = c.pages[0, 2]
    check(c, 4, "f32")


def test_wide_table():
    """A slice of a wider table, with more pages than the sequences have."""
    c = Batch([3, 1], [70, 500], 2, 64, 16, seed=15, wide=50)
    qs = queries(c, 4)
    k, v, pages, starts, lens = c.on()
    wide = torch.full((2, 200), 10 ** 6, dtype=torch.int32, device=DEV)
    wide[:, 7:7 + pages.shape[1]] = pages
    got = q.attend(qs.to(DEV), k, v, wide[:, 7:7 + pages.shape[1]], starts, lens)
    check_attend(got, *attend64(qs, c), "bf16", "bf16")


def test_far_pages():
    """Pages whose offsets pass 32 bits, in elements and bytes."""
    D, P, H = 128, 16, 1
    n_pages = 2 ** 32 // (P * D) + 40                 # 8 GiB of keys, of which a few pages are used
    k = torch.empty(n_pages, P, H, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty(n_pages, P, H, D, dtype=torch.bfloat16, device=DEV)
    for new, length in ((2, 100), (40, 100)):
        c = Batch([new], [length], H, D, P, seed=16)
        qs = queries(c, 2)
        ids = torch.randperm(40, generator=gen(1))[:7] + n_pages - 40
        for i in range(7):
            k[ids[i]], v[ids[i]] = c.k[c.pages[0, i].long()].to(DEV), c.v[c.pages[0, i].long()].to(DEV)
        got = q.attend(qs.to(DEV), k, v, ids.int().reshape(1, -1).to(DEV), c.starts.to(DEV), c.lens.to(DEV))
        check_attend(got, *attend64(qs, c), "bf16", "bf16")


def test_streams_and_graphs():
    c = Batch([5, 30, 1], [300, 100, 1000], 2, 64, 16, seed=17)
    qs = queries(c, 4).to(DEV)
    args = c.on()
    want = q.attend(qs, *args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = q.attend(qs, *args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    outs, graphs = [torch.empty_like(want) for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    for o, gr in zip(outs, graphs):
        with torch.cuda.graph(gr):
            q.attend(qs, *args, out=o)
    g = gen(3)
    for i in range(4):
        qs.copy_(torch.randn(qs.shape, generator=g).to(qs.dtype))
        args[4].copy_(c.lens - i)
        want = q.attend(qs, *args)
        torch.cuda.synchronize()
        for o, gr in zip(outs, graphs):
            o.zero_()
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_no_tokens():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    i = lambda *s: z(*s, dt=torch.int32)
    assert q.attend(z(0, 4, 64), z(3, 4, 2, 64), z(3, 4, 2, 64), i(1, 2), i(2), i(1)).shape == (0, 4, 64)
    out = torch.full((3, 4, 64), 2.0, device=DEV)
    q.attend(z(3, 4, 64), z(3, 4, 2, 64), z(3, 4, 2, 64), i(0, 2), i(1), i(0), out=out)
    assert (out == 2).all()


@pytest.mark.parametrize("D,window,many", [(256, 0, 1025), (256, 200, 1025), (128, 0, 2100)])
def test_shared_chunks_among_thousands(D, window, many):
    """Chunks whose keys several workgroups share, beside blocks of one part, among so many sequences that a workgroup of the join
    takes all rows of its own."""
    c = Batch([1, 17, 17, 0, 3], [500, 512, 300, 9, 70], 1, D, 16, seed=D)
    qs = queries(c, 2)
    kw = dict(window=window, sinks=3 if window else 0)
    want, reach = attend64(qs, c, **kw)
    order = ([0, 4, 0, 3, 4] * many)[:many - 6] + [1, 0, 2, 3, 1, 4]
    new, k, v, pages, begin, lens = of(c, qs, order)
    out = torch.full((new.shape[0] + 7, 2, D), 9.0, device=DEV)
    q.attend(torch.cat([new, new[:7]]), k, v, pages, begin, lens, out=out, max_new=17, max_length=512, **kw)
    s, n = c.starts.tolist(), int(begin[-1])
    rows = torch.tensor([s[b] + i for b in order for i in range(c.new[b])])
    check_attend(out[:n], want[rows], reach[rows], "bf16", "f32")
    assert (out[n:] == 9).all()


def peaked(new, length, D, gap, far, seed):
    """fp16 keys of which the first outweighs each other one by about 2^gap, and holds the value 0; or, if `far`, the last that all see."""
    c = Batch([new], [length], 1, D, 16, "f16", seed=seed)
    qs = queries(c, 2)
    qs[..., 0] = 8.0
    top = length - new if far else 0
    for j in range(length):
        at = c.row(0, j)
        c.k[at][..., 1:] *= 0.25
        c.k[at][..., 0] = gap * math.log(2.0) / 8.0 * D ** 0.5 if j == top else 0.0
        if j == top:
            c.v[at] = 0.0
    return c, qs


@pytest.mark.parametrize("gap", [16, 20, 24, 26])
@pytest.mark.parametrize("new,length", [(1, 4096), (13, 4096), (100, 4096), (20, 700)])
@pytest.mark.parametrize("D,far", [(64, False), (128, True)])
def test_peaks(new, length, D, far, gap):
    """A key that takes nearly all the weight, and adds nothing: what the others add, in one share of the keys and in several.

    check_attend's bound, which counts half a step of each weight, holds without more: fp16 weights are held to 2^-36 of the largest for
    bf16 outputs, 2^-10 of a weight of 2^-26, and to 2^-39 for fp32 ones, 2^-13 of it; rounded up as often as down, the errors of 700 keys
    or more add up to 2^-10 / sqrt(3 * 700) = 2.1e-5 of what they weigh, beside 2^-11, and to 2.7e-6, beside 2e-5."""
    c, qs = peaked(new, length, D, gap, far, seed=gap)
    want, reach = attend64(qs, c)
    for out in ("f32", "bf16"):
        check_attend(run(c, qs, out_dtype=TORCH[out]), want, reach, "f16", out, "shared")
        many = 140          # enough rows that a chunk's keys are one workgroup's
        new_q, *args = of(c, qs, [0] * many)
        got = q.attend(new_q, *args, out_dtype=TORCH[out], max_new=new, max_length=length)
        check_attend(got[-new:], want, reach, "f16", out, "one share")
        assert torch.equal(got, got[:new].repeat(many, 1, 1))


@pytest.mark.parametrize("new", [1, 5, 60])
@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f16", "bf16")])
def test_scale_zero_of_large_scores(new, dt, out):
    """A scale of 0 weighs all places alike, however large q . k is."""
    c = Batch([new], [100], 2, 64, 16, dt, seed=20)
    c.k *= 2.0 ** 58 if dt == "bf16" else 2.0 ** 12
    qs = queries(c, 4) * (2.0 ** 58 if dt == "bf16" else 2.0 ** 12)
    assert torch.isfinite(qs).all()
    check_attend(run(c, qs, scale=0.0, out_dtype=TORCH[out]), *attend64(qs, c, scale=0.0), dt, out)


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("T", [7, 60, 400])
@pytest.mark.parametrize("starts,ends", [((0, 7, 3), ((0, 7), (7, 7))), ((-5, 4, 100), ((0, 4), (4, 7))), ((7, 7, 7), ((7, 7), (7, 7))),
                                         ((HIGH, LOW, 5), ((7, 7), (0, 5))), ((3, 5, 6), ((3, 5), (5, 6))), ((6, LOW, LOW), ((6, 6), (0, 0))),
                                         ((7, -100, HIGH), ((7, 7), (0, 7)))])
def test_starts_of_any_value(T, starts, ends):
    """Starts are taken into the tokens: those of a sequence are computed, and no other row is touched. Sevenths of T."""
    at = lambda i: i if abs(i) > 1000 else i * T // 7
    c = Batch([1, 1], [T + 23, 500], 2, 64, 16, "bf16", seed=8)
    starts, ends = [at(i) for i in starts], [(at(a), at(z)) for a, z in ends]
    qs = torch.randn(T, 4, 64, generator=gen(9)).bfloat16()
    want, reach, mine = torch.zeros(T, 4, 64, dtype=torch.float64), torch.zeros(T, 4, 64, dtype=torch.float64), torch.zeros(T, dtype=torch.bool)
    for b, (a, z) in enumerate(ends):
        c.new, c.starts = [0, 0], torch.tensor([0, 0, 0])
        c.new[b], c.starts[b] = z - a, a
        w, r = attend64(qs, c)
        want[a:z], reach[a:z], mine[a:z] = w[a:z], r[a:z], True
    k, v, pages, _, lens = c.on()
    whole = torch.full((3 * T, 4, 64), 3.0, device=DEV)           # the rows before and behind the call's own
    q.attend(qs.to(DEV), k, v, pages, torch.tensor(starts, dtype=torch.int32, device=DEV), lens, out=whole[T:2 * T])
    out = whole[T:2 * T].cpu()
    check_attend(out[mine], want[mine], reach[mine], "bf16", "f32")
    assert (out[~mine] == 3).all() and (whole[:T] == 3).all() and (whole[2 * T:] == 3).all()


@pytest.mark.parametrize("new", [3, 13, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 5)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_seen_values(new, window, sinks, dt, junk):
    """An infinity or NaN among the values alone: no output that has met it is a number, in its column, and all else keeps its bits."""
    c = Batch([new], [400], 2, 128, 16, dt, seed=21, fill=0.0)
    qs = queries(c, 4, size=1.0)
    clean = run(c, qs, window=window, sinks=sinks, out_dtype=torch.float32)
    place = 400 - new // 2 - 1                         # the second half of the new tokens sees it
    c.v[c.row(0, place)][:, 5] = junk
    got = run(c, qs, window=window, sinks=sinks, out_dtype=torch.float32)
    sees = torch.arange(400 - new, 400) >= place
    assert sees.any() and not (new > 3 and sees.all())
    assert torch.equal(got[~sees.to(DEV)], clean[~sees.to(DEV)])
    other = torch.arange(128) != 5
    assert not torch.isfinite(got[sees.to(DEV)][..., 5]).any() and torch.isfinite(got[..., other.to(DEV)]).all()
    assert torch.equal(got[..., other.to(DEV)], clean[..., other.to(DEV)])


@pytest.mark.parametrize("new", [3, 13, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 5)])
@pytest.mark.parametrize("what", ["k", "kv"])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_seen_keys(new, window, sinks, what, junk):
    """Keys of infinities or NaN, whose scores are NaN where queries have both signs: nothing of the rows that see one is a number, and
    the others keep their bits."""
    c = Batch([new], [400], 2, 128, 16, seed=10, fill=0.0)
    qs = queries(c, 4)
    clean = run(c, qs, window=window, sinks=sinks, out_dtype=torch.float32)
    places = [400 - new // 2 - 1] + ([400 - new - 30, 9] if window else [])
    for j in places:
        c.k[c.row(0, j)] = junk
        if what == "kv":
            c.v[c.row(0, j)] = junk
    got = run(c, qs, window=window, sinks=sinks, out_dtype=torch.float32)
    for i in range(new):
        p = 400 - new + i
        if any(j <= p and (not window or j > p - window or j < sinks) for j in places):
            assert not torch.isfinite(got[i]).any(), i
        else:
            assert torch.equal(got[i], clean[i]), i


@pytest.mark.parametrize("new", [1, 4, 40])
def test_scores_of_minus_infinity(new):
    """A key whose score is -inf weighs nothing, and a row that sees no other is zeros."""
    c = Batch([new], [new + 2], 1, 64, 4, seed=22)
    qs = queries(c, 2)
    qs[..., 0] = -1.0
    ref = Batch([new], [new + 2], 1, 64, 4, seed=22)
    ref.pages[0, 0] = -1                               # places 0 to 3 hold nothing
    for j in range(4):
        if c.row(0, j):
            c.k[c.row(0, j)][..., 0] = math.inf
    check_attend(run(c, qs, out_dtype=torch.float32), *attend64(qs, ref), "bf16", "f32")


@pytest.mark.parametrize("T", [1, 16, 17, 40])
@pytest.mark.parametrize("Hq,Hkv,D", [(1024, 1024, 8), (1024, 1, 8), (1000, 8, 16), (1024, 2, 64), (1023, 1, 128)])
def test_many_heads(T, Hq, Hkv, D):
    n, G = T + 40, Hq // Hkv
    c = Batch([T], [n], Hkv, D, 16, seed=T)
    qs = queries(c, Hq, size=1.0)
    k, v = (torch.stack([t[c.row(0, j)] for j in range(n)]).double().permute(1, 0, 2) for t in (c.k, c.v))
    s = torch.matmul(qs.double().reshape(T, Hkv, G, D), k.transpose(1, 2)) / D ** 0.5
    w = torch.softmax(s.masked_fill((torch.arange(n) > 40 + torch.arange(T).unsqueeze(1)).reshape(T, 1, 1, n), -math.inf), -1)
    check_attend(run(c, qs, out_dtype=torch.float32), torch.matmul(w, v).reshape(T, Hq, D), torch.matmul(w, v.abs()).reshape(T, Hq, D), "bf16", "f32")


def test_as_many_sequences_as_there_may_be():
    """65535 sequences of one token, as blocks alone and as if there were a chunk among them."""
    B = 65535
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(4, 4, 1, 8, generator=g, device=DEV).bfloat16() for _ in range(2))
    qs = torch.randn(B, 2, 8, generator=g, device=DEV).bfloat16()
    at = torch.arange(B, device=DEV)
    pages, lens, starts = (at % 4).int().reshape(B, 1), (at % 4 + 1).int(), torch.arange(B + 1, device=DEV).int()
    got, again = (q.attend(qs, k, v, pages, starts, lens, max_new=n, out_dtype=torch.float32) for n in (1, 17))
    kk, vv = (t[at % 4, :, 0].double() for t in (k, v))
    s = torch.matmul(qs.double(), kk.transpose(1, 2).contiguous()) / 8 ** 0.5
    w = torch.softmax(s.masked_fill((torch.arange(4, device=DEV) >= lens.unsqueeze(1)).unsqueeze(1), -math.inf), -1)
    check_attend(got, torch.matmul(w, vv).cpu(), torch.matmul(w, vv.abs()).cpu(), "bf16", "f32")
    assert torch.equal(got, again)


@pytest.mark.parametrize("P,lengths", [(65536, [700, 900]), (40000, [3, 41000]), (4096, [4095, 4126])])
def test_large_pages(P, lengths):
    check(Batch([3, 20], lengths, 1, 16, P, seed=1), 2, "f32")
