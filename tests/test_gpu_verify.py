"""verify on the GPU against a plain 64-bit form, and its borders."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_gemv_amd as q
from ops_util import DEV, TORCH, gen

pytestmark = pytest.mark.gpu


def softmax(row, T):
    """p of one row of 64-bit logits: 0 at NaN and -inf, greedy at T <= 0, None if nothing counts."""
    row = np.where(np.isnan(row), -np.inf, row)
    top = row.max()
    if top == -np.inf:
        return None
    if not T > 0:
        p = np.zeros(len(row))
        p[int(np.argmax(row))] = 1.0
        return p
    with np.errstate(invalid="ignore"):
        e = np.where(row == top, 1.0, np.exp((row - top) / T))
    e = np.where(row == -np.inf, 0.0, e)
    return e / e.sum()


def sample(weights, u):
    c = np.cumsum(weights)
    over = np.nonzero(c > u * c[-1])[0]
    return int(over[0]) if len(over) else int(np.nonzero(weights > 0)[0][-1])


def want(logits, draft, u, probs, temp, lens):
    B, S1, V = logits.shape
    l = logits.double().numpy()
    qs = None if probs is None else probs.double().numpy()
    tokens, accepted = np.full((B, S1), -1), np.zeros(B, dtype=int)
    for b in range(B):
        n = S1 - 1 if lens is None else min(max(int(lens[b]), 0), S1 - 1)
        T = 1.0 if temp is None else float(temp[b])
        ub = u[b].double().numpy()
        j = 0
        while j < n:
            p, x = softmax(l[b, j], T), int(draft[b, j])
            qx = 1.0 if qs is None else qs[b, j, x] if 0 <= x < V else 0.0
            if p is None or not (0 <= x < V) or not ub[j] * qx < p[x]:
                break
            tokens[b, j] = x
            j += 1
        accepted[b] = j
        p = softmax(l[b, j], T)
        if p is None:
            continue
        w = p
        if j < n:
            qj = np.zeros(V)
            if qs is None:
                if 0 <= int(draft[b, j]) < V:
                    qj[int(draft[b, j])] = 1.0
            else:
                qj = qs[b, j]
            rest = np.maximum(p - qj, 0.0)
            w = rest if rest.sum() > 0 else p
        tokens[b, j] = sample(w, ub[n])
    return torch.from_numpy(tokens).int(), torch.from_numpy(accepted).int()


def problem(B, S, V, logits="f32", probs="f32", seed=1, noise=0.5):
    g = gen(seed)
    l = 2 * torch.randn(B, S + 1, V, generator=g)
    l = torch.where(torch.rand(B, S + 1, V, generator=g) < min(0.5, 20 / V), l + 6, l)
    d = l[:, :S] + noise * torch.randn(B, S, V, generator=g)
    pr = torch.softmax(d, -1)
    draft = torch.zeros(B, S, dtype=torch.int32)
    if S:
        draft = torch.multinomial(pr.reshape(B * S, V), 1, generator=g).reshape(B, S).int() if probs else d.argmax(-1).int()
    return l.to(TORCH[logits]), draft, torch.rand(B, S + 1, generator=g), pr.to(TORCH[probs]) if probs else None


def check(logits, draft, u, probs, temp=None, lens=None, **kw):
    to = lambda t: None if t is None else t.to(DEV)
    tokens, accepted = q.verify(to(logits), to(draft), to(u), draft_probs=to(probs), temperature=to(temp), lengths=to(lens), **kw)
    want_t, want_a = want(logits, draft, u, probs, temp, lens)
    assert torch.equal(accepted.cpu(), want_a), (accepted.cpu(), want_a)
    assert torch.equal(tokens.cpu(), want_t), (tokens.cpu(), want_t)
    return want_t, want_a


@pytest.mark.parametrize("logits", ["bf16", "f32"])
@pytest.mark.parametrize("probs", ["bf16", "f32", None])
@pytest.mark.parametrize("B,S,V", [(1, 0, 1), (1, 1, 2), (3, 2, 17), (5, 4, 1000), (4, 3, 4096), (4, 3, 4097), (2, 12, 50001)])
def test_types_and_sizes(logits, probs, B, S, V):
    for seed in range(4):
        check(*problem(B, S, V, logits, probs, seed=seed))


@pytest.mark.parametrize("probs", ["f32", None])
def test_temperatures_and_lengths(probs):
    B, S = 16, 6
    p = problem(B, S, 3001, "bf16", probs)
    temp = torch.tensor([0.0, 1.0, 0.3, 2.0, -1.0, 1e-6, 1e6, float("inf")] * 2)
    lens = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -3, 6, 6, 6, 6, 6, 0, 100], dtype=torch.int32)
    check(*p, temp=temp, lens=lens)
    check(*p, temp=temp)
    check(*p, lens=lens)


def test_all_accepted_and_all_rejected():
    l, draft, u, pr = problem(6, 5, 777)
    _, n = check(l, draft, torch.zeros_like(u), pr)
    assert (n == 5).all()
    never = torch.full_like(l, 0.0)
    for b in range(6):
        for j in range(5):
            never[b, j, draft[b, j]] = -math.inf
    _, n = check(never, draft, u, pr)
    assert (n == 0).all()


def test_masks():
    """-inf, the types' lowest values, NaN and +inf among the logits, and rows with nothing left."""
    l, draft, u, pr = problem(8, 3, 5000)
    l[0, :, 100:] = -math.inf
    l[1, :, ::2] = torch.finfo(torch.float32).min
    l[2, :, 7] = float("nan")
    l[3, 1] = -math.inf
    l[4, 0] = float("nan")
    l[5, 2, 4000] = math.inf
    l[5, 2, 4900] = math.inf
    l[6] = -math.inf
    l[7, :, :4999] = -math.inf
    for temp in (None, torch.zeros(8), torch.full((8,), 0.7)):
        check(l, draft, u, pr, temp=temp)
        check(l, draft, u, None, temp=temp)
    low = torch.full((1, 2, 300), torch.finfo(torch.bfloat16).min).to(torch.bfloat16)
    check(low, torch.tensor([[5]], dtype=torch.int32), torch.tensor([[0.9, 0.5]]), None)


def test_ties_go_to_the_lowest_index():
    l = torch.zeros(3, 2, 9000)
    l[:, :, [8000, 4500, 8999]] = 3.0
    draft = torch.tensor([[4500], [8000], [8999]], dtype=torch.int32)
    t, n = check(l, draft, torch.full((3, 2), 0.5), None, temp=torch.zeros(3))
    assert n.tolist() == [1, 0, 0] and t[:, 0].tolist() == [4500] * 3


def test_borders_of_a_uniform_row():
    """Equal powers of two: every prefix sum is exact, and a number on a border goes to the next index."""
    V = 8192
    l = torch.zeros(V // 64, 1, V)
    u = (torch.arange(V // 64) * 64 / V).reshape(-1, 1).float()
    t, _ = check(l, torch.zeros(V // 64, 0, dtype=torch.int32), u, None)
    assert t[:, 0].tolist() == [64 * i for i in range(V // 64)]


def test_numbers_outside_the_range():
    l, draft, u, pr = problem(4, 2, 600)
    l[:, :, 590:] = -math.inf
    u[:, 2] = torch.tensor([1.0, 2.0, 0.0, -1.0])
    u[:, :2] = 0.0
    check(l, draft, u, pr)


def test_nothing_left_of_the_target():
    """A drafter above the target everywhere: the rejected position is sampled from the target."""
    l, draft, u, pr = problem(4, 2, 600)
    check(l, draft, torch.full_like(u, 0.999), torch.ones_like(pr))


def test_tokens_outside_the_vocabulary():
    l, draft, u, pr = problem(4, 3, 500)
    draft[0, 0], draft[1, 1], draft[2, 2], draft[3, 0] = -1, 500, 2 ** 31 - 1, -2 ** 31
    check(l, draft, torch.zeros_like(u), pr)
    check(l, draft, torch.zeros_like(u), None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides(dt):
    """Rows at odd strides: a vocabulary cut from a padded one, positions cut from a longer block."""
    l, draft, u, pr = problem(3, 4, 999, dt, dt)
    big = torch.full((3, 8, 1031), 50.0).to(TORCH[dt])
    big[:, 2:7, 5:1004] = l
    bigq = torch.full((3, 6, 1001), 1.0).to(TORCH[dt])
    bigq[:, 1:5, 1:1000] = pr
    got = q.verify(big.to(DEV)[:, 2:7, 5:1004], draft.to(DEV), u.to(DEV), draft_probs=bigq.to(DEV)[:, 1:5, 1:1000])
    want_t, want_a = want(l, draft, u, pr, None, None)
    assert torch.equal(got[0].cpu(), want_t) and torch.equal(got[1].cpu(), want_a)
    swapped = l.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)       # position-major
    swapped_q = pr.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    got = q.verify(swapped, draft.to(DEV), u.to(DEV), draft_probs=swapped_q)
    assert torch.equal(got[0].cpu(), want_t) and torch.equal(got[1].cpu(), want_a)
    one = l[:1].to(DEV).expand(3, -1, -1)                                  # one row block for all requests
    got = q.verify(one, draft.to(DEV), u.to(DEV))
    want_t, want_a = want(l[:1].expand(3, -1, -1), draft, u, None, None, None)
    assert torch.equal(got[0].cpu(), want_t) and torch.equal(got[1].cpu(), want_a)


def test_requests_do_not_depend_on_the_batch():
    l, draft, u, pr = (None if t is None else t.to(DEV) for t in problem(9, 5, 10007))
    temp = torch.linspace(0, 1.5, 9, device=DEV)
    t, n = q.verify(l, draft, u, draft_probs=pr, temperature=temp)
    for b in (0, 4, 8):
        s = slice(b, b + 1)
        t1, n1 = q.verify(l[s], draft[s], u[s], draft_probs=pr[s], temperature=temp[s])
        assert torch.equal(t1[0], t[b]) and n1[0] == n[b]


def test_many_requests():
    """More rows than one launch's grid takes."""
    l, draft, u, pr = problem(10000, 6, 5, seed=4)
    check(l, draft, u, pr)


@pytest.mark.parametrize("logits", ["bf16", "f32"])
def test_many_rows(logits):
    """Rows enough that a wave walks several spans and a workgroup several chunks; masks over whole spans; temperatures."""
    B, S, V = 48, 7, 40001
    l, draft, u, pr = problem(B, S, V, logits, "bf16", seed=6)
    l[0, :, 2000:12000] = -math.inf
    l[1, :, 100:] = -math.inf
    l[2, :, :39990] = torch.finfo(l.dtype).min
    l[3, 1, 77] = float("nan")
    l[4, :, 30000] = math.inf
    temp = torch.full((B,), 0.8)
    temp[5], temp[6], temp[7], temp[8], temp[9] = 0.0, 1e-6, 1e-25, 1e25, 3.0
    lens = (torch.arange(B) * 3 % (S + 1)).int()
    check(l, draft, u, pr, temp=temp)
    check(l, draft, u, None, temp=temp, lens=lens)


@pytest.mark.parametrize("V", [524289, 1200001])
@pytest.mark.parametrize("logits,probs", [("bf16", "f32"), ("f32", "bf16"), ("f32", None)])
def test_large_vocabularies(logits, probs, V):
    """More chunks than a workgroup has threads."""
    for seed in range(3):
        l, draft, u, pr = problem(2, 1, V, logits, probs, seed=seed)
        check(l, draft, u, pr, temp=torch.tensor([1.0, 0.6]))


@pytest.mark.parametrize("V", [500, 5000])
def test_drafter_that_agrees(V):
    """Where the drafter's probabilities are the target's, rounded to fp32, what is left of them is their rounding."""
    l, _, u, _ = problem(3, 2, V, seed=8)
    pr = torch.softmax(l[:, :2].double(), -1).float()
    check(l, torch.full((3, 2), V, dtype=torch.int32), u, pr)           # no such token: rejected
    one = pr.clone()
    one[..., 3] += 0.25                                                   # but for one value, which is below the target's elsewhere
    check(l, torch.full((3, 2), V, dtype=torch.int32), u, one)


def test_long_draft():
    check(*problem(2, 255, 40, seed=5, noise=0.01))


def test_distribution():
    """What is emitted first follows the target, whatever the drafter: 20000 draws over 6 tokens."""
    g = gen(11)
    n, V = 20000, 6
    l = torch.randn(1, 1, V, generator=g)
    p = torch.softmax(l[0, 0].double(), -1)
    qd = torch.softmax(torch.randn(V, generator=g), -1)
    draft = torch.multinomial(qd, n, replacement=True, generator=g).int().reshape(n, 1)
    t, _ = q.verify(l.expand(n, 2, V).contiguous().to(DEV), draft.to(DEV), torch.rand(n, 2, generator=g).to(DEV),
                    draft_probs=qd.expand(n, 1, V).contiguous().to(DEV))
    got = torch.bincount(t[:, 0].cpu().long(), minlength=V).double() / n
    assert ((got - p).abs() < 5 * (p * (1 - p) / n).sqrt()).all()      # five standard deviations


def test_empty_stream_and_graph():
    e = q.verify(torch.empty(0, 3, 10, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 3, device=DEV))
    assert e[0].shape == (0, 3) and e[1].shape == (0,)
    l, draft, u, pr = (t.to(DEV) for t in problem(3, 4, 9001))
    base = q.verify(l, draft, u, draft_probs=pr)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = q.verify(l, draft, u, draft_probs=pr, stream=side)
    side.synchronize()
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = q.verify(l, draft, u, draft_probs=pr)
    for i in range(4):
        u.copy_(torch.rand(3, 5, generator=gen(i)))
        out[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        again = q.verify(l, draft, u, draft_probs=pr)
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1]), i
