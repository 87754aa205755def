"""verify where its sums and choices come near a border: finite masks, very small
temperatures, large logits, equal probabilities, numbers that fall on a prefix sum."""
import numpy as np
import pytest
import torch

from ops_util import DEV, TORCH, gen
from test_gpu_verify import check

import bit_quantized_gemv_amd as q

pytestmark = pytest.mark.gpu

MASKS = [-1e4, -1e9, -1e10, -1e12, -1e15]


def masked(B, S, V, dt, value, added, seed):
    """Logits with finite masks over 95 of 100 values, whole lanes' values, whole spans and the end of the row, and a
    drafter that keeps to what is left."""
    g = gen(seed)
    l = 2 * torch.randn(B, S + 1, V, generator=g)
    l = torch.where(torch.rand(B, S + 1, V, generator=g) < min(0.5, 20 / V), l + 6, l)
    i = torch.arange(V)
    gone = torch.rand(B, S + 1, V, generator=g) < 0.95
    gone[0::4] = (i // 8 % 64 < 60) & (i % 97 != 5)
    gone[1::4, :, V // 8:3 * V // 4] = True
    gone[2::4, :, V - V // 3:] = True
    gone[3::4, :, 5] = False
    near = l[:, :S] + 0.5 * torch.randn(B, S, V, generator=g)
    l = torch.where(gone, l + value if added else torch.tensor(value), l)
    probs = torch.softmax(torch.where(gone[:, :S], torch.tensor(-torch.inf), near), -1)
    draft = torch.multinomial(probs.reshape(B * S, V), 1, generator=g).reshape(B, S).int()
    return l.to(TORCH[dt]), draft, torch.rand(B, S + 1, generator=g), probs


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("added", [False, True])
def test_finite_masks(dt, value, added):
    """A mask of finite values is a probability of zero as -inf is: nothing of it may reach the rest of the row."""
    B, S = 24, 3
    temp = torch.linspace(0.1, 1.5, B)
    temp[3], temp[7] = 1.0, 0.0
    l, draft, u, probs = masked(B, S, 7001, dt, value, added, seed=int(-np.log10(-value)) + added + 100)
    _, n = check(l, draft, u, probs, temp=temp)
    assert n.sum() > B // 4             # drafts are accepted at all
    check(l, draft, u, None, temp=temp)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-1e4, -1e10])
def test_finite_masks_of_many_rows(dt, value):
    """The same where a wave walks several spans of a row."""
    B = 128
    temp = torch.linspace(0.2, 1.5, B)
    temp[2] = 1.0
    l, draft, u, probs = masked(B, 1, 140001, dt, value, False, seed=9)
    check(l, draft, u, probs, temp=temp)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1e-4, 1e-6, 1e-7, 1e-8, 1e-9, 1e-10, 1e-12, 1e-15, 2e-18, 1e-18, 1e-30])
def test_small_temperatures(dt, T):
    """All that is left is the largest value, or several equal ones, each with its share."""
    B, S, V = 24, 3, 5000
    g = gen(3)
    l = 10 + 2 * torch.randn(B, S + 1, V, generator=g)
    top = 20 + 30 * torch.rand(B, S + 1, 1, generator=g)
    at = torch.randint(0, V, (B, S + 1, 3), generator=g)
    l.scatter_(2, at[..., :1], top)
    l[1::3] = l[1::3].scatter(2, at[1::3, :, :2], top[1::3].expand(-1, -1, 2))
    l[2::3] = l[2::3].scatter(2, at[2::3], top[2::3].expand(-1, -1, 3))
    draft, u = at[:, :S, 0].int().contiguous(), torch.rand(B, S + 1, generator=g)
    probs = torch.full((B, S, V), 0.25 / V)
    probs.scatter_(2, at[:, :S, :1], 0.75)
    l = l.to(TORCH[dt])
    temp = torch.full((B,), T)
    _, n = check(l, draft, u, None, temp=temp)
    assert (n[::3] == S).all()          # a token of probability 1 is accepted
    check(l, draft, u, probs, temp=temp)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e6, 1e10, 1e14, 1e17])
def test_large_logits(dt, scale):
    B, S, V = 12, 2, 5000
    g = gen(4)
    l = scale * (1 + torch.rand(B, S + 1, V, generator=g)) * torch.where(torch.arange(B) % 2 == 0, 1.0, -1.0).reshape(B, 1, 1)
    l = l.to(TORCH[dt])
    draft = l[:, :S].float().argmax(-1).int()
    check(l, draft, torch.rand(B, S + 1, generator=g), None, temp=torch.linspace(0.3, 3.0, B))
    check(l, draft, torch.rand(B, S + 1, generator=g), None, temp=torch.linspace(0.3, 3.0, B) * scale)


@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_numbers_next_to_a_probability(side, dt):
    """A token is accepted while u < p: u is p in fp32, off by 2^-30 of it at most, above or below, at every position."""
    B, S, V, n, N = 64, 5, 4096, 20, 1 << 18
    live = (2 * torch.randn(N, n, generator=gen(8))).to(TORCH[dt])
    e = torch.exp(live.double())
    p = e / e.sum(1, keepdim=True)
    at = p.argmax(1, keepdim=True)
    off = ((p.gather(1, at).float().double() / p.gather(1, at) - 1) * side).squeeze(1)
    rows = torch.nonzero((off > 2.0 ** -40) & (off < 2.0 ** -30)).squeeze(1)[:B * S]
    assert len(rows) == B * S
    l = torch.full((B, S + 1, V), -torch.inf, dtype=TORCH[dt])
    l[:, :S, :200 * n:200] = live[rows].reshape(B, S, n)
    l[:, S, 0] = 0.0
    draft = (200 * at[rows]).reshape(B, S).int()
    u = torch.cat([p[rows].gather(1, at[rows]).float().reshape(B, S), torch.full((B, 1), 0.5)], 1)
    _, k = check(l, draft, u, None)
    assert (k == (0 if side > 0 else S)).all()
    u[:, 0] = 0.0                                     # the first of them later
    u[::2, 1] = 0.0
    check(l, draft, u, None)


@pytest.mark.parametrize("side", [1, -1])
def test_zero_takes_the_first_value_left(side):
    """u = 0 gives the lowest index of a positive weight, however small.  The first 2048 values have one that is not
    masked, and the drafter's probability of it, in fp32, is the target's but for 2^-30 of it, above or below."""
    B, V, n = 256, 4096, 20
    live = 2 * torch.randn(1 << 17, n, generator=gen(5))
    e = torch.exp(torch.cat([torch.full((1 << 17, 1), -12.0), live], 1).double())
    p = e / e.sum(1, keepdim=True)
    off = (p[:, 0].float().double() / p[:, 0] - 1) * side
    rows = torch.nonzero((off > 2.0 ** -40) & (off < 2.0 ** -30)).squeeze(1)[:B]
    assert len(rows) == B
    l = torch.full((B, 2, V), -torch.inf)
    l[..., 7], l[..., 2048:2048 + n] = -12.0, live[rows].unsqueeze(1)
    probs = torch.zeros(B, 1, V)
    probs[:, 0, 7], probs[:, 0, 2048:2048 + n] = p[rows, 0].float(), 0.5 * p[rows, 1:].float()
    t, _ = check(l, torch.full((B, 1), V, dtype=torch.int32), torch.zeros(B, 2), probs)        # no such token: rejected
    assert (t[:, 0] == (2048 if side > 0 else 7)).all()


def test_a_number_on_the_border_of_two_halves():
    """Two equal halves and u = 1/2: the last value of the first or, as in exact arithmetic, the first of the second."""
    B = 300
    h = 2 * torch.randn(B, 1, 4096, generator=gen(6))
    h[..., :8] = -torch.inf
    t, _ = q.verify(torch.cat([h, h], -1).to(DEV), torch.zeros(B, 0, dtype=torch.int32, device=DEV), torch.full((B, 1), 0.5, device=DEV))
    assert set(t[:, 0].tolist()) <= {4095, 4104}


@pytest.mark.parametrize("first", [1, 8, 600, 5000])
def test_numbers_below_zero_take_the_first_value(first):
    l = torch.randn(4, 1, 9000, generator=gen(7))
    l[..., :first] = -torch.inf
    t, _ = q.verify(l.to(DEV), torch.zeros(4, 0, dtype=torch.int32, device=DEV), torch.full((4, 1), -0.5, device=DEV))
    assert t[:, 0].tolist() == [first] * 4


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_signalling_nan(dt):
    """NaNs of every bit pattern have probability 0 and hide nothing beside them."""
    l, draft, u, probs = masked(16, 2, 5001, dt, -1e4, False, seed=77)
    bits = l.view(torch.int16 if dt == "bf16" else torch.int32)
    patterns = [0x7f81, -127, 0x7fff, 0x7fc0] if dt == "bf16" else [0x7f800001, -(0x7fffff - 1), 0x7fffffff, 0x7fc00000]
    for k, pattern in enumerate(patterns):
        bits[k::4, :, k::7] = pattern
    assert l.isnan().float().mean() > 0.1
    check(l, draft, u, probs, temp=torch.linspace(0.0, 1.5, 16))
    check(l, draft, u, None)
