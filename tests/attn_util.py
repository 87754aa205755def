"""Helpers of the tests of norms, rotation and attention over a cache in pages:
seeded inputs, and plain 64-bit forms of the definitions, on the CPU."""
from __future__ import annotations

import math

import torch

from ops_util import DEV, TORCH, gen  # noqa: F401

# half a step of rounding, relative to the value
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


class Batch:
    """Sequences of `new` new tokens and `lengths` places over a pool of pages in random order; slots that hold nothing are NaN."""

    def __init__(self, new, lengths, H, D, P, dt="bf16", seed=0, spare=2, wide=0, order="page", fill=math.nan):
        g = gen(seed)
        self.new, self.lengths, self.H, self.D, self.P, self.dt = list(new), list(lengths), H, D, P, dt
        counts = [-(-max(n, 0) // P) for n in lengths]
        total, most = sum(counts) + spare, max(counts + [1]) + wide
        perm = torch.randperm(total, generator=g).int()
        self.pages = torch.full((len(new), most), -1, dtype=torch.int32)
        kv = torch.full((2, total, P, H, D), fill)
        at = 0
        for b, (c, n) in enumerate(zip(counts, lengths)):
            self.pages[b, :c] = perm[at:at + c]
            for i in range(c):
                m = min(P, n - i * P)
                kv[:, perm[at + i].long(), :m] = torch.randn(2, m, H, D, generator=g)
            at += c
        kv = kv.to(TORCH[dt])
        if order == "head":         # [page][head][slot][D]
            kv = kv.transpose(2, 3).contiguous().transpose(2, 3)
        elif order == "one":        # keys and values of a page side by side
            kv = kv.transpose(0, 1).contiguous().transpose(0, 1)
        self.k, self.v = kv[0], kv[1]
        self.starts = torch.tensor([0] + list(new)).cumsum(0).int()
        self.lens = torch.tensor(lengths, dtype=torch.int32)
        self.T = int(self.starts[-1])

    def on(self, dev=DEV):
        """k, v, pages, starts, lengths on the device, strides kept."""
        put = lambda t: torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device=dev).copy_(t)
        if self.k.untyped_storage().data_ptr() == self.v.untyped_storage().data_ptr() and self.k.stride(0) == 2 * self.P * self.H * self.D:
            both = torch.empty(self.k.shape[0], 2, *self.k.shape[1:], dtype=self.k.dtype, device=dev)
            both[:, 0], both[:, 1] = self.k.to(dev), self.v.to(dev)
            return both[:, 0], both[:, 1], self.pages.to(dev), self.starts.to(dev), self.lens.to(dev)
        return put(self.k), put(self.v), self.pages.to(dev), self.starts.to(dev), self.lens.to(dev)

    def row(self, b, j):
        """(page, slot) of place j, or None."""
        if j < 0 or j >= self.pages.shape[1] * self.P:
            return None
        p = int(self.pages[b, j // self.P])
        return (p, j % self.P) if 0 <= p < self.k.shape[0] else None


def attend64(q, c: Batch, window=0, sinks=0, scale=None):
    """(out, reach): the definition in 64 bits, and sum of weight * |v|, which roundings of the weights go with."""
    T, Hq, D = q.shape
    G = Hq // c.H
    scale = D ** -0.5 if scale is None else scale
    out, reach = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for b, (n, length) in enumerate(zip(c.new, c.lengths)):
        length = min(length, c.pages.shape[1] * c.P)
        rows = [c.row(b, j) for j in range(length)]
        held = torch.tensor([r is not None for r in rows], dtype=torch.bool)
        pages = torch.tensor([r[0] if r else 0 for r in rows], dtype=torch.long)
        slots = torch.tensor([r[1] if r else 0 for r in rows], dtype=torch.long)
        k, v = c.k[pages, slots].double(), c.v[pages, slots].double()     # [length][H][D]
        j = torch.arange(length)
        for i in range(n):
            p = length - n + i
            sees = held & (j <= p)
            if window:
                sees &= (j > p - window) | (j < sinks)
            t = int(c.starts[b]) + i
            if not sees.any():
                continue
            for h in range(Hq):
                s = (k[sees, h // G] @ q[t, h].double()) * scale
                w = torch.softmax(s, 0)
                out[t, h] = w @ v[sees, h // G]
                reach[t, h] = w @ v[sees, h // G].abs()
    return out, reach


def check_attend(got, want, reach, dt, out, what=""):
    """fp32 sums: 2e-5 of a row's largest value (the library's bar). The weights are rounded to the cache's type, half a step of each
    (in two pieces for fp32 outputs: half a step of half a step, twice where the second piece is cut off), and the result once to bf16."""
    g = got.detach().cpu().double()
    assert g.shape == want.shape and torch.isfinite(g).all(), what
    weights = HALF[dt] if out == "bf16" else 2 * HALF[dt] ** 2
    lim = 2e-5 * reach.amax(-1, keepdim=True) + weights * reach
    if out == "bf16":
        lim = lim * (1 + HALF["bf16"]) + HALF["bf16"] * want.abs()
    over = (g - want).abs() - lim
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} off, worst {float(((g - want).abs() / lim.clamp(min=1e-300)).max()):.2f} of the bound"


def rotate64(x, weight, eps, angles, interleaved):
    """Norm and rotation of x [T][H][D] in 64 bits; angles [T][R / 2]. Also the size that fp32 roundings go with."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    half = angles.shape[-1]
    out, size = x.clone(), x.abs()
    for i in range(half):
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = torch.cos(angles[:, i]).unsqueeze(1), torch.sin(angles[:, i]).unsqueeze(1)
        a, b = x[..., u], x[..., w]
        out[..., u], out[..., w] = a * c - b * s, b * c + a * s
        size[..., u] = size[..., w] = a.abs() + b.abs()
    return out, size


def check_rounded(got, want, size, kind, what=""):
    """A result computed in fp32 by about 16 roundings (2^-20 of its terms) and rounded once (below the normal numbers: half a step of those)."""
    g = got.detach().cpu().double()
    assert g.shape == want.shape and torch.isfinite(g).all(), what
    lim = 2.0 ** -20 * size * (1 + HALF[kind]) + HALF[kind] * want.abs() + torch.finfo(TORCH[kind]).smallest_normal * HALF[kind]
    over = (g - want).abs() - lim
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} off, worst {float(((g - want).abs() / lim.clamp(min=1e-300)).max()):.2f} of the bound"
