"""Helpers of the tests of the operators beside qmv: seeded inputs and plain
64-bit forms of their definitions, on the CPU."""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda:0"
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# Normwise bar of an fp32 output row, the library's: max |y - ref| <= TOL * max |ref|.
TOL = 2e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def matrix(g, lead, K, bits, gs, sb):
    w = torch.randint(-2 ** 31, 2 ** 31, (*lead, K * bits // 32), generator=g).to(torch.int32)
    top = 2 ** bits - 1
    s = (0.5 + torch.rand(*lead, K // gs, generator=g)) / (top * 0.3 * K ** 0.5)
    b = -s * (0.5 * top + 0.3 * torch.randn(*lead, K // gs, generator=g))
    return w, s.to(TORCH[sb]), b.to(TORCH[sb])


def dequantize(w, s, b, bits, gs):
    """scale * code + bias in 64 bits."""
    u = w.numpy().view(np.uint32)
    codes = np.stack([(u >> (bits * j)) & (2 ** bits - 1) for j in range(32 // bits)], -1)
    codes = torch.from_numpy(codes.reshape(*s.shape, gs).astype(np.float64))
    return (codes * s.double().unsqueeze(-1) + b.double().unsqueeze(-1)).reshape(*w.shape[:-1], -1)


def check_rows(got, want, what, dtype, tol=TOL):
    """Every row of `got` against the 64-bit `want`: fp32 within tol of the row's
    largest value; bf16 also off by its rounding, half a step (2^-8 of the value)."""
    g = got.detach().cpu().double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    if g.numel() == 0:
        return
    lim = tol * want.abs().amax(-1, keepdim=True).expand_as(want)
    if dtype == "bf16":
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    over = (g - want).abs() > lim
    worst = float(((g - want).abs() / want.abs().amax(-1, keepdim=True).clamp(min=1e-300)).max())
    assert not over.any(), f"{what}: {int(over.sum())} values off, worst {worst:.3e} of the row's largest"
