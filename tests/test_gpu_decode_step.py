"""The operators together, as a serving program calls them (examples/decode_step.py),
against the same step in 64 bits on the CPU."""
import os
import sys

import pytest
import torch

from ops_util import DEV, dequantize

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import decode_step  # noqa: E402

pytestmark = pytest.mark.gpu


def logits64(m, tokens, adapters):
    """The model's logits with the operators' results in 64 bits; what the model holds in bf16 is rounded as it is there."""
    cpu = lambda t: t.cpu()
    x = cpu(m.embed)[tokens.cpu().long()].double()
    mats = [dequantize(*map(cpu, w), 4, 64) for w in (m.proj, m.gate_up, m.down, m.head)]
    h = x @ mats[0].T
    for i, a in enumerate(adapters.tolist()):
        if a >= 0:
            h[i] += m.scaling[a].item() * (cpu(m.lora_b)[a].double() @ (cpu(m.lora_a)[a].double() @ x[i]))
    h = h.bfloat16().double()
    r = h @ cpu(m.router).double().T
    y = torch.zeros_like(h)
    F = m.down[0].shape[-1] * 8
    for i in range(len(h)):
        top = torch.topk(r[i], m.k)
        for w, e in zip(torch.softmax(top.values, -1), top.indices.tolist()):
            gu = mats[1][e] @ h[i]
            y[i] += w * (mats[2][e] @ (gu[:F] * torch.sigmoid(gu[:F]) * gu[F:]))
    h = (h.bfloat16() + y.bfloat16()).double()
    return h @ mats[3].T


def test_logits():
    m = decode_step.Model()
    g = torch.Generator().manual_seed(3)
    tokens = torch.randint(0, m.V, (24,), generator=g).int()
    adapters = (torch.arange(24) % 7 - 1).int()
    got = m.logits(tokens.to(DEV), adapters.to(DEV)).cpu().double()
    want = logits64(m, tokens, adapters)
    # the two bf16 roundings of the hidden state may fall either way: one step, 2^-8, of each of its values
    off = (got - want).norm(dim=-1) / want.norm(dim=-1)
    assert (off < 2 * 2.0 ** -8).all(), off


def test_step_follows_its_logits():
    """Greedy requests accept the drafted tokens that are the largest logit, and get that of the first that is not."""
    m = decode_step.Model(seed=2)
    B, S = 4, 3
    g = torch.Generator().manual_seed(4)
    last = torch.randint(0, m.V, (B,), generator=g).int().to(DEV)
    adapters = torch.tensor([-1, 0, 5, 5], dtype=torch.int32, device=DEV)
    draft = torch.randint(0, m.V, (B, S), generator=g).int().to(DEV)
    for j in range(S):          # requests 1.. are drafted right up to position b - 1
        tokens = torch.cat([last.unsqueeze(1), draft], 1)
        best = m.logits(tokens.reshape(-1), adapters.repeat_interleave(S + 1)).reshape(B, S + 1, -1).argmax(-1).int()
        for b in range(B):
            if j < b:
                draft[b, j] = best[b, j]
    tokens, accepted = decode_step.step(m, last, draft, adapters, torch.rand(B, S + 1, device=DEV), temperature=torch.zeros(B, device=DEV))
    seq = torch.cat([last.unsqueeze(1), draft], 1)
    best = m.logits(seq.reshape(-1), adapters.repeat_interleave(S + 1)).reshape(B, S + 1, -1).argmax(-1).int()
    assert accepted.tolist() == [0, 1, 2, 3]
    for b in range(B):
        n = accepted[b]
        assert torch.equal(tokens[b, :n], draft[b, :n]) and tokens[b, n] == best[b, n] and (tokens[b, n + 1:] == -1).all()


def test_the_example_runs(capsys):
    decode_step.main()
    assert capsys.readouterr().out.count("accepted") == 4
