"""One verify step of a speculative decoder on random weights, with the
library's operators as a serving program calls them:

  affine_lora  a projection shared by all requests, each with its own adapter
  moe          the layer's experts, on the projection's outputs
  affine       the head: logits of every drafted position and the one after
  verify       the drafted tokens accepted or replaced

Run on an MI355X: python examples/decode_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_gemv_amd as q  # noqa: E402


def quantized(g, *lead, K, bits=4, gs=64):
    """Random packed codes, scales and biases of a matrix (or a stack of them) of K columns and about unit gain."""
    dev = g.device
    w = torch.randint(-2 ** 31, 2 ** 31 - 1, (*lead, K * bits // 32), generator=g, device=dev, dtype=torch.int32)
    top = 2 ** bits - 1
    s = (0.5 + torch.rand(*lead, K // gs, generator=g, device=dev)) / (0.3 * top * K ** 0.5)
    return w, s.bfloat16(), (-0.5 * top * s).bfloat16()


class Model:
    """A toy layer and head: D wide, E experts of which k are chosen, V tokens, L adapters of rank R."""

    def __init__(self, D=512, F=256, E=16, k=4, V=4096, L=6, R=16, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        half = lambda *s: torch.randn(*s, generator=g, device=device).bfloat16()
        self.k, self.V = k, V
        self.embed = half(V, D)
        self.proj = quantized(g, D, K=D)
        self.lora_a, self.lora_b = half(L, R, D) / D ** 0.5, half(L, D, R) * (0.3 / R ** 0.5)
        self.scaling = torch.linspace(0.5, 2.0, L, device=device)
        self.router = half(E, D) / D ** 0.5
        self.gate_up, self.down = quantized(g, E, 2 * F, K=D), quantized(g, E, D, K=F)
        self.head = quantized(g, V, K=D)

    def logits(self, tokens, adapters):
        """tokens, adapters: [n]; logits fp32 [n][V]."""
        x = self.embed[tokens]
        h = q.affine_lora(*self.proj, x, self.lora_a, self.lora_b, adapters, scaling=self.scaling, bits=4, group_size=64)
        h = h + q.moe(h, self.router, self.gate_up, self.down, top_k=self.k, bits=4, group_size=64)
        return q.affine(*self.head, h, bits=4, group_size=64, out_dtype=torch.float32)


def step(model, last, draft, adapters, uniforms, draft_probs=None, temperature=None):
    """last [B]: each request's newest token; draft [B][S]; adapters [B] (-1: none); uniforms [B][S + 1].
    Returns (tokens [B][S + 1], accepted [B]) of `verify`."""
    B, S = draft.shape
    tokens = torch.cat([last.unsqueeze(1), draft], 1)
    logits = model.logits(tokens.reshape(-1), adapters.repeat_interleave(S + 1).contiguous())
    return q.verify(logits.reshape(B, S + 1, model.V), draft, uniforms, draft_probs=draft_probs, temperature=temperature)


def main():
    dev = "cuda"
    model, B, S = Model(device=dev), 5, 3
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    last = torch.randint(0, model.V, (B,), generator=g, device=dev, dtype=torch.int32)
    adapters = torch.tensor([0, 3, -1, 3, 5], dtype=torch.int32, device=dev)
    temperature = torch.tensor([1.0, 0.7, 1.0, 0.0, 1.3], device=dev)
    for i in range(4):
        # a drafter that is right about the first token it gives, and guesses the others
        first = model.logits(last, adapters).argmax(-1).int()
        guess = torch.randint(0, model.V, (B, S - 1), generator=g, device=dev, dtype=torch.int32)
        draft = torch.cat([first.unsqueeze(1), guess], 1)
        tokens, accepted = step(model, last, draft, adapters, torch.rand(B, S + 1, generator=g, device=dev), temperature=temperature)
        last = tokens.gather(1, accepted.long().unsqueeze(1)).squeeze(1)
        print(f"step {i}: accepted {accepted.tolist()}, next tokens {last.tolist()}")


if __name__ == "__main__":
    main()
