"""The attention of a quantized decoder layer on random weights, with the
library's operators as a serving program calls them:

  affine  the projection to queries, keys and values, and the one back
  append  norms and rotation of queries and keys, keys and values to the cache's pages
  attend  attention over the pages

Prompts enter the cache in chunks, beside sequences that decode or verify drafted tokens.

Run on an MI355X: python examples/attention_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_gemv_amd as q  # noqa: E402
from examples.decode_step import quantized  # noqa: E402


class Pool:
    """Pages of keys and values, handed out to sequences as they grow."""

    def __init__(self, pages, page_size, heads, D, most, device):
        self.k, self.v = (torch.zeros(pages, page_size, heads, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.free, self.page_size, self.most, self.device = list(range(pages)), page_size, most, device
        self.tables, self.lengths = {}, {}

    def grow(self, name, tokens):
        """Room for that many more tokens of a sequence."""
        table = self.tables.setdefault(name, [])
        self.lengths[name] = self.lengths.get(name, 0) + tokens
        while len(table) * self.page_size < self.lengths[name]:
            table.append(self.free.pop())

    def shrink(self, name, tokens):
        """The last tokens of a sequence (drafted ones that were rejected) leave it."""
        self.lengths[name] -= tokens

    def batch(self, names, new):
        """pages, starts, lengths of a call: these sequences with so many new tokens each."""
        pages = torch.zeros(len(names), self.most, dtype=torch.int32)
        for i, n in enumerate(names):
            pages[i, :len(self.tables[n])] = torch.tensor(self.tables[n], dtype=torch.int32)
        starts = torch.tensor([0] + list(new)).cumsum(0).int()
        lengths = torch.tensor([self.lengths[n] for n in names], dtype=torch.int32)
        return pages.to(self.device), starts.to(self.device), lengths.to(self.device)


class Attention:
    """width values a token, Hq query heads on Hkv heads of D; a window of the newest places and some first ones, if given."""

    def __init__(self, width=512, Hq=8, Hkv=2, D=64, window=0, sinks=0, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.heads, self.window, self.sinks = (Hq, Hkv, D), window, sinks
        self.qkv, self.back = quantized(g, (Hq + 2 * Hkv) * D, K=width), quantized(g, width, K=Hq * D)
        self.q_weight, self.k_weight = ((1 + 0.1 * torch.randn(D, generator=g, device=device)).bfloat16() for _ in range(2))
        self.freqs = 10000.0 ** (-torch.arange(D // 2, device=device) / (D // 2))

    def project(self, x):
        """Queries, keys and values of tokens x [T][width], views of one product."""
        Hq, Hkv, D = self.heads
        y = q.affine(*self.qkv, x, bits=4, group_size=64)
        return [part.unflatten(1, (-1, D)) for part in y.split((Hq * D, Hkv * D, Hkv * D), 1)]

    def __call__(self, x, pool, pages, starts, lengths, max_new, max_length):
        qs, ks, vs = self.project(x)
        qs = q.append(qs, ks, vs, self.freqs, pool.k, pool.v, pages, starts, lengths, q_weight=self.q_weight, k_weight=self.k_weight)
        o = q.attend(qs, pool.k, pool.v, pages, starts, lengths, window=self.window, sinks=self.sinks, max_new=max_new, max_length=max_length)
        return x + q.affine(*self.back, o.flatten(1), bits=4, group_size=64)


def step(layer, pool, names, xs):
    """New tokens xs[i] [n][width] of sequences: their outputs."""
    new = [x.shape[0] for x in xs]
    for n, count in zip(names, new):
        pool.grow(n, count)
    y = layer(torch.cat(xs), pool, *pool.batch(names, new), max(new), max(pool.lengths[n] for n in names))
    return list(y.split(new))


def main():
    dev = "cuda"
    layer, pool = Attention(window=96, sinks=4, device=dev), Pool(64, 16, 2, 64, 32, dev)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    tokens = lambda n: torch.randn(n, 512, generator=g, device=dev).bfloat16()
    step(layer, pool, ["a"], [tokens(150)])                                       # a prompt
    step(layer, pool, ["a", "b"], [tokens(1), tokens(64)])                        # a token, and a chunk of the next prompt
    step(layer, pool, ["a", "b"], [tokens(5), tokens(30)])                        # drafted tokens, and the rest of it
    pool.shrink("a", 2)                                                           # two of them were rejected
    for i in range(3):
        a, b = step(layer, pool, ["a", "b"], [tokens(1), tokens(5)])
        pool.shrink("b", 4 - i)
        print(f"step {i}: lengths {pool.lengths}, norms {a.float().norm():.3f} {b.float().norm():.3f}")


if __name__ == "__main__":
    main()
