"""A small decoder that answers with low-bit weights and an 8-bit or 4-bit key-value cache.

The layers' products are the library's low-bit linears, what stands between them its
decoder operators: kv_append (norms of the heads, rotation, cache write), attention, sample.  A batch of
prompts of different lengths goes through in one ragged call; each further token is
one replay of a captured CUDA graph, in which the lengths and the sampled tokens stay on
the device.  Weights are random: the point is the calls, not the text.

    python examples/decode.py [--layers 4] [--batch 4] [--steps 64] [--cache-bits 8] [--head-norms]
"""
from __future__ import annotations

import argparse
import sys
import time
from pathlib import Path

import torch
from torch.nn import functional as F

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import bit_groupwise_weight_gb300 as lb  # noqa: E402


class Layer(torch.nn.Module):
    def __init__(self, width, heads, kv_heads, dim, hidden, bits, group, pages, page, cache_bits=8, head_norms=False):
        super().__init__()
        def linear(n, k):
            return torch.nn.Linear(k, n, bias=False, device="cuda", dtype=torch.bfloat16)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.norm1, self.norm2 = (torch.ones(width, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.qkv = lb.LowbitLinear.from_linear(linear((heads + 2 * kv_heads) * dim, width), bits, group)
        self.o = lb.LowbitLinear.from_linear(linear(width, heads * dim), bits, group)
        self.gate_up = lb.LowbitGateUp.from_linears(linear(hidden, width), linear(hidden, width), bits, group)
        self.down = lb.LowbitLinear.from_linear(linear(width, hidden), bits, group)
        self.cache = lb.empty_cache(pages, kv_heads, dim, page, bits=cache_bits)
        self.q_norm = self.k_norm = torch.ones(dim, device="cuda", dtype=torch.bfloat16) if head_norms else None

    def forward(self, x, table, lens, cu_q, max_q, turns):
        qkv = self.qkv(F.rms_norm(x, x.shape[-1:], self.norm1)).view(-1, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = lb.kv_append(q, k, v, *self.cache, table, lens, cu_q, max_q, turns=turns, q_norm=self.q_norm, k_norm=self.k_norm)
        x = x + self.o(lb.attention(q, *self.cache, table, lens, cu_q, max_q).flatten(1))
        return x + self.down(self.gate_up(F.rms_norm(x, x.shape[-1:], self.norm2)))


class Decoder(torch.nn.Module):
    """`batch` sequences of up to `length` tokens, each with pages of its own."""

    def __init__(self, layers=4, width=1024, heads=16, kv_heads=4, dim=64, hidden=2816, vocab=32000, bits=4, group=64, batch=4,
                 length=1024, page=64, seed=0, cache_bits=8, head_norms=False):
        super().__init__()
        torch.manual_seed(seed)
        per = -(-length // page)
        self.table = torch.randperm(batch * per, device="cuda").to(torch.int32).view(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.last = torch.zeros(batch, dtype=torch.int64, device="cuda")
        self.turns = lb.rotary_turns(dim, base=500000.0, device="cuda")
        self.embed = torch.randn(vocab, width, device="cuda").to(torch.bfloat16)
        self.norm = torch.ones(width, device="cuda", dtype=torch.bfloat16)
        self.layers = torch.nn.ModuleList(Layer(width, heads, kv_heads, dim, hidden, bits, group, batch * per, page,
                                                cache_bits, head_norms)
                                          for _ in range(layers))
        self.head = lb.LowbitLinear.from_linear(
            torch.nn.Linear(width, vocab, bias=False, device="cuda", dtype=torch.bfloat16), bits, group)

    def logits(self, tokens, lens, cu_q=None, max_q=None, last=None):
        """Logits of the tokens at rows `last` (None: all) after all have gone through."""
        x = self.embed[tokens]
        for layer in self.layers:
            x = layer(x, self.table, lens, cu_q, max_q, self.turns)
        return self.head(F.rms_norm(x if last is None else x[last], x.shape[-1:], self.norm))

    @torch.no_grad()
    def prompt(self, prompts, u, **settings):
        """Prompts (lists of token numbers) in; each one's first new token out."""
        counts = [len(p) for p in prompts]
        cu_q = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
        self.lens.copy_(torch.tensor(counts, dtype=torch.int32))
        tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
        logits = self.logits(tokens, self.lens, cu_q, max(counts), cu_q[1:].long() - 1)
        lb.sample(logits, u, out=self.last, **settings)
        return self.last.clone()

    @torch.no_grad()
    def step(self, u, **settings):
        """One more token of every sequence, all on the device."""
        self.lens += 1
        lb.sample(self.logits(self.last, self.lens), u, out=self.last, **settings)

    def capture(self, u, **settings):
        """`step` as a graph; u is read at each replay.  The state is left as it was."""
        lens, last = self.lens.clone(), self.last.clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.step(u, **settings)                       # loads the kernels; its token is written again later
        torch.cuda.current_stream().wait_stream(stream)
        self.lens.copy_(lens), self.last.copy_(last)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(u, **settings)
        return graph


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--layers", type=int, default=4)
    a.add_argument("--batch", type=int, default=4)
    a.add_argument("--steps", type=int, default=64)
    a.add_argument("--cache-bits", type=int, default=8, choices=(4, 8))
    a.add_argument("--head-norms", action="store_true")
    a = a.parse_args()
    settings = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    model = Decoder(layers=a.layers, batch=a.batch, cache_bits=a.cache_bits, head_norms=a.head_norms)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompts = [[(37 * i + 11 * b) % 32000 for i in range(5 + 40 * b % 700)] for b in range(a.batch)]
    u = torch.rand(a.batch, generator=gen, device="cuda")
    answers = [model.prompt(prompts, u, **settings)]
    graph = model.capture(u, **settings)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        u.copy_(torch.rand(a.batch, generator=gen, device="cuda"))
        graph.replay()
        answers.append(model.last.clone())
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    for b, line in enumerate(torch.stack(answers, 1).tolist()):
        print(f"prompt of {len(prompts[b])} tokens ->", *line[:12], "...")
    print(f"{a.steps} steps of {a.batch} sequences: {took / a.steps * 1e6:.0f} us a step, {a.steps * a.batch / took:.0f} tokens/s")


if __name__ == "__main__":
    main()
