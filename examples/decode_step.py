"""One decode step of several requests: the products and the operators around them.

    python examples/decode_step.py [--requests 8] [--length 300] [--steps 4]

A skeleton of a decode layer and lm_head in synthetic weights, without norms and
position encoding (the model's own business): every step

  q | k | v   = one merged Q4NX projection, each request with its own adapter   q4nx_gemm_lora
  k, v        go into the requests' 4-bit paged caches                          q4nx_kv_append
  q           attends to them                                                   q4nx_kv_attention
  o           = a Q4NX projection of the heads, with adapters as well           q4nx_gemm_lora
  logits      = a Q8 lm_head                                                    q4nx_gemm_m64
  tokens      = the most likely ones, with their log-probabilities              q4nx_logprobs

The page table hands out pages as the requests grow; nothing waits for the
GPU between the calls of a step.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dequant_gemv_gb300 as q4  # noqa: E402
import synth  # noqa: E402


@dataclass
class Sizes:
    hidden: int = 1024
    heads: int = 16
    kv_heads: int = 8
    head_dim: int = 128
    vocab: int = 4096
    page_tokens: int = 64
    rank: int = 16
    adapters: int = 3


class Model:
    """Weights of the step: Q4NX projections, an lm_head, the adapters of two projections, the token embeddings."""

    def __init__(self, s: Sizes, device="cuda", seed: int = 0):
        self.s, self.device = s, torch.device(device)
        g = torch.Generator(device=device).manual_seed(seed)
        qkv, heads = (s.heads + 2 * s.kv_heads) * s.head_dim, s.heads * s.head_dim

        def weight(kind, rows, cols, n):
            _, w = synth.make(kind, rows, cols, synth.rng(90, n, rows + cols + seed))
            return q4.Weight(torch.from_numpy(w).to(device), kind, rows, cols)

        def adapters(rows, cols):
            n = lambda *shape: torch.randn(*shape, generator=g, device=device)  # noqa: E731
            return q4.Adapters((n(s.adapters, s.rank, cols) * cols ** -0.5).bfloat16(), (n(s.adapters, rows, s.rank) * 0.05).bfloat16(),
                               torch.ones(s.adapters, device=device))

        self.qkv, self.o = weight(synth.Q4_1, qkv, s.hidden, 1), weight(synth.Q4_1, s.hidden, heads, 2)
        self.lm_head = weight(synth.Q8_BLK, s.vocab, s.hidden, 3)
        self.qkv_adapters, self.o_adapters = adapters(qkv, s.hidden), adapters(s.hidden, heads)
        self.embedding = torch.randn(s.vocab, s.hidden, generator=g, device=device).bfloat16()


class Requests:
    """Several requests' caches: how many tokens each holds, and the pages handed to it."""

    def __init__(self, model: Model, count: int, most_tokens: int, adapter_ids):
        s, dev = model.s, model.device
        self.model, self.count = model, count
        cols = -(-most_tokens // s.page_tokens)
        self.cache = q4.KVCache.alloc(count * cols, s.kv_heads, s.head_dim, s.page_tokens, dev)
        # pages in an order of their own, as a server's free list would give them
        self.table = torch.from_numpy(np.random.default_rng(7).permutation(count * cols).astype(np.int32).reshape(count, cols)).to(dev)
        self.lens = torch.zeros(count, dtype=torch.int32, device=dev)
        self.q_start = torch.arange(count + 1, dtype=torch.int32, device=dev)
        self.adapter_ids = torch.tensor(adapter_ids, dtype=torch.int32, device=dev)

    def prompt(self, lengths):
        """Fill the caches with prompts' keys and values (synthetic ones: a prefill's output)."""
        s, dev = self.model.s, self.model.device
        start = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        self.lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
        g = torch.Generator(device=dev).manual_seed(11)
        k, v = (torch.randn(sum(lengths), s.kv_heads, s.head_dim, generator=g, device=dev).bfloat16() for _ in range(2))
        q4.q4nx_kv_append(self.cache, k, v, start, self.lens, self.table)
        return k, v

    def step(self, tokens: torch.Tensor, top: int = 5) -> dict:
        """One new token per request (int32 or int64 [count]) through the model; the next tokens and their log-probabilities."""
        m, s = self.model, self.model.s
        x = m.embedding[tokens.long()]
        qkv = q4.q4nx_gemm_lora(m.qkv, x, m.qkv_adapters, self.adapter_ids)
        qkv = qkv.unflatten(1, (-1, s.head_dim))                       # views: the operators take strided rows
        q, k, v = qkv[:, :s.heads], qkv[:, s.heads:s.heads + s.kv_heads], qkv[:, s.heads + s.kv_heads:]
        self.lens += 1
        q4.q4nx_kv_append(self.cache, k, v, self.q_start, self.lens, self.table)
        a = q4.q4nx_kv_attention(self.cache, q, self.q_start, self.lens, self.table)
        h = x + q4.q4nx_gemm_lora(m.o, a.flatten(1), m.o_adapters, self.adapter_ids)
        logits = q4.q4nx_gemm_m64(m.lm_head, h, out_dtype="f32")
        likely = q4.q4nx_logprobs(logits, top=top)
        chosen = likely.top_idx[:, 0].contiguous()
        return dict(x=x, qkv=qkv, attention=a, hidden=h, logits=logits, tokens=chosen, logprobs=likely)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--length", type=int, default=300)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    if not 1 <= a.requests <= 64:
        ap.error("the products take 1..64 tokens a call")
    model = Model(Sizes())
    lengths = [max(1, a.length * (b + 1) // a.requests) for b in range(a.requests)]
    reqs = Requests(model, a.requests, a.length + a.steps, [b % (model.s.adapters + 1) - 1 for b in range(a.requests)])
    reqs.prompt(lengths)
    tokens = torch.arange(a.requests, device=model.device)
    for n in range(a.steps):
        out = reqs.step(tokens)
        tokens = out["tokens"]
        lp = out["logprobs"]
        print(f"step {n}: tokens {tokens.tolist()}, log-probabilities {[round(v, 3) for v in lp.top_logprob[:, 0].tolist()]}, "
              f"entropies {[round(v, 2) for v in lp.entropy.tolist()]}")
    q4.q4nx_check(device=model.device)


if __name__ == "__main__":
    main()
