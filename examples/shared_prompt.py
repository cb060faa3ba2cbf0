"""Decode steps of several requests behind one system prompt, a layer's operators in the order in which it needs them.

    python examples/shared_prompt.py [--requests 8] [--prompt 200] [--steps 4] [--encoder 77]

A skeleton of a layer in synthetic weights, without norms (the model's own business): every step

  q | k | v   = W x + bias, one merged Q4NX projection                           q4nx_gemm_epilogue
  k, v        go into the requests' 4-bit paged caches, q and k turned by their
              positions on the way                                               q4nx_kv_append_rotary
  a           = attention to them, the prompt once for all requests              q4nx_kv_attention_shared
  h           = x + Wo a                                                         q4nx_gemm_epilogue
  c           = attention of Wc h to an encoder's states of another length       q4nx_gemm_m64, q4nx_kv_attention_cross
  h           = h + Wd c                                                         q4nx_gemm_epilogue
  x           = h + Wdown (silu(Wgate h) * (Wup h))                              q4nx_gemm_m64, q4nx_gemm_epilogue twice

The prompt's pages stand in the tables of all requests; where it ends inside a page, each
request has a copy of that page for itself, whose part of the prompt nothing reads.
Residuals are added in place.  Nothing waits for the GPU between the calls of a step.
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
    inner: int = 2048
    heads: int = 16
    kv_heads: int = 8
    head_dim: int = 128
    page_tokens: int = 64
    positions: int = 4096


class Layer:
    def __init__(self, s: Sizes, device="cuda", seed: int = 0):
        self.s, self.device = s, torch.device(device)
        g = torch.Generator(device=device).manual_seed(seed)
        width, qkv = s.heads * s.head_dim, (s.heads + 2 * s.kv_heads) * s.head_dim

        def weight(rows, cols, n):
            _, w = synth.make(synth.Q4_1, rows, cols, synth.rng(91, n, rows + cols + seed))
            return q4.Weight(torch.from_numpy(w).to(device), synth.Q4_1, rows, cols)

        shapes = dict(qkv=(qkv, s.hidden), o=(s.hidden, width), c=(width, s.hidden), d=(s.hidden, width),
                      gate=(s.inner, s.hidden), up=(s.inner, s.hidden), down=(s.hidden, s.inner))
        for n, (name, shape) in enumerate(shapes.items()):
            setattr(self, name, weight(*shape, n))
        self.bias = (torch.randn(qkv, generator=g, device=device) * 0.1).bfloat16()
        self.rotary = q4.Rotary.make(s.positions, s.head_dim, base=1e6, device=device)


class Requests:
    """Requests behind a common prompt, each with an encoder's states: their caches, tables and lengths."""

    def __init__(self, layer: Layer, count: int, prompt: int, most: int, encoder: list[int]):
        s, dev = layer.s, layer.device
        self.layer, self.count, self.prompt = layer, count, prompt
        whole, cols = prompt // s.page_tokens, -(-(prompt + most) // s.page_tokens)
        own = cols - whole                                          # pages of each request for itself
        rng = np.random.default_rng(7)
        pages = rng.permutation(whole + count * own).astype(np.int32)
        table = np.concatenate([np.tile(pages[:whole], (count, 1)), pages[whole:].reshape(count, own)], 1)
        to = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
        self.cache = q4.KVCache.alloc(len(pages), s.kv_heads, s.head_dim, s.page_tokens, dev)
        self.table, self.lens, self.q_start = to(table), to([prompt] * count), to(range(count + 1))
        self.first, self.shared = to([0, count]), to([prompt])
        # the encoder's states, one cache for all requests
        need = [-(-n // s.page_tokens) for n in encoder]
        rows = np.full((count, max(max(need), 1)), -1, np.int32)
        at = np.cumsum([0] + need)
        for b, n in enumerate(need):
            rows[b, :n] = np.arange(at[b], at[b] + n)
        self.states = q4.KVCache.alloc(max(int(at[-1]), 1), s.kv_heads, s.head_dim, s.page_tokens, dev)
        self.states_table, self.states_lens = to(rows), to(encoder)
        g = torch.Generator(device=dev).manual_seed(11)
        draw = lambda n: torch.randn(n, s.kv_heads, s.head_dim, generator=g, device=dev).bfloat16()  # noqa: E731
        if prompt:                                                  # a prefill's keys and values, through the first request's table
            q4.q4nx_kv_append_rotary(self.cache, layer.rotary, None, draw(prompt), draw(prompt), to([0, prompt]), self.lens[:1], self.table[:1])
        if sum(encoder):
            q4.q4nx_kv_append(self.states, draw(sum(encoder)), draw(sum(encoder)), to([0, *np.cumsum(encoder)]), self.states_lens, self.states_table)

    def step(self, x: torch.Tensor) -> dict:
        """One new token of every request, bf16 [count, hidden], through the layer."""
        p, s = self.layer, self.layer.s
        qkv = q4.q4nx_gemm_epilogue(p.qkv, x, bias=p.bias).unflatten(1, (-1, s.head_dim))
        q, k, v = qkv[:, :s.heads], qkv[:, s.heads:s.heads + s.kv_heads], qkv[:, s.heads + s.kv_heads:]
        self.lens += 1
        turned = q4.q4nx_kv_append_rotary(self.cache, p.rotary, q, k, v, self.q_start, self.lens, self.table)
        a = q4.q4nx_kv_attention_shared(self.cache, turned, self.q_start, self.lens, self.table, self.first, self.shared)
        h = q4.q4nx_gemm_epilogue(p.o, a.flatten(1), residual=x)
        cq = q4.q4nx_gemm_m64(p.c, h).unflatten(1, (s.heads, s.head_dim))
        c = q4.q4nx_kv_attention_cross(self.states, cq, self.q_start, self.states_lens, self.states_table)
        mid = q4.q4nx_gemm_epilogue(p.d, c.flatten(1), residual=h)
        gated = q4.q4nx_gemm_epilogue(p.gate, mid, act="silu", mul=q4.q4nx_gemm_m64(p.up, mid))
        out = mid.clone()
        q4.q4nx_gemm_epilogue(p.down, gated, residual=out, out=out)
        return dict(qkv=qkv, turned=turned, attention=a, h=h, cross_q=cq, cross=c, mid=mid, gated=gated, out=out)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--encoder", type=int, default=77)
    a = ap.parse_args()
    if not 1 <= a.requests <= 64:
        ap.error("the products take 1..64 tokens a call")
    layer = Layer(Sizes(positions=a.prompt + a.steps))
    reqs = Requests(layer, a.requests, a.prompt, a.steps, [max(1, a.encoder * (b + 1) // a.requests) for b in range(a.requests)])
    x = torch.randn(a.requests, layer.s.hidden, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    for n in range(a.steps):
        x = reqs.step(x)["out"]
        x = x / x.float().pow(2).mean(1, keepdim=True).sqrt().bfloat16()      # in the place of the model's norm
        print(f"step {n}: lengths {reqs.lens.tolist()}, outputs {[round(v, 3) for v in x[:, 0].tolist()]}")
    q4.q4nx_check(device=layer.device)


if __name__ == "__main__":
    main()
