"""The attention half of a layer, served for many requests with adapters of their own.

    python -m trellis_quantized_weight_gb300.attention_block --requests 8 --prompt 300 --steps 64

A step takes the packed rows of any mix of prompts, drafts and single tokens:

    qkv = gemm(x)  + the requests' adapters         one packed-weight projection
    q   = kv_append(k, v, q)                        rotary, and into the paged 8-bit cache
    o   = kv_attention(q)                           over the cache
    y   = gemm(o)  + the requests' adapters

Lengths and page ids are device arrays, so a step of fixed row counts can be captured in a CUDA
graph once and replayed while the sequences grow.  The command fills the cache with ragged
prompts, then replays captured single-token steps and prints their time.
"""
from __future__ import annotations

import argparse
from typing import NamedTuple

import torch

from . import gemm, kv_append, kv_attention, kv_cache, lora_add, rope_table


class Packed(NamedTuple):
    """A projection: codes int32 [N, K k / 32], scales bf16 [N], and adapters a [n, R, K], b [n, N, R]."""
    codes: torch.Tensor
    scales: torch.Tensor
    a: torch.Tensor
    b: torch.Tensor
    factors: torch.Tensor

    @classmethod
    def random(cls, K, N, k, adapters, rank, device, generator):
        def normal(*shape):
            return torch.randn(*shape, device=device, generator=generator)
        codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K * k // 32), device=device, generator=generator,
                              dtype=torch.int64).int()
        return cls(codes, torch.full((N,), K ** -0.5, device=device).bfloat16(),
                   (normal(adapters, rank, K) * K ** -0.5).bfloat16(), (normal(adapters, N, rank) * 0.1).bfloat16(),
                   torch.ones(adapters, device=device))


class AttentionBlock:
    """q_heads and kv_heads of head_dim over hidden features; k bits a weight; contexts of up to `positions` tokens
    (later ones would be rotated as the last)."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, k=4, adapters=4, rank=16, positions=32768, device="cuda",
                 seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.k, self.q_heads, self.kv_heads, self.head_dim = k, q_heads, kv_heads, head_dim
        self.qkv = Packed.random(hidden, (q_heads + 2 * kv_heads) * head_dim, k, adapters, rank, device, g)
        self.o = Packed.random(q_heads * head_dim, hidden, k, adapters, rank, device, g)
        self.rope = rope_table(positions, head_dim, device=device)

    def project(self, p, x, starts, which):
        y = gemm(x, p.codes, p.scales, self.k)
        return lora_add(y, x, p.a, p.b, p.factors, starts, which, out=y)

    def step(self, x, cache, starts, kv_len, pages, which, max_q, window=0):
        """x: bf16 [tokens, hidden], rows starts[s] .. starts[s + 1] of request s, whose cache holds kv_len[s]
        tokens with these; which[s]: its adapter, or -1.  bf16 [tokens, hidden]."""
        tokens, hq, hk, d = x.shape[0], self.q_heads, self.kv_heads, self.head_dim
        qkv = self.project(self.qkv, x, starts, which).view(tokens, hq + 2 * hk, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        q = kv_append(cache, k, v, starts, kv_len, pages, q=q, rope=self.rope, max_q=max_q)
        o = kv_attention(q, cache, starts, kv_len, pages, window=window, max_q=max_q)
        return self.project(self.o, o.view(tokens, hq * d), starts, which)


def capture(step, stream):
    """A graph of step(), whose buffers a first call outside the graph has set up."""
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
    return graph, out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--q-heads", type=int, default=40)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128, choices=(64, 128, 256))
    ap.add_argument("--page", type=int, default=64, choices=(16, 32, 64, 128))
    args = ap.parse_args(argv)

    dev, S = "cuda", args.requests
    new = [max(1, args.prompt * (s + 1) // S) for s in range(S)]
    longest = max(new) + args.steps + 1                                   # one step runs before the capture
    block = AttentionBlock(args.hidden, args.q_heads, args.kv_heads, args.head_dim, positions=longest)
    cols = -(-longest // args.page)
    pages = torch.randperm(S * cols, device=dev).int().view(S, cols)
    cache = kv_cache(S * cols, args.kv_heads, args.page, args.head_dim)
    which = torch.arange(S, device=dev).remainder(5).int() - 1            # every fifth request has none
    starts = torch.tensor([0] + new, device=dev).cumsum(0).int()
    kv_len = torch.tensor(new, device=dev).int()
    x = torch.randn(sum(new), args.hidden, device=dev).bfloat16()
    block.step(x, cache, starts, kv_len, pages, which, max(new))

    one = torch.arange(S + 1, device=dev).int()
    row = torch.randn(S, args.hidden, device=dev).bfloat16()

    def decode():
        kv_len.add_(1)
        return block.step(row, cache, one, kv_len, pages, which, 1)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph, out = capture(decode, stream)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(stream):
        begin.record()
        for _ in range(args.steps):
            graph.replay()
        end.record()
    end.synchronize()
    us = begin.elapsed_time(end) * 1e3 / args.steps
    print(f"{S} requests of up to {max(new)} + {args.steps} tokens: {us:.1f} us a step "
          f"({S / us * 1e6:.0f} tokens/s of one layer's attention half), |out| {out.float().abs().mean().item():.3f}")


if __name__ == "__main__":
    main()
