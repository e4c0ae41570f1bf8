"""The attention half of a layer, and with it a whole one, served for many requests with adapters of their own.

    python -m trellis_quantized_weight_gb300.attention_block --requests 8 --prompt 300 --samples 2 --steps 64 --inner 17408

A step takes the packed rows of any mix of prompts, drafts and single tokens:

    kv_grow             lengths counted up, the pages for them taken from the pool
    n   = rms_norm(x)                               of the residual stream with what came before added
    qkv = gemm(n)  + the requests' adapters         one packed-weight projection
    q   = kv_append(k, v, q)                        rotary, and into the paged 8-bit cache
    o   = kv_attention(q)                           over the cache
    y   = gemm(o)  + the requests' adapters
    m   = rms_norm_q8(y)                            again with the stream's addition, to 8 bits
    z   = gemm_q4(silu(gemm_q4(m)) * gemm_q4(m))    a gated half with 4-bit weights

Lengths, page ids and the pool's counts are device arrays, so a step of fixed row counts can be captured in
a CUDA graph once and replayed while the sequences grow.  The command fills the cache with ragged
prompts, forks each into its samples, then replays captured single-token steps and prints their time.
"""
from __future__ import annotations

import argparse
from typing import NamedTuple

import torch

from . import (gemm, gemm_q4, kv_append, kv_attention, kv_cache, kv_fork, kv_grow, kv_pool, lora_add, rms_norm, rms_norm_q8,
               rope_table)


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


class Grouped(NamedTuple):
    """A projection with 4-bit weights: codes int32 [N, K / 8], scales and biases bf16 [N, K / group]."""
    codes: torch.Tensor
    scales: torch.Tensor
    biases: torch.Tensor

    @classmethod
    def random(cls, K, N, group, device, generator):
        codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K // 8), device=device, generator=generator, dtype=torch.int64).int()
        scales = torch.full((N, K // group), 0.2 * K ** -0.5, device=device).bfloat16()
        return cls(codes, scales, (-7.5 * scales.float()).bfloat16())


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


class Layer:
    """An attention block and a gated half of `inner` features with 4-bit weights, each behind a norm."""

    def __init__(self, block, inner, group=64, device="cuda", seed=1):
        g = torch.Generator(device=device).manual_seed(seed)
        hidden = block.o.codes.shape[0]
        self.block = block
        self.norms = [(1 + 0.1 * torch.randn(hidden, device=device, generator=g)).bfloat16() for _ in range(2)]
        self.gate, self.up = (Grouped.random(hidden, inner, group, device, g) for _ in range(2))
        self.down = Grouped.random(inner, hidden, group, device, g)

    def step(self, x, residual, *args, **kw):
        """x: bf16 [tokens, hidden], what came before, still to be added to the stream `residual`, which is updated in place
        (in a first layer x is the tokens' embeddings and the stream is zeros); the rest as AttentionBlock.step takes it.
        bf16 [tokens, hidden], to be added by what comes after."""
        n, _ = rms_norm(x, self.norms[0], residual=residual, residual_out=residual)
        y = self.block.step(n, *args, **kw)
        codes, scales, _ = rms_norm_q8(y, self.norms[1], residual=residual, residual_out=residual)
        gate, up = (gemm_q4(codes, *w, x_scales=scales) for w in (self.gate, self.up))
        return gemm_q4(torch.nn.functional.silu(gate).mul_(up), *self.down)


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
    ap.add_argument("--samples", type=int, default=1, help="continuations of each prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--inner", type=int, default=0, help="features of a gated half with 4-bit weights; 0: the attention half alone")
    ap.add_argument("--q-heads", type=int, default=40)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128, choices=(64, 128, 256))
    ap.add_argument("--page", type=int, default=64, choices=(16, 32, 64, 128))
    args = ap.parse_args(argv)

    dev, S, n = "cuda", args.requests, args.samples
    new = [max(1, args.prompt * (s + 1) // S) for s in range(S)]
    longest = max(new) + args.steps + 1                                   # one step runs before the capture
    block = AttentionBlock(args.hidden, args.q_heads, args.kv_heads, args.head_dim, positions=longest)
    layer = Layer(block, args.inner) if args.inner else None

    def run(x, residual, *a):
        return layer.step(x, residual, *a) if layer else block.step(x, *a)

    # request s has the slots s n .. s n + n - 1; its prompt goes to the first
    cols = -(-longest // args.page)
    cache = kv_cache(S * n * (cols + 1), args.kv_heads, args.page, args.head_dim)
    refs, pages = kv_pool(S * n * (cols + 1)), torch.zeros(S * n, cols, dtype=torch.int32, device=dev)
    kv_len = torch.zeros(S * n, dtype=torch.int32, device=dev)
    slot = torch.arange(S * n, device=dev).int()
    lead = slot // n * n
    which = (lead // n).remainder(5) - 1                                  # every fifth request has none
    rows = torch.tensor(new, device=dev).int()
    taken = torch.zeros(S * n, dtype=torch.int32, device=dev)
    taken[::n] = rows
    starts = torch.zeros(S * n + 1, dtype=torch.int32, device=dev)
    starts[1:] = taken.cumsum(0)
    kv_grow(cache, refs, kv_len, pages, taken)
    x = torch.randn(sum(new), args.hidden, device=dev).bfloat16()
    run(x, torch.zeros_like(x), cache, starts, kv_len, pages, which, max(new))
    kv_fork(cache, refs, kv_len, pages, lead)

    one, starts = torch.ones_like(slot), torch.arange(S * n + 1, device=dev).int()
    row = torch.randn(S * n, args.hidden, device=dev).bfloat16()
    residual = torch.empty_like(row)

    def decode():
        kv_grow(cache, refs, kv_len, pages, one)
        if layer:
            residual.zero_()                                              # a token's stream begins with its own row
        return run(row, residual, cache, starts, kv_len, pages, which, 1)

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
    print(f"{S} requests x {n} of up to {max(new)} + {args.steps} tokens: {us:.1f} us a step ({S * n / us * 1e6:.0f} tokens/s of one "
          f"{'layer' if layer else 'attention half'}), |out| {out.float().abs().mean().item():.3f}")


if __name__ == "__main__":
    main()
