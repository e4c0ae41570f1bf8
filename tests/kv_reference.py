"""Plain 64-bit restatements of the cache operators and the adapters, and random inputs for them.

Sequences are taken one at a time, with no code of the library: the tests' reference.
"""
from __future__ import annotations

import math

import torch

BLOCK = 16


class Step:
    """Packed rows of several sequences and a paged cache that holds `total` tokens of each."""

    def __init__(self, seed, new, total, hq, hk, d, page, device="cuda", spare=2, used_only=True):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.new, self.total, self.hq, self.hk, self.d, self.page = list(new), list(total), hq, hk, d, page
        self.tokens = sum(new)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.start = starts[:-1]
        need = [-(-max(t, 0) // page) for t in total]
        self.cols = max(1, max(need))
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        table = torch.full((len(new), self.cols), self.num_pages + 7, dtype=torch.int32)   # unused entries: out of range
        at = 0
        for i, k in enumerate(need):
            table[i, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
            at += k
        self.table = table
        self.dev = torch.device(device)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=self.dev)
        self.kv_len = torch.tensor(total, dtype=torch.int32, device=self.dev)
        self.pages = table.to(self.dev)
        self.gen = g

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen)

    def cache(self):
        """Random contents in the tokens' slots; NaN codes and NaN scales everywhere else."""
        shape = (self.num_pages, self.hk, self.page, self.d)
        out = []
        for _ in range(2):
            codes = torch.full(shape, 0x7F, dtype=torch.uint8)
            scales = torch.full(shape[:2] + (self.page // BLOCK,), math.nan)
            for i, t in enumerate(self.total):
                for b in range(0, max(t, 0), BLOCK):
                    ph, off = int(self.table[i, b // self.page]), b % self.page
                    n = min(BLOCK, t - b)
                    val = (self.randn(self.hk, n, self.d) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
                    codes[ph, :, off:off + n] = val.view(torch.uint8)
                    e = torch.randint(-9, -4, (self.hk,), generator=self.gen)
                    scales[ph, :, off // BLOCK] = torch.exp2(e.float())
            out.append((codes, scales))
        (kc, ks), (vc, vs) = out
        return [kc.to(self.dev).view(torch.float8_e4m3fn), vc.to(self.dev).view(torch.float8_e4m3fn),
                ks.to(self.dev), vs.to(self.dev)]


def stored(step, codes, scales, i, count):
    """The first `count` stored values of sequence i: float64 [heads, count, d]."""
    ids = step.table[i, :-(-count // step.page)].long().to(codes.device)
    x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
    x = x * scales[ids].double().repeat_interleave(BLOCK, -1)[..., None]
    return x.transpose(0, 1).reshape(step.hk, -1, step.d)[:, :count]


def attention(step, q, cache, scale, window=0):
    """(out, sum of p |v| / sum of p) in float64."""
    g = step.hq // step.hk
    out = torch.zeros(step.tokens, step.hq, step.d, dtype=torch.float64, device=step.dev)
    size = torch.zeros_like(out)
    for i, (n, t) in enumerate(zip(step.new, step.total)):
        if n == 0 or t <= 0:
            continue
        k, v = stored(step, cache[0], cache[2], i, t), stored(step, cache[1], cache[3], i, t)
        for r in range(n):
            pos = t - n + r
            lo = max(0, pos + 1 - window) if window else 0
            if pos < 0:
                continue
            x = q[step.start[i] + r].double().view(step.hk, g, step.d) @ k[:, lo:pos + 1].transpose(1, 2) * scale
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            out[step.start[i] + r] = (p @ v[:, lo:pos + 1]).reshape(step.hq, step.d)
            size[step.start[i] + r] = (p @ v[:, lo:pos + 1].abs()).reshape(step.hq, step.d)
    return out, size


def rotate(x, pos, table, rot, interleaved):
    """x [heads, d] float64 at position pos."""
    if table is None or pos < 0:
        return x
    y = x.clone()
    cos, sin = table[pos, :rot // 2].double(), table[pos, rot // 2:].double()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    y[:, ia] = x[:, ia] * cos - x[:, ib] * sin
    y[:, ib] = x[:, ib] * cos + x[:, ia] * sin
    return y


def power(a):
    """The smallest power of two s >= 2^-60 with a <= 448 s."""
    e = -60
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e
