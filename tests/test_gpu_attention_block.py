"""The attention half of a layer on a GB300: projections, adapters, cache and attention together.

Each operator has its own tests against 64-bit references; these hold the way they are joined.
Tolerance of the whole against a plain 64-bit layer over the decoded weights: the 8-bit cache rounds
a key or value by at most 2^-4 of itself plus 2^-9 of its block's largest; with unit-variance rows
the score error is then below 2^-4 |q||k| / sqrt(D) in the worst case and about 2^-5 / sqrt(3)
in the mean square, so outputs differ by a few per cent of their size.  A wrong position, head,
row or page gives an unrelated row, an error of about the size itself: the bound is a quarter of it
in the mean square.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def make(new, lens_before=None, page=32, hq=8, hk=2, d=64, hidden=512, seed=0):
    import trellis_quantized_weight_gb300 as tq
    from trellis_quantized_weight_gb300.attention_block import AttentionBlock
    block = AttentionBlock(hidden, hq, hk, d, rank=16, adapters=3, positions=2048, seed=seed)
    S = len(new)
    cols = 16
    g = torch.Generator().manual_seed(seed)
    pages = torch.randperm(S * cols, generator=g).int().view(S, cols).cuda()
    cache = tq.kv_cache(S * cols, hk, page, d)
    x = torch.randn(sum(new), hidden, generator=g).bfloat16().cuda()
    starts = torch.tensor([0] + new).cumsum(0).int().cuda()
    kv_len = torch.tensor(new).int().cuda()
    which = torch.tensor([s % 4 - 1 for s in range(S)]).int().cuda()
    return block, cache, x, starts, kv_len, pages, which


def plain(block, x, new, which):
    """The layer in 64 bits, prompts only."""
    import trellis_quantized_weight_gb300 as tq

    def project(p, x, K):
        w = tq.decode(p.codes, p.scales, K, block.k).double()
        y = x @ w.T
        at = 0
        for n, ad in zip(new, which.tolist()):
            if ad >= 0:
                y[at:at + n] += (x[at:at + n] @ p.a[ad].double().T) @ p.b[ad].double().T
            at += n
        return y
    hq, hk, d = block.q_heads, block.kv_heads, block.head_dim
    qkv = project(block.qkv, x.double(), x.shape[1]).view(-1, hq + 2 * hk, d)
    at, outs = 0, []
    half = d // 2
    for n in new:
        rows = qkv[at:at + n]
        pos = torch.arange(n, device=x.device, dtype=torch.float64)[:, None]
        angle = pos * 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
        c, s = angle.cos()[:, None], angle.sin()[:, None]

        def turn(t):
            a, b = t[..., :half], t[..., half:]
            return torch.cat([a * c - b * s, b * c + a * s], -1)
        q, k, v = turn(rows[:, :hq]), turn(rows[:, hq:hq + hk]), rows[:, hq + hk:]
        k, v = k.repeat_interleave(hq // hk, 1), v.repeat_interleave(hq // hk, 1)
        score = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        score = score.masked_fill(torch.ones(n, n, device=x.device).triu(1).bool(), float("-inf"))
        outs.append(torch.einsum("hij,jhd->ihd", score.softmax(-1), v).reshape(n, hq * d))
        at += n
    return project(block.o, torch.cat(outs), hq * d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_against_a_plain_layer(d):
    new = [40, 1, 130, 7]
    block, cache, x, starts, kv_len, pages, which = make(new, d=d)
    got = block.step(x, cache, starts, kv_len, pages, which, max(new)).double()
    ref = plain(block, x, new, which)
    assert (got - ref).square().mean().sqrt() < 0.25 * ref.square().mean().sqrt()


def test_tokens_one_by_one_against_a_plain_layer():
    new = [33, 2, 80]
    block, cache, x, starts, kv_len, pages, which = make(new)
    ref = plain(block, x, new, which)
    first = [n // 2 for n in new]
    at = starts.tolist()
    rows = torch.cat([x[at[s]:at[s] + first[s]] for s in range(3)])
    seen = torch.tensor(first).int().cuda()
    st = torch.tensor([0] + first).cumsum(0).int().cuda()
    block.step(rows, cache, st, seen, pages, which, max(first))
    one = torch.arange(4).int().cuda()
    for i in range(min(n - f for n, f in zip(new, first))):
        seen += 1
        idx = [at[s] + first[s] + i for s in range(3)]
        got = block.step(x[idx], cache, one, seen, pages, which, 1).double()
        want = ref[idx]
        assert (got - want).square().mean().sqrt() < 0.25 * want.square().mean().sqrt()


def test_a_request_does_not_see_another():
    new = [50, 20, 64]
    block, cache, x, starts, kv_len, pages, which = make(new)
    a = block.step(x, cache, starts, kv_len, pages, which, 64)
    block, cache, _, starts, kv_len, pages, which = make(new)
    x2 = x.clone()
    x2[50:70] = 3.0
    b = block.step(x2, cache, starts, kv_len, pages, which, 64)
    assert torch.equal(a[:50], b[:50]) and torch.equal(a[70:], b[70:]) and not torch.equal(a[50:70], b[50:70])


def test_a_captured_step_follows_the_lengths():
    from trellis_quantized_weight_gb300.attention_block import capture
    new = [31, 5]

    def run(graphed):
        block, cache, x, starts, kv_len, pages, which = make(new)
        block.step(x, cache, starts, kv_len, pages, which, 31)
        one, row = torch.arange(3).int().cuda(), x[:2].clone()

        def decode():
            kv_len.add_(1)
            return block.step(row, cache, one, kv_len, pages, which, 1)
        outs = []
        if graphed:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            graph, out = capture(decode, stream)                 # one step outside the graph
            with torch.cuda.stream(stream):
                for _ in range(20):
                    graph.replay()
                    outs.append(out.clone())
            stream.synchronize()
            return outs
        return [decode() for _ in range(21)][1:]
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_the_command_runs(capsys):
    from trellis_quantized_weight_gb300 import attention_block
    attention_block.main(["--requests", "3", "--prompt", "40", "--steps", "4", "--hidden", "512", "--q-heads", "8",
                          "--kv-heads", "2", "--head-dim", "64", "--page", "16"])
    assert "us a step" in capsys.readouterr().out
