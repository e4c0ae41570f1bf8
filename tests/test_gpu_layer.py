"""A whole layer on a GB300: pages, norms, packed and 4-bit projections, cache and attention together.

Each operator has its own tests against 64-bit references; these hold the way they are joined.  Tolerance of the
gated half against a plain 64-bit one: the 8-bit rows round each activation by at most 2^-4 of itself (2^-4 / sqrt(3) in
the mean square), which enters two factors of the gate's product: outputs differ by less than 2^-3 of their size in the
mean square.  A wrong scale, row or weight gives an error of the size itself.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def make(S, cols=12, page=16, spare=0, hidden=512, inner=768, hq=8, hk=2, d=64, seed=0):
    import trellis_quantized_weight_gb300 as tq
    from trellis_quantized_weight_gb300.attention_block import AttentionBlock, Layer
    layer = Layer(AttentionBlock(hidden, hq, hk, d, rank=16, adapters=3, positions=2048, seed=seed), inner, seed=seed + 1)
    n = S * cols + spare
    cache, refs = tq.kv_cache(n, hk, page, d), tq.kv_pool(n)
    return layer, cache, refs, torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(S, cols, dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prompt(layer, cache, refs, kv_len, pages, new, hidden=512, seed=3):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(seed)
    assert tq.kv_grow(cache, refs, kv_len, pages, ints(new)).all()
    x = torch.randn(sum(new), hidden, generator=g).bfloat16().cuda()
    residual = torch.randn(sum(new), hidden, generator=g).bfloat16().cuda()
    starts = ints([0] + new).cumsum(0).int()
    return x, residual, layer.step(x, residual, cache, starts, kv_len, pages, ints([s % 4 - 1 for s in range(len(new))]), max(new))


def dense(w):
    q = torch.stack([(w.codes.long() >> (4 * i)) & 15 for i in range(8)], -1).flatten(1).double().unflatten(1, (w.scales.shape[1], -1))
    return (w.scales.double()[..., None] * q + w.biases.double()[..., None]).flatten(1)


def norm(h, w):
    return h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()


@pytest.mark.parametrize("new", [[5], [1, 1, 1], [40, 1, 77, 16], [130, 33]])
def test_the_gated_half_and_the_stream(new, monkeypatch):
    layer, cache, refs, kv_len, pages = make(len(new))
    seen = {}
    inner = layer.block.step
    monkeypatch.setattr(layer.block, "step", lambda n, *a: seen.setdefault("y", inner(seen.setdefault("n", n), *a)))
    x, stream, out = prompt(layer, cache, refs, kv_len, pages, new)
    g = torch.Generator().manual_seed(3)
    x0 = torch.randn(sum(new), 512, generator=g).bfloat16().cuda().double()
    h = x0 + torch.randn(sum(new), 512, generator=g).bfloat16().cuda().double()
    assert torch.equal(x0, x.double())
    want = norm(h, layer.norms[0])
    assert ((seen["n"].double() - want).abs() <= want.abs() * 2.0 ** -7).all()
    h1 = h.bfloat16().double() + seen["y"].double()
    assert ((stream.double() - h1).abs() <= h1.abs() * 2.0 ** -7 + 1e-6).all()
    m = norm(h1, layer.norms[1])
    gate, up = m @ dense(layer.gate).T, m @ dense(layer.up).T
    ref = (gate * torch.sigmoid(gate) * up) @ dense(layer.down).T
    assert (out.double() - ref).pow(2).mean().sqrt() <= ref.pow(2).mean().sqrt() * 2.0 ** -3


def decode(layer, cache, refs, kv_len, pages, steps, seed=9):
    import trellis_quantized_weight_gb300 as tq
    S = kv_len.numel()
    g = torch.Generator().manual_seed(seed)
    rows = [torch.randn(S, 512, generator=g).bfloat16().cuda() for _ in range(steps)]
    one, starts, which = ints([1] * S), ints(list(range(S + 1))), ints([0] * S)
    row, residual = torch.empty_like(rows[0]), torch.zeros_like(rows[0])

    def step():
        ok = tq.kv_grow(cache, refs, kv_len, pages, one)
        return ok, layer.step(row, residual, cache, starts, kv_len, pages, which, 1)
    return rows, row, residual, step


def test_forked_sequences_go_on_as_copies_would():
    """Six sequences with their prompts each, and two that are forked into three: the same bits from then on, over page ends,
    and the shared pages as they were."""
    import trellis_quantized_weight_gb300 as tq
    new = [37, 37, 37, 50, 50, 50]
    outs = []
    for forked in (False, True):
        layer, cache, refs, kv_len, pages = make(6, spare=8)
        # the rows of the sequences of a group are alike, so that their caches are
        g = torch.Generator().manual_seed(1)
        a, b = (torch.randn(n, 512, generator=g).bfloat16() for n in (37, 50))
        x = torch.cat([a, a, a, b, b, b]).cuda()
        assert tq.kv_grow(cache, refs, kv_len, pages, ints(new)).all()
        starts = ints([0] + new).cumsum(0).int()
        layer.step(x, torch.zeros_like(x), cache, starts, kv_len, pages, ints([0] * 6), 50)
        if forked:
            assert tq.kv_fork(cache, refs, kv_len, pages, ints([0, 0, 0, 5, 5, 5])).all()
            assert kv_len.tolist() == new and refs.max() == 3
            # 37 tokens: two whole pages in common and a third one each; 50: three and a fourth each
            assert int((refs > 0).sum()) == (2 + 3) + (3 + 3)
        rows, row, residual, step = decode(layer, cache, refs, kv_len, pages, 30)
        got = []
        for r in rows:
            row.copy_(r)
            ok, out = step()
            assert ok.all()
            got.append(out.clone())
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_captured_steps_hand_out_pages_as_eager_ones():
    results = []
    for captured in (False, True):
        layer, cache, refs, kv_len, pages = make(3)
        prompt(layer, cache, refs, kv_len, pages, [30, 1, 16])
        rows, row, residual, step = decode(layer, cache, refs, kv_len, pages, 25)
        if captured:
            stream = torch.cuda.Stream(priority=-1)          # not of the pool whose streams other tests look into
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    ok, out = step()
        got = []
        for r in rows:
            row.copy_(r)
            if captured:
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
            else:
                ok, out = step()
            assert ok.all()
            got.append(out.clone())
        results.append((got, kv_len.tolist(), pages.tolist(), refs.tolist()))
    for a, b in zip(results[0][0], results[1][0]):
        assert torch.equal(a, b)
    assert results[0][1:] == results[1][1:]


def test_a_moved_cache_goes_on():
    import trellis_quantized_weight_gb300 as tq
    layer, cache, refs, kv_len, pages = make(4, spare=40)
    prompt(layer, cache, refs, kv_len, pages, [30, 1, 16, 100])
    assert tq.kv_fork(cache, refs, kv_len, pages, ints([3, 3, 2, 3])).all()
    into = tq.kv_cache(60, 2, 16, 64)
    refs2, len2, pages2 = tq.kv_compact(cache, refs, kv_len, pages, into)
    assert len2.tolist() == [100, 100, 16, 100] and int((refs2 > 0).sum()) == int(pages2.max()) + 1
    got = []
    for c in ((cache, refs, kv_len, pages), (into, refs2, len2, pages2)):
        rows, row, residual, step = decode(layer, *c, 20)
        outs = []
        for r in rows:
            row.copy_(r)
            ok, out = step()
            assert ok.all()
            outs.append(out.clone())
        got.append(outs)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_the_command(capsys, monkeypatch):
    from trellis_quantized_weight_gb300 import attention_block

    class Stream(torch.cuda.Stream):                # of the other pool
        def __new__(cls, *a, **kw):
            return super().__new__(cls, *a, **{**kw, "priority": -1})
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    attention_block.main(["--requests", "3", "--prompt", "70", "--samples", "2", "--steps", "20", "--hidden", "512", "--inner", "768",
                          "--q-heads", "4", "--kv-heads", "1", "--head-dim", "64", "--page", "16"])
    out = capsys.readouterr().out
    assert "3 requests x 2" in out and "of one layer" in out
