"""One stream's workspace under several users, on a GB300."""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def adapters(seed, M, K=512, N=1000, rank=32):
    g = torch.Generator().manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(y=torch.randn(M, N, generator=g).bfloat16().cuda(), x=torch.randn(M, K, generator=g).bfloat16().cuda(),
                a=torch.randn(2, rank, K, generator=g).bfloat16().cuda(), b=torch.randn(2, N, rank, generator=g).bfloat16().cuda(),
                scales=torch.ones(2, device="cuda"), starts=torch.tensor([0, M], **i32), which=torch.tensor([seed % 2], **i32))


def test_two_threads_on_one_stream():
    """Each thread's adapters add their own sums, whichever way the threads' launches fall."""
    import trellis_quantized_weight_gb300 as tq
    cases = [adapters(s, M) for s, M in enumerate((5, 5, 900, 33))]
    want = [tq.lora_add(**c) for c in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    go = threading.Barrier(len(cases))

    def work(i):
        go.wait()
        for _ in range(100):
            got[i].append(tq.lora_add(**cases[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert len(outs) == 100 and all(torch.equal(w, o) for o in outs)


def decode_step(stream):
    """A captured attention block step of single tokens, and what a prompt step needs beside it."""
    import trellis_quantized_weight_gb300 as tq
    from trellis_quantized_weight_gb300.attention_block import AttentionBlock, capture
    block = AttentionBlock(512, 32, 2, 256, rank=64, adapters=2, positions=2048)
    cache = tq.kv_cache(64, 2, 64, 256)
    pages = torch.arange(64, device="cuda").int().view(2, 32)
    g = torch.Generator().manual_seed(1)
    prompt = torch.randn(1600, 512, generator=g).bfloat16().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    which = torch.tensor([0, 1], **i32)
    kv_len = torch.tensor([700, 900], **i32)
    small = torch.tensor([0, 4, 8], **i32)
    eight = torch.tensor([4, 4], **i32)
    block.step(prompt[:8], cache, small, eight, pages, which, 4)          # the cache holds something
    row, one = prompt[:2].clone(), torch.arange(3, **i32)
    with torch.cuda.stream(stream):
        kv_len.copy_(eight + 1)
    torch.cuda.synchronize()
    graph, out = capture(lambda: block.step(row, cache, one, kv_len, pages, which, 1), stream)

    def prefill(cache):
        return block.step(prompt, cache, torch.tensor([0, 700, 1600], **i32), torch.tensor([700, 900], **i32), pages, which, 900)
    return block, cache, graph, out, prefill


def test_a_captured_step_outlives_a_larger_call():
    """A prompt on the capture's stream needs a larger workspace; replays keep theirs, whatever is allocated since."""
    import trellis_quantized_weight_gb300 as tq
    from trellis_quantized_weight_gb300 import binding
    stream = torch.cuda.Stream()
    block, cache, graph, out, prefill = decode_step(stream)
    with torch.cuda.stream(stream):
        graph.replay()
        want = out.clone()
        ws = binding._ws_cache[(0, stream.cuda_stream)]
        assert ws.in_graph
        before = ws.size
        prefill(tq.kv_cache(64, 2, 64, 256))
        assert ws.size > before and len(ws.kept) == 1                       # it did outgrow the captured one
        filled = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(300)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
        assert all(bool((t == 0xFF).all()) for t in filled)
    stream.synchronize()


def test_a_step_captured_without_a_first_call():
    """Its workspace is the graph's own; a call outside finds a sound one before and after the replays."""
    import trellis_quantized_weight_gb300 as tq
    c = adapters(1, 40)
    want = tq.lora_add(**c)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tq.lora_add(**c, out=out)
        tq.lora_add(**c, out=out)
    with torch.cuda.stream(s):
        assert torch.equal(tq.lora_add(**c), want)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want) and torch.equal(tq.lora_add(**c), want)
    s.synchronize()
