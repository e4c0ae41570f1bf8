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
