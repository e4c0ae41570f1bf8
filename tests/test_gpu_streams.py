"""Calls with stream= : where their results' memory comes from, and how long their inputs' memory is held."""
import pytest

torch = pytest.importorskip("torch")
import helpers as H  # noqa: E402

pytestmark = pytest.mark.gpu


def calls():
    """name -> (tensors of a call, the call on a stream)"""
    import trellis_quantized_weight_gb300 as tq
    from trellis_quantized_weight_gb300 import synth
    i32 = dict(dtype=torch.int32, device="cuda")

    def bf16(*shape):
        return torch.randn(*shape, device="cuda").bfloat16()
    x, codes, scales = synth.small(5, 1024, 300, 3, seed=5).generate()
    x, codes, scales = H.dev_bf16(x), H.dev_codes(codes), H.dev_bf16(scales)
    cache = tq.kv_cache(8, 2, 64, 128)
    step = (torch.tensor([0, 40], **i32), torch.tensor([90], **i32), torch.arange(8, **i32).view(1, 8))
    table = tq.rope_table(4096, 128)
    return {
        "decode": ([codes, scales], lambda t, s: tq.decode(*t, 1024, 3, stream=s)),
        "gemm": ([x, codes, scales], lambda t, s: tq.gemm(*t, 3, stream=s)),
        "gateup": ([x, codes, scales, codes.clone(), scales.clone()], lambda t, s: tq.gemm_gateup(*t, 3, stream=s)),
        "packed": ([x, x.clone(), codes, scales], lambda t, s: tq.gemm_packed(t[:2], t[2], t[3], 3, stream=s)),
        "rope_table": ([], lambda t, s: tq.rope_table(4096, 128, stream=s)),
        "kv_append": ([*cache, bf16(40, 2, 128), bf16(40, 2, 128), *step, bf16(40, 8, 128), table],
                      lambda t, s: tq.kv_append(t[:4], *t[4:9], q=t[9], rope=t[10], stream=s)),
        "kv_attention": ([bf16(40, 8, 128), *cache, *step], lambda t, s: tq.kv_attention(t[0], t[1:5], *t[5:], stream=s)),
        "lora_add": ([bf16(40, 1000), bf16(40, 512), bf16(2, 16, 512), bf16(2, 1000, 16), torch.ones(2, device="cuda"),
                      torch.tensor([0, 40], **i32), torch.zeros(1, **i32)], lambda t, s: tq.lora_add(*t, stream=s)),
    }


NAMES = ["decode", "gemm", "gateup", "packed", "rope_table", "kv_append", "kv_attention", "lora_add"]


def flat(out):
    return [out] if isinstance(out, torch.Tensor) else [t for t in out if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_results_come_from_the_streams_memory(name):
    """Memory that the current stream frees is in its own order only: a call on another stream must not write there."""
    tensors, call = calls()[name]
    want = [t.clone() for t in flat(call(tensors, None))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = flat(call(tensors, s))
    s.synchronize()
    home = {}
    for seg in torch.cuda.memory_snapshot():
        home[(seg["address"], seg["address"] + seg["total_size"])] = seg["stream"]
    for t, w in zip(got, want):
        assert torch.equal(t, w)
        assert [st for (lo, hi), st in home.items() if lo <= t.data_ptr() < hi] == [s.cuda_stream]


@pytest.mark.parametrize("name", [n for n in NAMES if n != "rope_table"])
def test_inputs_are_held_until_the_stream_is_done(name):
    """Inputs that the caller drops while the call still waits on its stream are not handed out again."""
    tensors, call = calls()[name]
    call(tensors, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    tensors = [t.clone() for t in tensors]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)                     # some 0.2 s
    out = flat(call(tensors, s))
    mine = [(t.data_ptr(), t.numel() * t.element_size()) for t in tensors]
    sizes = [(t.shape, t.dtype) for t in tensors]
    del tensors, out
    new = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2) for shape, dtype in sizes]
    assert not s.query(), "the stream was done too early for this test to say anything"
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in new]
    assert not any(lo < p + n and p < hi for lo, hi in spans for p, n in mine)
    s.synchronize()
