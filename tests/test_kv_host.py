"""The cache operators and the adapters refuse bad arguments on the host (no GPU: every
case fails validation before any CUDA call, in the documented order)."""
import ctypes

import pytest

P = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from trellis_quantized_weight_gb300 import build, binding
    build.build()
    return binding.load()


APPEND = dict(q=P, q_stride=2048, k=P, k_stride=512, v=P, v_stride=512, starts=P, kv_len=P, pages=P, tokens=4, seqs=2, max_q=2,
              page_cols=3, num_pages=9, q_heads=8, kv_heads=2, head_dim=128, page_size=16, rope=P, rope_rows=100, rot=64,
              interleaved=0, k_codes=P, v_codes=P, k_scales=P, v_scales=P, q_out=P, stream=None)
ATTEND = dict(q=P, q_stride=2048, starts=P, kv_len=P, pages=P, tokens=4, seqs=2, max_q=2, page_cols=3, num_pages=9, q_heads=8,
              kv_heads=2, head_dim=128, page_size=16, scale=0.1, window=0, k_codes=P, v_codes=P, k_scales=P, v_scales=P, out=P,
              workspace=P, workspace_bytes=1 << 30, stream=None)
COMMON = [
    (dict(starts=0), -1), (dict(kv_len=0), -1), (dict(pages=0), -1), (dict(k_codes=0), -1), (dict(v_codes=0), -1),
    (dict(k_scales=0), -1), (dict(v_scales=0), -1),
    (dict(tokens=-1), -2), (dict(seqs=0), -2), (dict(max_q=0), -2), (dict(page_cols=0), -2), (dict(num_pages=0), -2),
    (dict(kv_heads=0), -2), (dict(q_heads=1), -2), (dict(q_heads=7), -2), (dict(seqs=16385), -3), (dict(q_heads=1026), -3),
    (dict(head_dim=96), -3), (dict(head_dim=0), -3), (dict(page_size=8), -3), (dict(page_size=48), -3), (dict(page_size=256), -3),
    (dict(starts=P + 2), -4), (dict(kv_len=P + 1), -4), (dict(pages=P + 2), -4), (dict(k_codes=P + 8), -4),
    (dict(v_codes=P + 4), -4), (dict(k_scales=P + 2), -4), (dict(v_scales=P + 1), -4),
]


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(k=0), -1), (dict(v=0), -1), (dict(q=0), -1), (dict(q_out=0), -1),
    (dict(k_stride=248), -2), (dict(v_stride=0), -2), (dict(q_stride=1016), -2), (dict(rope_rows=0), -2),
    (dict(rot=8), -3), (dict(rot=0), -3), (dict(rot=40), -3), (dict(rot=144), -3),
    (dict(k=P + 2), -4), (dict(v=P + 8), -4), (dict(q=P + 4), -4), (dict(q_out=P + 2), -4), (dict(rope=P + 4), -4),
    (dict(k_stride=515), -4), (dict(v_stride=516), -4), (dict(q_stride=2050), -4),
])
def test_append_refuses(lib, change, want):
    assert lib.trellis_kv_append(*{**APPEND, **change}.values()) == want


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(q=0), -1), (dict(out=0), -1), (dict(q_stride=1016), -2), (dict(window=-1), -2), (dict(scale=float("nan")), -2),
    (dict(scale=float("inf")), -2), (dict(q=P + 2), -4), (dict(out=P + 8), -4), (dict(q_stride=2052), -4),
])
def test_attention_refuses(lib, change, want):
    assert lib.trellis_kv_attention(*{**ATTEND, **change}.values()) == want


@pytest.mark.parametrize("args,want", [
    ((-1, 2, 1, 8, 2, 128), -2), ((4, 0, 1, 8, 2, 128), -2), ((4, 2, 0, 8, 2, 128), -2), ((4, 2, 1, 7, 2, 128), -2),
    ((4, 2, 1, 8, 0, 128), -2), ((4, 99999, 1, 8, 2, 128), -3), ((4, 2, 1, 8, 2, 80), -3)])
def test_attention_workspace_size_refuses(lib, args, want):
    n = ctypes.c_size_t(0)
    assert lib.trellis_kv_attention_workspace_size(*args, ctypes.byref(n)) == want
    assert lib.trellis_kv_attention_workspace_size(4, 2, 1, 8, 2, 128, None) == -1


LORA = dict(y=P, x=P, a=P, b=P, scales=P, starts=P, which=P, M=4, K=64, N=33, R=16, adapters=2, segments=2, out=P, workspace=P,
            workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,want", [
    *[(dict([(n, 0)]), -1) for n in ("y", "x", "a", "b", "scales", "starts", "which", "out")],
    (dict(M=-1), -2), (dict(K=0), -2), (dict(K=60), -2), (dict(N=0), -2), (dict(R=0), -2), (dict(R=12), -2), (dict(adapters=0), -2),
    (dict(segments=0), -2), (dict(R=136), -3), (dict(M=65537), -3), (dict(segments=65537), -3),
    (dict(x=P + 2), -4), (dict(a=P + 8), -4), (dict(b=P + 8), -4), (dict(y=P + 1), -4), (dict(out=P + 1), -4),
    (dict(scales=P + 2), -4), (dict(starts=P + 2), -4), (dict(which=P + 2), -4)])
def test_lora_refuses(lib, change, want):
    assert lib.trellis_lora_add(*{**LORA, **change}.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(table=0), -1), (dict(rows=0), -2), (dict(base=0.0), -2), (dict(base=float("nan")), -2), (dict(stretch=0.5), -2),
    (dict(original=-1.0), -2), (dict(gain=0.0), -2), (dict(gain=float("inf")), -2), (dict(original=100.0, low=2.0, high=2.0), -2),
    (dict(rot=264), -3), (dict(rot=8), -3), (dict(table=P + 4), -4)])
def test_rope_table_refuses(lib, change, want):
    args = dict(table=P, rows=8, rot=64, base=1e4, stretch=1.0, original=0.0, low=1.0, high=32.0, gain=1.0, stream=None)
    assert lib.trellis_rope_table(*{**args, **change}.values()) == want


def test_the_binding_refuses_host_tensors():
    import torch
    import trellis_quantized_weight_gb300 as tq
    z = lambda *s, **k: torch.zeros(*s, **k)  # noqa: E731
    cache = (z(2, 1, 16, 64).to(torch.float8_e4m3fn),) * 2 + (z(2, 1, 1),) * 2
    i = z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.kv_attention(z(1, 1, 64).bfloat16(), cache, i, i[:1], i.view(1, 2))
    with pytest.raises(ValueError):
        tq.kv_append(cache, z(1, 1, 64).bfloat16(), z(1, 1, 64).bfloat16(), i, i[:1], i.view(1, 2))
    with pytest.raises(ValueError):
        tq.lora_add(z(1, 8).bfloat16(), z(1, 8).bfloat16(), z(1, 8, 8).bfloat16(), z(1, 8, 8).bfloat16(), z(1), i, i[:1])
    with pytest.raises(ValueError):
        tq.rope_table(0, 64)
