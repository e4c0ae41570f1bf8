"""The page operators, the norm and the 4-bit product refuse bad arguments on the host (no GPU: every
case fails validation before any CUDA call, in the documented order)."""
import ctypes

import pytest

P, Q = 0x10000, 0x10000000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from trellis_quantized_weight_gb300 import build, binding
    build.build()
    return binding.load()


POOL = dict(refs=P, kv_len=P, pages=P)
SIZES = dict(seqs=3, page_cols=5, num_pages=20, page_size=16)
WORK = dict(workspace=P, workspace_bytes=1 << 30, stream=None)
GROW = dict(POOL, grow=P, **SIZES, ok=P, **WORK)
CACHE = dict(kv_heads=2, head_dim=64, k_codes=P, v_codes=P, k_scales=P, v_scales=P)
FORK = dict(POOL, parents=P, **SIZES, **CACHE, ok=P, **WORK)
COMPACT = dict(POOL, **SIZES, **CACHE, num_pages_out=9, k_codes_out=Q, v_codes_out=Q + (1 << 20), k_scales_out=Q + (2 << 20),
               v_scales_out=Q + (3 << 20), refs_out=Q + (4 << 20), kv_len_out=Q + (5 << 20), pages_out=Q + (6 << 20), **WORK)
NORM = dict(x=P, x_stride=256, residual=P, weight=P, rows=4, heads=2, width=128, eps=1e-6, out=P, codes=0, scales=0, residual_out=Q, stream=None)
Q4 = dict(x=P, x_scales=0, codes=P, scales=P, biases=P, M=3, K=256, N=50, group=64, out=Q, workspace=P, workspace_bytes=1 << 30, stream=None)

SHARED = [(dict(refs=0), -1), (dict(kv_len=0), -1), (dict(pages=0), -1), (dict(seqs=0), -2), (dict(page_cols=0), -2), (dict(num_pages=0), -2),
          (dict(seqs=16385), -3), (dict(num_pages=(1 << 24) + 1), -3), (dict(page_cols=(1 << 24) + 1), -3), (dict(page_size=8), -3),
          (dict(page_size=48), -3), (dict(refs=P + 2), -4), (dict(kv_len=P + 1), -4), (dict(pages=P + 2), -4),
          (dict(workspace=0), -7), (dict(workspace_bytes=1 << 20), -7), (dict(workspace=P + 64), -4)]
HEADS = [(dict(k_codes=0), -1), (dict(v_codes=0), -1), (dict(k_scales=0), -1), (dict(v_scales=0), -1), (dict(kv_heads=0), -2),
         (dict(kv_heads=1025), -3), (dict(head_dim=96), -3), (dict(k_codes=P + 8), -4), (dict(v_codes=P + 4), -4), (dict(k_scales=P + 2), -4),
         (dict(v_scales=P + 1), -4)]


@pytest.mark.parametrize("change,want", SHARED + [(dict(grow=0), -1), (dict(ok=0), -1), (dict(grow=P + 2), -4)])
def test_grow_refuses(lib, change, want):
    assert lib.trellis_kv_grow(*{**GROW, **change}.values()) == want


@pytest.mark.parametrize("change,want", SHARED + HEADS + [(dict(parents=0), -1), (dict(ok=0), -1), (dict(parents=P + 2), -4)])
def test_fork_refuses(lib, change, want):
    assert lib.trellis_kv_fork(*{**FORK, **change}.values()) == want


@pytest.mark.parametrize("change,want", SHARED + HEADS + [
    (dict(refs_out=0), -1), (dict(kv_len_out=0), -1), (dict(pages_out=0), -1), (dict(k_codes_out=0), -1), (dict(v_scales_out=0), -1),
    (dict(num_pages_out=0), -2), (dict(num_pages_out=(1 << 24) + 1), -3), (dict(refs_out=Q + 2), -4), (dict(k_codes_out=Q + 8), -4),
    (dict(k_codes_out=P), -2), (dict(v_scales_out=P + 16), -2), (dict(k_codes_out=Q + (1 << 20)), -2), (dict(refs_out=P), -2),
    (dict(pages_out=Q + (5 << 20) + 4), -2), (dict(kv_len_out=P + 8), -2)])
def test_compact_refuses(lib, change, want):
    assert lib.trellis_kv_compact(*{**COMPACT, **change}.values()) == want


@pytest.mark.parametrize("args,want", [((0, 5, 20), -2), ((3, 0, 20), -2), ((3, 5, 0), -2), ((16385, 5, 20), -3), ((3, 5, (1 << 24) + 1), -3)])
def test_workspace_size(lib, args, want):
    n = ctypes.c_size_t(0)
    assert lib.trellis_kv_pages_workspace_size(*args, ctypes.byref(n)) == want
    assert lib.trellis_kv_pages_workspace_size(3, 5, 20, None) == -1
    assert lib.trellis_kv_pages_workspace_size(3, 5, 20, ctypes.byref(n)) == 0 and n.value > 1 << 20


@pytest.mark.parametrize("change,want", [
    (dict(x=0), -1), (dict(weight=0), -1), (dict(out=0), -1), (dict(codes=P), -1), (dict(codes=P, out=0), -1), (dict(scales=P), -1),
    (dict(residual=0), -1), (dict(residual_out=0), -1), (dict(rows=-1), -2), (dict(heads=0), -2), (dict(width=0), -2), (dict(eps=-1.0), -2),
    (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2), (dict(x_stride=255), -2), (dict(width=(1 << 20) + 1, heads=1, x_stride=1 << 21), -3),
    (dict(rows=2 ** 31 - 1, heads=2), -3), (dict(x=P + 1), -4), (dict(residual=P + 1), -4), (dict(out=P + 1), -4),
    (dict(out=0, codes=P, scales=P + 2), -4), (dict(residual_out=P), -2)])
def test_norm_refuses(lib, change, want):
    assert lib.trellis_rms_norm(*{**NORM, **change}.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(x=0), -1), (dict(codes=0), -1), (dict(scales=0), -1), (dict(out=0), -1), (dict(M=-1), -2), (dict(K=0), -2), (dict(N=0), -2),
    (dict(group=16), -3), (dict(group=256), -3), (dict(K=224), -2), (dict(M=65537), -3), (dict(K=(1 << 20) + 64), -3), (dict(N=(1 << 20) + 1), -3),
    (dict(out=P), -2), (dict(out=P + 1534), -2), (dict(x_scales=P, out=P + 766), -2),
    (dict(x=P + 8), -4), (dict(codes=P + 8), -4), (dict(scales=P + 1), -4), (dict(biases=P + 1), -4), (dict(x_scales=P + 2), -4), (dict(out=P + 1), -4),
    (dict(x_scales=P, M=33, out=Q, workspace=0), -7), (dict(x_scales=P, M=33, workspace_bytes=1 << 20), -7),
    (dict(x_scales=P, M=33, workspace=P + 64), -4)])
def test_gemm_q4_refuses(lib, change, want):
    assert lib.trellis_gemm_q4(*{**Q4, **change}.values()) == want


def test_nothing_to_do(lib):
    assert lib.trellis_rms_norm(*{**NORM, "rows": 0}.values()) == 0
    assert lib.trellis_gemm_q4(*{**Q4, "M": 0}.values()) == 0


@pytest.mark.parametrize("args,want", [((-1, 256, 5, 64, 0), -2), ((1, 0, 5, 64, 0), -2), ((1, 256, 0, 64, 0), -2),
                                       ((1, 256, 5, 48, 0), -3), ((1, 96, 5, 64, 0), -2), ((65537, 256, 5, 64, 0), -3)])
def test_gemm_q4_workspace_size(lib, args, want):
    n = ctypes.c_size_t(7)
    assert lib.trellis_gemm_q4_workspace_size(*args, ctypes.byref(n)) == want
    assert lib.trellis_gemm_q4_workspace_size(1, 256, 5, 64, 0, None) == -1
    assert lib.trellis_gemm_q4_workspace_size(300, 256, 5, 64, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.trellis_gemm_q4_workspace_size(32, 256, 5, 64, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.trellis_gemm_q4_workspace_size(300, 256, 5, 64, 1, ctypes.byref(n)) == 0 and n.value >= 300 * 512
