"""Outputs that overlap what a call still reads, or each other, are refused on the host (no GPU: every case fails
validation before any CUDA call)."""
import pytest

SHAPE = -2
X, R, W, Y, H, C, S, Z = (0x10000000 * i for i in range(1, 9))       # never dereferenced; each far from the others


@pytest.fixture(scope="module")
def lib():
    from trellis_quantized_weight_gb300 import build, binding
    build.build()
    return binding.load()


# 4 tokens of 2 rows of 128 values: 2048 bytes in all, 512 a token
NORM = dict(x=X, x_stride=256, residual=R, weight=W, rows=4, heads=2, width=128, eps=1e-6, out=Y, codes=0, scales=0, residual_out=H, stream=None)
EIGHT = dict(NORM, out=0, codes=C, scales=S)                          # 1024 bytes of codes, 32 of scales
APART = dict(NORM, x_stride=1024)                                     # tokens 2048 bytes apart


@pytest.mark.parametrize("base,change", [
    (NORM, dict(out=X + 2)), (NORM, dict(out=X - 2046)), (NORM, dict(out=X + 2046)), (NORM, dict(residual_out=X + 512)),
    (NORM, dict(out=R + 2)), (NORM, dict(residual_out=R - 512)), (NORM, dict(out=W + 254)), (NORM, dict(residual_out=W - 2046)),
    (NORM, dict(out=W)), (NORM, dict(out=H)), (NORM, dict(out=H + 2046)), (NORM, dict(residual_out=Y + 2)),
    (APART, dict(out=X)), (APART, dict(residual_out=X)), (APART, dict(out=X + 510)), (APART, dict(out=X + 3 * 2048 + 510)),
    (APART, dict(out=X + 514)), (APART, dict(residual_out=X - 2046)),
    (EIGHT, dict(codes=X)), (EIGHT, dict(codes=X + 2040)), (EIGHT, dict(codes=R)), (EIGHT, dict(codes=W)), (EIGHT, dict(codes=H + 1024)),
    (EIGHT, dict(scales=X + 2044)), (EIGHT, dict(scales=R)), (EIGHT, dict(scales=W + 252)), (EIGHT, dict(scales=H)),
    (EIGHT, dict(scales=C + 1020)), (EIGHT, dict(codes=S + 24)),
    (dict(EIGHT, x_stride=2048), dict(scales=X + 3 * 4096))])
def test_norm_refuses(lib, base, change):
    assert lib.trellis_rms_norm(*{**base, **change}.values()) == SHAPE


# 3 rows of 256 and 50: x 1536 bytes (768 in 8 bits), codes 6400, scales and biases 400 each, out 300
Q4 = dict(x=X, x_scales=0, codes=C, scales=S, biases=Z, M=3, K=256, N=50, group=64, out=Y, workspace=W, workspace_bytes=1 << 27, stream=None)


@pytest.mark.parametrize("change", [
    dict(out=C), dict(out=C + 6398), dict(out=C - 298), dict(out=S), dict(out=S + 398), dict(out=Z - 2), dict(out=Z + 200),
    dict(x_scales=R, out=R), dict(x_scales=R, out=R + 10), dict(x_scales=R, out=X + 766), dict(out=X + 1534),
    dict(x_scales=R, M=33, out=R + 130)])
def test_gemm_q4_refuses(lib, change):
    assert lib.trellis_gemm_q4(*{**Q4, **change}.values()) == SHAPE
