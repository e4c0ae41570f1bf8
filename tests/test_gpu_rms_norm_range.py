"""trellis_rms_norm of rows whose squares fp32 does not hold, against 64 bits on a GB300.

bf16 reaches from 2^-133 to 2^128, so squares of finite values reach from 2^-266 to 2^256.  Tolerances as for other rows: a
bf16 rounding, 2^-8, and 2^-17 for the arithmetic before it; scales 2^-17; codes 2^-4 of the value or 2^-10 of the scale.
Below 2^-126 fp32 keeps multiples of 2^-149, which the products with the weights of the 8-bit form are rounded to: half of
that times the factor is added where rows are so small.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -17
WIDTHS = [1, 64, 100, 515, 640, 5120, 8192, 17408, 40000]
ROWS = [3, 4000]


def reference(h, w, eps):
    factor = 1 / (h.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return h * factor * w.double(), factor


def check(x, w, eps, residual=None):
    import trellis_quantized_weight_gb300 as tq
    h = x.double() if residual is None else x.double() + residual.double()
    y, factor = reference(h, w, eps)
    assert y.isfinite().all()
    got = tq.rms_norm(x, w, eps, residual=residual)
    got = got if residual is None else got[0]
    assert torch.all((got.double() - y).abs() <= y.abs() * (2.0 ** -8 + FP32) + 1e-38)
    codes, scales = tq.rms_norm_q8(x, w, eps, residual=residual)[:2]
    low = 2.0 ** -150 * factor
    want = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    assert torch.all((scales.double() - want).abs() <= want * FP32 + low[..., 0] / 448)
    s = scales.double()[..., None]
    assert torch.all((codes.float().double() * s - y).abs() <= y.abs() * (2.0 ** -4 + FP32) + s * 2.0 ** -10 + low)


def data(rows, width, size, seed):
    if rows * width > 1 << 24:
        rows = 330
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g)
    x[x.abs() < 0.1] = 0.1
    w = 1 + 0.3 * torch.rand(width, generator=g)
    return (x * size).bfloat16().cuda(), w.bfloat16().cuda()


@pytest.mark.parametrize("size", [2.0 ** 50, 2.0 ** 62, 2.0 ** 83, 2.0 ** 120])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", ROWS)
def test_large_rows(rows, width, size):
    x, w = data(rows, width, size, width)
    for eps in (1e-6, 0.0):
        check(x, w, eps)
    check(x, w, 1e-6, residual=x.roll(1, 0))


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -60, 2.0 ** -75, 2.0 ** -100, 2.0 ** -125])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", ROWS)
def test_small_rows(rows, width, size):
    x, w = data(rows, width, size, width)
    for eps in (0.0, 1e-30, size * size / 3 if size > 2.0 ** -70 else 1e-37):
        check(x, w, float(torch.tensor(eps, dtype=torch.float32)))
    check(x, w, 0.0, residual=x.roll(1, 0).abs() * x.sign() * 0.25)         # of one sign: no sum of zero, which an eps of 0 has no norm of


@pytest.mark.parametrize("width", WIDTHS[1:])
@pytest.mark.parametrize("rows", ROWS)
def test_rows_of_every_size_side_by_side(rows, width):
    """Small, ordinary and large values in one row, and rows of each size next to each other."""
    x, w = data(rows, width, 1.0, 5)
    x = x.float()
    x[::3, ::5] *= 2.0 ** 100
    x[::3, 1::5] *= 2.0 ** -100
    x[1::3, ::7] *= 2.0 ** -110
    x[1::3, 1::7] *= 2.0 ** 30
    x[2::6] *= 2.0 ** 55
    x[5::6] *= 2.0 ** -80
    for eps in (1e-6, 0.0):
        check(x.bfloat16(), w, eps)


@pytest.mark.parametrize("width", [96, 5120, 40000])
def test_the_row_that_an_eps_of_zero_left_out(width):
    x, w = data(4, width, 1.0, 1)
    x[0], x[1] = 1e-30, 1e25
    check(x, w, 0.0)
    check(x, w, 1e-6)


@pytest.mark.parametrize("width", [96, 5120, 40000])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_large_rows_beside_rows_that_are_not_finite(width, eps):
    import trellis_quantized_weight_gb300 as tq
    x, w = data(600, width, 2.0 ** 90, 2)
    x[1::4, width // 2] = float("inf")
    x[2::4, 3] = float("nan")
    keep = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
    keep[1::4] = keep[2::4] = False
    y, _ = reference(x[keep].double(), w, eps)
    got = tq.rms_norm(x, w, eps)
    assert torch.all((got[keep].double() - y).abs() <= y.abs() * (2.0 ** -8 + FP32) + 1e-38)
    assert got[2::4].isnan().all() and got[1::4, width // 2].isnan().all()
    assert not got[1::4, :width // 2].any() and not got[1::4, width // 2 + 1:].any()
    codes, scales = tq.rms_norm_q8(x, w, eps)
    assert scales[keep].isfinite().all() and scales[~keep].isnan().all()
    assert torch.all((codes[keep].float().double() * scales[keep].double()[:, None] - y).abs()
                     <= y.abs() * (2.0 ** -4 + FP32) + scales[keep].double()[:, None] * 2.0 ** -10)
