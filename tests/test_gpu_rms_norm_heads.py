"""trellis_rms_norm of heads where rows are many or have a residual, against 64 bits on a GB300.  Tolerances as for rows."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -17


def check(x, w, residual=None):
    import trellis_quantized_weight_gb300 as tq
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    got = tq.rms_norm(x, w, residual=residual)
    eight = tq.rms_norm_q8(x, w, residual=residual)
    if residual is not None:
        (got, stream), want = got, (x.float() + residual.float()).bfloat16()
        assert torch.equal(stream, want) and torch.equal(eight[2], want)
    assert got.shape == x.shape and torch.all((got.double() - y).abs() <= y.abs() * (2.0 ** -8 + FP32) + 1e-38)
    codes, scales = eight[:2]
    assert codes.shape == x.shape and scales.shape == x.shape[:2]
    s = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    assert torch.all((scales.double() - s).abs() <= s * FP32)
    s = scales.double()[..., None]
    assert torch.all((codes.float().double() * s - y).abs() <= y.abs() * (2.0 ** -4 + FP32) + s * 2.0 ** -10)


# few rows and enough of them for the next one to be on its way while one is at work
@pytest.mark.parametrize("tokens,heads,width,extra", [(7, 5, 128, 2), (300, 40, 128, 16), (33, 3, 515, 1), (2100, 5, 1024, 2), (4001, 3, 640, 0),
                                                      (1300, 2, 5120, 1), (160, 2, 20000, 1), (3, 2, 40000, 1)])
@pytest.mark.parametrize("residual", [False, True])
def test_heads(tokens, heads, width, extra, residual):
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(tokens, (heads + extra) * width, generator=g, device="cuda").bfloat16()[:, :heads * width].unflatten(1, (heads, width))
    w = (1 + 0.3 * torch.randn(width, generator=g, device="cuda")).bfloat16()
    check(x, w, (torch.randn(tokens, heads, width, generator=g, device="cuda") * 4).bfloat16() if residual else None)


def test_heads_in_place():
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(2100, 5, 1024, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(1024).bfloat16().cuda()
    want, stream = tq.rms_norm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    tq.rms_norm(x1, w, residual=r1, residual_out=r1, out=x1)
    assert torch.equal(x1, want) and torch.equal(r1, stream)


def test_rows_of_no_values_have_no_scale():
    """The 8-bit form would hand out scales that nothing has written."""
    import trellis_quantized_weight_gb300 as tq
    none, w = torch.empty(4, 0).bfloat16().cuda(), torch.empty(0).bfloat16().cuda()
    with pytest.raises(ValueError):
        tq.rms_norm_q8(none, w)
    assert tq.rms_norm(none, w).shape == (4, 0)
    assert [t.shape for t in tq.rms_norm_q8(none[:0], w)] == [(0, 0), (0,)]
    assert [t.shape for t in tq.rms_norm_q8(torch.empty(4, 0, 64).bfloat16().cuda(), torch.ones(64).bfloat16().cuda())] == [(4, 0, 64), (4, 0)]
