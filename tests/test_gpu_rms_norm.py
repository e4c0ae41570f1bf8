"""trellis_rms_norm against a plain 64-bit implementation on a GB300.

Tolerances.  bf16 outputs: a rounding, 2^-8 of the value, and the fp32 arithmetic before it: a sum of n squares in
parts of at most 32 values and trees of at most 2^5 * 2^5 parts (or, past 32768 values, n / 1024 a thread) is within
(32 + 10 + n / 1024) 2^-24 of itself, half of that goes into the root; the root, the quotient, the factor and the weight
add 6 roundings: below 2^-17 in all for n <= 2^16.  Scales: 2^-17 of themselves.  Codes: an e4m3 rounding is 2^-4 of the value, or
half a subnormal step, 2^-10 of the scale; the value itself is within 2^-17.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -17


def reference(x, w, eps, residual=None):
    h = x.double() if residual is None else x.double() + residual.double()
    return h, h / (h.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()


def check_y(got, y):
    err = (got.double() - y).abs()
    assert torch.all(err <= y.abs() * (2.0 ** -8 + FP32) + 1e-38), err.max()


def check_q8(codes, scales, y):
    top = y.abs().amax(-1)
    want = (top / 448).clamp(min=2.0 ** -100)
    assert torch.all((scales.double() - want).abs() <= want * FP32)
    s = scales.double()[..., None]
    err = (codes.float().double() * s - y).abs()
    assert torch.all(err <= y.abs() * (2.0 ** -4 + FP32) + s * 2.0 ** -10), err.max()


def data(rows, width, seed, big=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g)
    r = torch.randn(rows, width, generator=g) * 4
    if big:
        r[:, ::37] *= 50
    w = 1 + 0.3 * torch.randn(width, generator=g)
    return [t.bfloat16().cuda() for t in (x, r, w)]


# a warp's row of one, two and more units, each CTA size, odd widths, one past what the registers hold
WIDTHS = [1, 2, 7, 8, 63, 64, 128, 250, 256, 264, 511, 512, 520, 1001, 2048, 4088, 4096, 5120, 8192, 8200, 8193, 17408, 32768, 32769,
          32776, 65536]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_norm(width, rows):
    import trellis_quantized_weight_gb300 as tq
    if rows * width > 1 << 24:
        rows = 170
    x, r, w = data(rows, width, width + rows)
    h, y = reference(x, w, 1e-6, r)
    got, got_h = tq.rms_norm(x, w, residual=r)
    check_y(got, y)
    assert torch.equal(got_h, (x.float() + r.float()).bfloat16())
    codes, scales, got_h = tq.rms_norm_q8(x, w, residual=r)
    check_q8(codes, scales, y)
    assert torch.equal(got_h, (x.float() + r.float()).bfloat16())
    _, y = reference(x, w, 1e-3)
    check_y(tq.rms_norm(x, w, 1e-3), y)
    check_q8(*tq.rms_norm_q8(x, w, 1e-3), y)


@pytest.mark.parametrize("rows,width,pitch", [(9001, 520, 520), (10000, 1024, 1032), (2000, 5120, 5120), (3001, 4104, 4112), (1217, 8192, 8192),
                                              (700, 16384, 16384), (305, 16384, 16392), (9729, 640, 640)])
def test_rows_ahead(rows, width, pitch):
    """Many rows a CTA: the next one is on its way while one is at work, in place too."""
    import trellis_quantized_weight_gb300 as tq
    x, r, w = data(rows, pitch, 7)
    x, r, w = x[:, :width], r[:, :width].contiguous(), w[:width].contiguous()
    h, y = reference(x, w, 1e-6, r)
    got, got_h = tq.rms_norm(x, w, residual=r)
    check_y(got, y)
    assert torch.equal(got_h, (x.float() + r.float()).bfloat16())
    codes, scales, _ = tq.rms_norm_q8(x, w, residual=r)
    check_q8(codes, scales, y)
    stream = r.clone()
    again, _ = tq.rms_norm(x, w, residual=stream, residual_out=stream)
    assert torch.equal(again, got) and torch.equal(stream, got_h)
    if pitch == width:
        out = x.clone()
        tq.rms_norm(out, w, residual=r, out=out)
        assert torch.equal(out, got)
    _, y = reference(x, w, 1e-6)
    check_y(tq.rms_norm(x, w), y)
    check_q8(*tq.rms_norm_q8(x, w), y)


@pytest.mark.parametrize("tokens,heads,width,extra", [(1, 8, 128, 0), (5, 40, 128, 16), (300, 3, 64, 1), (33, 2, 256, 4), (7, 5, 100, 3),
                                                      (2, 3, 1024, 1)])
def test_heads_of_a_projection(tokens, heads, width, extra):
    import trellis_quantized_weight_gb300 as tq
    x, _, w = data(tokens, (heads + extra) * width, 5)
    w = w[:width].contiguous()
    x = x[:, :heads * width].unflatten(1, (heads, width))
    _, y = reference(x, w, 1e-6)
    check_y(tq.rms_norm(x, w), y)
    codes, scales = tq.rms_norm_q8(x, w)
    assert codes.shape == x.shape and scales.shape == x.shape[:2]
    check_q8(codes, scales, y)


@pytest.mark.parametrize("offset,width,pitch", [(0, 640, 648), (1, 640, 648), (3, 640, 641), (0, 100, 104), (4, 96, 200)])
def test_strided_and_unaligned_rows(offset, width, pitch):
    import trellis_quantized_weight_gb300 as tq
    base = torch.randn(9 * pitch + offset).bfloat16().cuda()
    x = base[offset:offset + 9 * pitch].view(9, pitch)[:, :width]
    w = torch.randn(width).bfloat16().cuda()
    _, y = reference(x, w, 1e-6)
    check_y(tq.rms_norm(x, w), y)
    check_q8(*tq.rms_norm_q8(x, w), y)


@pytest.mark.parametrize("width", [64, 515, 5120, 40000])
def test_in_place(width):
    import trellis_quantized_weight_gb300 as tq
    x, r, w = data(50, width, 9)
    want, want_h = tq.rms_norm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    y, h = tq.rms_norm(x1, w, residual=r1, residual_out=r1, out=x1)
    assert y is x1 and h is r1 and torch.equal(x1, want) and torch.equal(r1, want_h)
    x2, r2 = x.clone(), r.clone()
    tq.rms_norm(x2, w, residual=r2, residual_out=x2, out=r2)
    assert torch.equal(r2, want) and torch.equal(x2, want_h)


@pytest.mark.parametrize("width", [96, 5120, 40000])
def test_rows_of_zeros_and_not_finite(width):
    import trellis_quantized_weight_gb300 as tq
    x, _, w = data(6, width, 3)
    w = w.abs()
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, width - 1] = float("inf")
    x[3] = 1e-30
    _, y = reference(x, w, 1e-6)
    got = tq.rms_norm(x, w)
    assert torch.all(got[0] == 0) and got[1].isnan().all() and got[2, width - 1].isnan() and (got[2, :width - 1] == 0).all()
    check_y(got[3:], y[3:])
    codes, scales = tq.rms_norm_q8(x, w)
    assert scales[0].item() == 2.0 ** -100 and torch.all(codes[0].float() == 0)
    assert scales[1:3].isnan().all()
    check_q8(codes[3:], scales[3:], y[3:])
    zero_eps = tq.rms_norm(x[3:], w, 0.0)
    check_y(zero_eps[1:], reference(x[4:], w, 0.0)[1])


@pytest.mark.parametrize("width", [96, 640, 5120, 40000])
@pytest.mark.parametrize("rows", [2, 4000])
def test_rows_next_to_nothing(width, rows):
    """With a small eps the quotient of factor and scale is past fp32, the codes are not."""
    import trellis_quantized_weight_gb300 as tq
    if rows * width > 1 << 25:
        rows = 320
    g = torch.Generator().manual_seed(3)
    x = (torch.rand(rows, width, generator=g) * 2.0 ** -120 + 2.0 ** -122).bfloat16().cuda()
    x[::2] = 0
    w = (torch.rand(width, generator=g) + 0.25).bfloat16().cuda()
    for eps in (1e-20, 1e-30):
        _, y = reference(x, w, eps)
        check_y(tq.rms_norm(x, w, eps), y)
        codes, scales = tq.rms_norm_q8(x, w, eps)
        check_q8(codes, scales, y)
        assert not codes[::2].float().any()


def test_largest_value_becomes_448():
    import trellis_quantized_weight_gb300 as tq
    x = torch.zeros(1, 128).bfloat16().cuda()
    x[0, 7] = -3
    codes, scales = tq.rms_norm_q8(x, torch.ones(128).bfloat16().cuda(), 0.0)
    assert codes.float()[0, 7] == -448 and torch.isclose(scales[0], torch.tensor(128 ** 0.5 / 448).cuda(), rtol=1e-5)


def test_no_rows_and_refusals():
    import trellis_quantized_weight_gb300 as tq
    w = torch.ones(64).bfloat16().cuda()
    x = torch.ones(4, 64).bfloat16().cuda()
    assert tq.rms_norm(x[:0], w).shape == (0, 64)
    assert [t.shape for t in tq.rms_norm_q8(x[:0], w)] == [(0, 64), (0,)]
    for bad in (lambda: tq.rms_norm(x.float(), w), lambda: tq.rms_norm(x, w[:32]), lambda: tq.rms_norm(x, w.float()),
                lambda: tq.rms_norm(x.T.contiguous().T, torch.ones(64).bfloat16().cuda()), lambda: tq.rms_norm(x[0], w),
                lambda: tq.rms_norm(x, w, residual=x[:2]), lambda: tq.rms_norm(x, w, residual_out=x),
                lambda: tq.rms_norm(x, w, residual=x.clone(), residual_out=x, out=x), lambda: tq.rms_norm(x.cpu(), w),
                lambda: tq.rms_norm(x, w.cpu()), lambda: tq.rms_norm(x, w, out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(tq.TrellisError):
            tq.rms_norm(x, w, eps)


def test_on_a_given_stream_and_captured():
    import trellis_quantized_weight_gb300 as tq
    x, r, w = data(300, 5120, 1)
    want, want_h = tq.rms_norm(x, w, residual=r)
    codes, scales, _ = tq.rms_norm_q8(x, w, residual=r)
    stream = torch.cuda.Stream(priority=-1)
    torch.cuda.synchronize()
    got, got_h = tq.rms_norm(x, w, residual=r, stream=stream)
    eight = tq.rms_norm_q8(x, w, residual=r, stream=stream)
    stream.synchronize()
    assert torch.equal(got, want) and torch.equal(got_h, want_h)
    assert torch.equal(eight[0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(eight[1], scales) and torch.equal(eight[2], want_h)
    stream_r = r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, _ = tq.rms_norm(x, w, residual=stream_r, residual_out=stream_r)
        y8, s8 = tq.rms_norm_q8(y, w)
    with torch.cuda.stream(stream):
        for _ in range(2):
            stream_r.copy_(r)
            graph.replay()
            assert torch.equal(y, want) and torch.equal(stream_r, want_h)
            again = tq.rms_norm_q8(want, w)
            assert torch.equal(y8.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(s8, again[1])
    stream.synchronize()


def test_many_rows():
    """More values than 32 bits count."""
    import trellis_quantized_weight_gb300 as tq
    rows = (1 << 31) // 8192 + 5
    x = torch.zeros(rows, 8192, dtype=torch.bfloat16, device="cuda")
    x[-1], x[0] = 3, -2
    w = torch.ones(8192).bfloat16().cuda()
    y = tq.rms_norm(x, w, 0.0625)
    assert torch.all(y[0] == torch.tensor(-2 / 4.0625 ** 0.5).bfloat16().item()) and not y[1:-1:1009].any()
    assert torch.all(y[-1] == torch.tensor(3 / 9.0625 ** 0.5).bfloat16().item())
    del y
    codes, scales = tq.rms_norm_q8(x, w, 0.0625)
    assert torch.all(codes[-1].float() == 448) and torch.all(codes[0].float() == -448) and not codes[1:-1:1009].float().any()
