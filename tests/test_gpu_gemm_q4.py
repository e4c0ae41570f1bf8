"""trellis_gemm_q4 against a plain 64-bit implementation on a GB300.

The weights are the definition's: scale * code + bias (or scale * (code - 8)), rounded once to bf16.  Tolerance, element by
element: 2^-8 |ref| + size (K / 16 + 16) 2^-22, with size = s_m sum_k |x w|.  The first term is the result's rounding.
Products are exact; a step of the tensor cores adds 16 of them to the sum so far, each of the 17 terms cut or rounded within
2^-24 of the largest: at most 4 units of 2^-24 of the sum of magnitudes as the terms of a step share that sum.  The joins of
a cluster's parts and the activations' scale are the 16.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def weights(N, K, group, bias, g):
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, dtype=torch.int64).int().cuda()
    scales = ((torch.rand(N, K // group, generator=g) + 0.5) * 0.05).bfloat16().cuda()
    biases = (-scales.float() * (6 + 3 * torch.rand(N, K // group, generator=g).cuda())).bfloat16() if bias else None
    return codes, scales, biases


def reference(x, codes, scales, biases, x_scales=None):
    """(the product, the sum of magnitudes) in 64 bits."""
    N, K = codes.shape[0], codes.shape[1] * 8
    groups = scales.shape[1]
    q = torch.stack([(codes.long() >> (4 * i)) & 15 for i in range(8)], -1).view(N, groups, -1).double()
    s = scales.double()[..., None]
    w = s * q + biases.double()[..., None] if biases is not None else s * (q - 8)
    w = w.view(N, K).float().bfloat16().double()
    x = x.float().double()
    ref, size = x @ w.T, x.abs() @ w.abs().T
    if x_scales is not None:
        ref, size = ref * x_scales.double()[:, None], size * x_scales.double().abs()[:, None]
    return ref, size


def check(got, ref, size, K):
    tol = ref.abs() * 2.0 ** -8 + size * (K / 16 + 16) * 2.0 ** -22
    err = (got.double() - ref).abs()
    assert got.dtype == torch.bfloat16 and torch.all(err <= tol), ((err - tol).max(), err.max())


def run(M, K, N, group, bias, eight, seed=0, offset=0.0):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(seed)
    codes, scales, biases = weights(N, K, group, bias, g)
    x = torch.randn(M, K, generator=g) + offset
    x_scales = None
    if eight:
        x = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
        x_scales = (torch.rand(M, generator=g) * 0.02 + 0.001).cuda()
    else:
        x = x.bfloat16().cuda()
    got = tq.gemm_q4(x, codes, scales, biases, x_scales=x_scales)
    ref, size = reference(x, codes, scales, biases, x_scales)
    check(got, ref, size, K)
    return got


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130])
def test_rows(M, group, bias):
    run(M, 1280, 200, group, bias, M % 2 == 0, seed=M)


@pytest.mark.parametrize("K,group", [(32, 32), (64, 64), (96, 32), (128, 128), (160, 32), (192, 64), (384, 128), (4064, 32), (4160, 64), (8320, 128),
                                     (17408, 64)])
@pytest.mark.parametrize("M", [1, 12, 40, 200])
def test_depths(M, K, group):
    for bias in (False, True):
        run(M, K, 77, group, bias, bias, seed=K)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 127, 129, 1000, 5121])
@pytest.mark.parametrize("M", [1, 11, 64, 129])
def test_widths(M, N):
    run(M, 512, N, 64, True, False, seed=N)


@pytest.mark.parametrize("M", [3, 16, 50, 300])
def test_activations_with_a_mean(M):
    # the sums of a group are large against its centred part
    run(M, 2560, 300, 128, True, False, offset=8.0)
    run(M, 2560, 300, 32, False, True, offset=1.0)


@pytest.mark.parametrize("M,K,N,group", [(1, 5120, 17408, 64), (2000, 1024, 1000, 128), (257, 5120, 640, 64)])
def test_larger(M, K, N, group):
    run(M, K, N, group, True, False)
    run(M, K, N, group, False, True)


@pytest.mark.parametrize("K,group", [(32, 32), (64, 64), (128, 128), (128, 32), (256, 128), (384, 128), (640, 32), (1152, 64)])
@pytest.mark.parametrize("M", [40, 2049])
def test_many_tiles_of_few_stages(M, K, group):
    # each CTA takes ten tiles or five, one right after the other
    N = 200_000 if M == 40 else 5121
    for bias in (False, True):
        run(M, K, N, group, bias, bias, seed=K)


@pytest.mark.parametrize("M", [1, 12, 100])
def test_every_code(M):
    """Each code at each place of a word, by one-hot activations: exact but for the result's rounding."""
    import trellis_quantized_weight_gb300 as tq
    K, N = 128, 16
    q = (torch.arange(K)[None] + torch.arange(N)[:, None]) % 16
    codes = (q.view(N, -1, 8) << (4 * torch.arange(8))).sum(-1)
    codes = torch.where(codes >= 2 ** 31, codes - 2 ** 32, codes).int().cuda()
    x = torch.eye(K).bfloat16().cuda()
    for group in (32, 64, 128):
        s = torch.full((N, K // group), 0.5).bfloat16().cuda()
        for k0 in range(0, K, M):
            rows = x[k0:k0 + M].contiguous()
            want = 0.5 * (q.T[k0:k0 + M].float() - 8)
            assert torch.equal(tq.gemm_q4(rows, codes, s).float().cpu(), want)
            assert torch.equal(tq.gemm_q4(rows, codes, s, s).float().cpu(), want + 4.5)


@pytest.mark.parametrize("M", [1, 9, 64, 200])
def test_rows_that_are_not_finite_stay_alone(M):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(1)
    codes, scales, biases = weights(100, 640, 64, True, g)
    x = torch.randn(M, 640, generator=g).bfloat16().cuda()
    want = tq.gemm_q4(x, codes, scales, biases)
    y = x.clone()
    y[M // 2, 333] = float("inf")
    y[0, 5] = float("nan")
    got = tq.gemm_q4(y, codes, scales, biases)
    for m in range(M):
        if m in (0, M // 2):
            assert not got[m].isfinite().any()
        else:
            assert torch.equal(got[m], want[m])


@pytest.mark.parametrize("M", [1, 11, 64, 300])
def test_equal_calls_give_equal_bits(M):
    a, b = run(M, 5120, 1111, 64, True, False, seed=4), run(M, 5120, 1111, 64, True, False, seed=4)
    assert torch.equal(a, b)


def test_no_rows_out_and_refusals():
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(1)
    codes, scales, biases = weights(48, 256, 64, True, g)
    x = torch.randn(3, 256).bfloat16().cuda()
    assert tq.gemm_q4(x[:0], codes, scales).shape == (0, 48)
    out = torch.empty(3, 48).bfloat16().cuda()
    assert tq.gemm_q4(x, codes, scales, biases, out=out) is out
    assert torch.equal(out, tq.gemm_q4(x, codes.view(torch.uint32), scales, biases))
    x8, xs = tq.rms_norm_q8(x, torch.ones(256).bfloat16().cuda())
    for bad in (lambda: tq.gemm_q4(x8, codes, scales), lambda: tq.gemm_q4(x, codes, scales, x_scales=xs),
                lambda: tq.gemm_q4(x8, codes, scales, x_scales=xs[:2]), lambda: tq.gemm_q4(x[:, :128], codes, scales),
                lambda: tq.gemm_q4(x, codes[:, :16], scales), lambda: tq.gemm_q4(x, codes, scales[:40]),
                lambda: tq.gemm_q4(x, codes, scales, biases[:, :2]), lambda: tq.gemm_q4(x, codes, scales.float()),
                lambda: tq.gemm_q4(x.cpu(), codes, scales), lambda: tq.gemm_q4(x, codes.long(), scales),
                lambda: tq.gemm_q4(x, codes, scales, out=out[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tq.TrellisError):
        tq.gemm_q4(x, codes, torch.ones(48, 16).bfloat16().cuda())


@pytest.mark.parametrize("M,K,N,group,bias,eight", [(300, 5120, 1111, 32, True, False), (300, 5120, 1111, 64, True, False),
                                                    (16, 5120, 1111, 32, True, False), (64, 1152, 3001, 128, False, True),
                                                    (2000, 1024, 1000, 128, True, False)])
def test_many_calls_give_equal_bits(M, K, N, group, bias, eight):
    """Operands that a slow reader still needs are not overwritten: a few calls in a hundred differed where they could be."""
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(4)
    codes, scales, biases = weights(N, K, group, bias, g)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    x_scales = None
    if eight:
        x, x_scales = tq.rms_norm_q8(x, torch.ones(K).bfloat16().cuda())
    first = tq.gemm_q4(x, codes, scales, biases, x_scales=x_scales)
    check(first, *reference(x, codes, scales, biases, x_scales), K)
    differ = sum(not torch.equal(tq.gemm_q4(x, codes, scales, biases, x_scales=x_scales), first) for _ in range(300))
    assert differ == 0
    assert tq.load().trellis_device_status(None) == 0


@pytest.mark.parametrize("M,K,N,group,eight", [(3, 5120, 1111, 64, False), (3, 5120, 1111, 64, True), (200, 1280, 700, 32, True)])
def test_captured_and_replayed(M, K, N, group, eight):
    """Clusters of CTAs and the widened rows' workspace in a graph; inputs change between replays."""
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(2)
    codes, scales, biases = weights(N, K, group, True, g)
    xs = [torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(3)]
    x_scales = None
    if eight:
        one = torch.ones(K).bfloat16().cuda()
        xs, rows = zip(*(tq.rms_norm_q8(x, one) for x in xs))
        x_scales = rows[0].clone()
    want = [tq.gemm_q4(x, codes, scales, biases, x_scales=rows[i] if eight else None) for i, x in enumerate(xs)]
    x, out = xs[0].clone(), torch.empty_like(want[0])
    stream = torch.cuda.Stream(priority=-1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tq.gemm_q4(x, codes, scales, biases, x_scales=x_scales, out=out)
    with torch.cuda.stream(stream):
        for i in (1, 2, 0, 1):
            x.copy_(xs[i])
            if eight:
                x_scales.copy_(rows[i])
            out.zero_()
            graph.replay()
            assert torch.equal(out, want[i])
    stream.synchronize()


def test_on_two_streams_at_once():
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(2)
    codes, scales, biases = weights(3000, 5120, 64, True, g)
    one = torch.ones(5120).bfloat16().cuda()
    streams = [torch.cuda.Stream(priority=-1) for _ in range(2)]
    inputs = [tq.rms_norm_q8(torch.randn(M, 5120, generator=g).bfloat16().cuda(), one) for M in (9, 150)]
    want = [tq.gemm_q4(x, codes, scales, biases, x_scales=s) for x, s in inputs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(tq.gemm_q4(inputs[i][0], codes, scales, biases, x_scales=inputs[i][1], stream=streams[i]))
    for s in streams:
        s.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("M,group", [(1, 32), (3, 128), (40, 64), (200, 32)])
@pytest.mark.parametrize("bias", [False, True])
def test_scales_around_a_quarter(M, group, bias):
    """Weights are made in one of two ways, by the scales of 32 rows; both round the same number once."""
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(8)
    codes, _, _ = weights(200, 1280, group, bias, g)
    kinds = torch.tensor([0.0, 2.0 ** -20, 0.125, 0.2490234375, 0.25, -0.2490234375, -0.25, 0.375, 5.0]).bfloat16()
    picked = torch.randint(0, 9, (200, 1280 // group), generator=g)
    picked[32:64] = picked[32:64].clamp(max=3)                   # all of them below
    picked[64:96] = picked[64:96].clamp(min=4)
    scales = kinds[picked].cuda()
    biases = (torch.randn(200, 1280 // group, generator=g) * scales.float().cpu() * 8).bfloat16().cuda() if bias else None
    x = torch.randn(M, 1280, generator=g).bfloat16().cuda()
    check(tq.gemm_q4(x, codes, scales, biases), *reference(x, codes, scales, biases), 1280)
    one = torch.zeros(M, 1280).bfloat16().cuda()
    one[:, 777] = 1                                              # a weight alone: exact
    w = reference(torch.eye(1280)[777:778].bfloat16().cuda(), codes, scales, biases)[0]
    assert torch.equal(tq.gemm_q4(one, codes, scales, biases).double(), w.expand(M, -1))


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -60, 2.0 ** 60])
def test_small_and_large_scales(scale):
    """Weights below the normal numbers round as they are stored: to multiples of 2^-133."""
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(5)
    codes, _, _ = weights(40, 256, 32, False, g)
    s = (torch.rand(40, 8, generator=g).cuda() + 0.5).bfloat16() * scale
    q = torch.stack([(codes.long() >> (4 * i)) & 15 for i in range(8)], -1).view(40, 8, 32).double() - 8
    w = s.double()[..., None] * q
    w = (torch.round(w * 2.0 ** 133) * 2.0 ** -133 if scale < 2.0 ** -120 else w.float().bfloat16().double()).view(40, 256)
    for bias in (None, torch.zeros_like(s)):
        x = torch.zeros(256, 256).bfloat16().cuda()
        x.fill_diagonal_(2.0 ** 20 if scale < 1 else 2.0 ** -20)
        want = w.T * float(x[0, 0]) if bias is None else (s.double()[..., None] * (q + 8)).view(40, 256).T * float(x[0, 0])
        if bias is not None:
            v = (s.double()[..., None] * (q + 8)).view(40, 256)
            v = torch.round(v * 2.0 ** 133) * 2.0 ** -133 if scale < 2.0 ** -120 else v.float().bfloat16().double()
            want = v.T * float(x[0, 0])
        assert torch.equal(tq.gemm_q4(x, codes, s, bias).double(), want.float().bfloat16().double())
