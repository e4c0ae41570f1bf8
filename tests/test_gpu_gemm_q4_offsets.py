"""trellis_gemm_q4 where groups lie far from zero, against the definition as it is, scale * code + bias, in 64 bits.

A weight is rounded once to bf16, by at most 2^-8 of what is rounded: of the weight itself where |bias| <= 32 |scale|, and
of scale * code + (bias - o), o = bf16(bias + 8 scale), beyond.  o is the bf16 number next to bias + 8 scale and bias is one,
so |bias - o| <= 16 |scale|, the codes lie in 0 .. 15, and the number that is rounded is at most 16 |scale|.  That bounds a
weight's error e: 2^-8 |w|, or 2^-4 |scale|.

An output is within sum |x| e + 2^-8 |ref| + the sums' error: a step of the tensor cores takes 16 products and the sum so
far, each cut within 2^-24 of the largest, in two passes where groups are far from zero.  The errors of single weights have
either sign and do not know of the activations, so in the mean square over all outputs they add as squares: that is the test
that tells a loss of the codes (a weight rounded at the bias' size is off by 2^-8 |bias| / 2 and more).
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def make(N, K, group, ratio, g, size=0.01):
    """Weights with biases `ratio` scales from zero, either way."""
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, dtype=torch.int64).int().cuda()
    scales = ((torch.rand(N, K // group, generator=g) + 0.5) * size)
    scales *= torch.randint(0, 2, scales.shape, generator=g) * 2 - 1
    scales = scales.bfloat16().cuda()
    away = (torch.rand(scales.shape, generator=g) * 0.5 + 0.75) * ratio * (torch.randint(0, 2, scales.shape, generator=g) * 2 - 1)
    return codes, scales, (scales.float() * away.cuda()).bfloat16()


def dense(codes, scales, biases):
    """(weights, the bound of a weight's error) [N, K] in 64 bits."""
    N, K = codes.shape[0], codes.shape[1] * 8
    q = torch.stack([(codes.long() >> (4 * i)) & 15 for i in range(8)], -1).view(N, scales.shape[1], -1).double()
    s, b = scales.double()[..., None], biases.double()[..., None]
    w = s * q + b
    e = torch.where(b.abs() > 32 * s.abs(), 2.0 ** -4 * s.abs(), 2.0 ** -8 * w.abs())
    return w.view(N, K), e.view(N, K)


def centred(M, K, group, g):
    """Activations whose groups add up to nothing: what the biases give is nothing, the codes are the whole product."""
    x = torch.randn(M, K // group, group, generator=g)
    return (x - x.mean(-1, keepdim=True)).view(M, K)


def check(got, x, w, e):
    x = x.double()
    K, ref = x.shape[1], x @ w.T
    most = torch.stack([torch.maximum((row * w).abs().amax(1), (row * w).cumsum(1).abs().amax(1)) for row in x])
    sums = (2 * K / 16 + 16) * 17 * 2.0 ** -24 * 2 * most
    err = (got.double() - ref).abs()
    assert torch.all(err <= x.abs() @ e.T + 2.0 ** -8 * ref.abs() + sums)
    square = ((2.0 ** -8 * ref) ** 2 + x ** 2 @ (e ** 2).T).mean()
    assert err.pow(2).mean().sqrt() <= square.sqrt() + sums.pow(2).mean().sqrt(), (err.pow(2).mean().sqrt(), square.sqrt(), ref.pow(2).mean().sqrt())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("ratio", [7.5, 30, 100, 512, 4096])
@pytest.mark.parametrize("M,N,K", [(1, 3000, 1280), (12, 300, 640), (40, 200, 1408), (130, 150, 1280), (3, 200, 8320)])
def test_biases_away_from_zero(M, N, K, ratio, group):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(K + group)
    codes, scales, biases = make(N, K, group, ratio, g)
    x = centred(M, K, group, g).bfloat16().cuda()
    check(tq.gemm_q4(x, codes, scales, biases), x, *dense(codes, scales, biases))


@pytest.mark.parametrize("M", [1, 20, 70])
def test_eight_bit_rows(M):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(M)
    codes, scales, biases = make(200, 1280, 64, 1024, g)
    x = (centred(M, 1280, 64, g) * 50).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    one = torch.full((M,), 0.25).cuda()
    got = tq.gemm_q4(x, codes, scales, biases, x_scales=one)
    check(got, x.float() * 0.25, *dense(codes, scales, biases))


@pytest.mark.parametrize("M,N,K,group", [(1, 20000, 256, 32), (33, 20000, 384, 64), (200, 5121, 640, 32), (2049, 1500, 1152, 128)])
def test_some_groups_among_many_tiles(M, N, K, group):
    """Few of the groups are far from zero, so that runs of scales with and without them follow each other."""
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(N)
    codes, scales, biases = make(N, K, group, 1000, g)
    near = (scales.float() * -7.5).bfloat16()
    some = (torch.rand(scales.shape, generator=g) < 2e-3).cuda()
    assert some.any()
    plain = tq.gemm_q4(x := centred(M, K, group, g).bfloat16().cuda(), codes, scales, near)
    got = tq.gemm_q4(x, codes, scales, torch.where(some, biases, near))
    rows = some.any(1)
    assert torch.equal(got[:, ~rows], plain[:, ~rows])               # the others' bits are as they were
    check(got[:, rows], x, *(t[rows] for t in dense(codes, scales, torch.where(some, biases, near))))


@pytest.mark.parametrize("M", [1, 9, 64, 200])
@pytest.mark.parametrize("size", [2.0 ** -100, 0.3, 2.0 ** 60])
def test_single_weights(M, size):
    """By one-hot activations: each weight within its bound and the result's rounding; groups of one value exact."""
    import trellis_quantized_weight_gb300 as tq
    K, group = 256, 32
    g = torch.Generator().manual_seed(M)
    codes, scales, biases = make(120, K, group, 300, g, size)
    scales[::7] = 0
    biases[:, ::3] = (scales.float() * 2)[:, ::3].bfloat16()
    biases[::14] = size
    w, e = dense(codes, scales, biases)
    x = torch.eye(K).bfloat16().cuda()
    for k0 in range(0, K, M):
        got = tq.gemm_q4(x[k0:k0 + M].contiguous(), codes, scales, biases).double()
        want, off = w.T[k0:k0 + M], e.T[k0:k0 + M]
        assert torch.all((got - want).abs() <= off * (1 + 2.0 ** -8) + want.abs() * (2.0 ** -8 + 2.0 ** -20))
        assert torch.equal(got[:, ::7], want[:, ::7])


@pytest.mark.parametrize("M,K,N,group", [(300, 5120, 1111, 32), (16, 5120, 1111, 32), (64, 1152, 3001, 128), (1, 640, 9000, 64), (2000, 1024, 1000, 128)])
def test_many_calls_give_equal_bits(M, K, N, group):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(4)
    codes, scales, biases = make(N, K, group, 500, g)
    near = (scales.float() * -7.5).bfloat16()
    biases = torch.where((torch.rand(scales.shape, generator=g) < 0.02).cuda(), biases, near)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    first = tq.gemm_q4(x, codes, scales, biases)
    differ = sum(not torch.equal(tq.gemm_q4(x, codes, scales, biases), first) for _ in range(200))
    assert differ == 0
    assert tq.load().trellis_device_status(None) == 0


def test_biases_that_are_not_finite_stay_in_their_columns():
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(4)
    codes, scales, biases = make(100, 640, 64, 500, g)
    x = torch.rand(5, 640, generator=g).bfloat16().cuda() + 1
    want = tq.gemm_q4(x, codes, scales, biases)
    bad = biases.clone()
    bad[7, 3], bad[50, 0] = float("inf"), float("nan")
    got = tq.gemm_q4(x, codes, scales, bad)
    keep = torch.ones(100, dtype=torch.bool, device="cuda")
    keep[7] = keep[50] = False
    assert torch.equal(got[:, keep], want[:, keep])
    assert torch.all(got[:, 7] == float("inf")) and got[:, 50].isnan().all()


def test_captured_and_on_two_streams_at_once():
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(1)
    jobs, want = [], []
    for M, K, N, group in ((3, 5120, 1111, 32), (150, 1280, 3000, 64)):         # a cluster's parts, and whole tiles
        codes, scales, biases = make(N, K, group, 500, g)
        biases = torch.where((torch.rand(scales.shape, generator=g) < 0.05).cuda(), biases, (scales.float() * -7.5).bfloat16())
        jobs.append((torch.randn(M, K, generator=g).bfloat16().cuda(), codes, scales, biases))
        want.append(tq.gemm_q4(*jobs[-1]))
    streams = [torch.cuda.Stream(priority=-1) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[tq.gemm_q4(*jobs[i], stream=streams[i]) for i in range(2)] for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for pair in got for y, w in zip(pair, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = [tq.gemm_q4(*job) for job in jobs]
    for _ in range(5):
        for y in out:
            y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(out, want))
