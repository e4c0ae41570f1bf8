"""trellis_lora_add against a plain 64-bit implementation on a GB300.

Tolerance, element by element: 2^-8 |ref| + 2^-15 size, size = |s| sum_r |B| sum_k |A x|.  The result's
rounding to bf16 is at most 2^-9 |ref|.  h = x A^T is an fp32 sum of exact products (each of the at most
K / 16 additions of 16 products rounds within 2^-23 of the sum's size, here below 2^-15.5 for K <= 17408
by a wide margin: rounding errors of a sum grow as its square root); it is split into two bf16, 2^-16 of
itself; the second sum is short.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def check(new, which, K, N, R, adapters, seed=0, out=None, alias=False, y_wide=0):
    import trellis_quantized_weight_gb300 as tq
    g = torch.Generator().manual_seed(seed)
    M = sum(new)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    y = torch.randn(M, N, generator=g).bfloat16().cuda()
    a = (torch.randn(adapters, R, K, generator=g) / K ** 0.5).bfloat16().cuda()
    b = torch.randn(adapters, N, R, generator=g).bfloat16().cuda()
    s = (torch.rand(adapters, generator=g) + 0.5).cuda()
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    starts = torch.tensor(at, dtype=torch.int32, device="cuda")
    w = torch.tensor(which, dtype=torch.int32, device="cuda")
    ref, size = y.double().clone(), torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for i, n in enumerate(new):
        if 0 <= which[i] < adapters and n:
            r = slice(at[i], at[i + 1])
            A, B = a[which[i]].double(), b[which[i]].double()
            ref[r] += float(s[which[i]]) * (x[r].double() @ A.T) @ B.T
            size[r] = float(s[which[i]]) * (x[r].double().abs() @ A.abs().T) @ B.abs().T
    y0 = y.clone()
    got = tq.lora_add(y, x, a, b, s, starts, w, out=y if alias else out)
    err = (got.double() - ref).abs()
    tol = ref.abs() * 2.0 ** -8 + size * 2.0 ** -15
    assert not torch.isnan(got).any()
    assert (err <= tol).all(), f"worst {float((err / tol).max())}"
    for i, n in enumerate(new):
        if not 0 <= which[i] < adapters:
            assert torch.equal(got[at[i]:at[i + 1]], y0[at[i]:at[i + 1]])
    if not alias:
        assert torch.equal(y, y0)
    again = tq.lora_add(y0.clone() if alias else y, x, a, b, s, starts, w)
    assert torch.equal(again, got)
    return got


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("new", [[1], [1, 1, 1], [3, 0, 17, 16], [65, 1, 200]])
def test_ranks(R, new):
    check(new, [i % 3 for i in range(len(new))], 520, 300, R, 3, seed=R)


@pytest.mark.parametrize("K", [8, 24, 32, 40, 256, 264, 5120, 17408])
def test_inner_sizes(K):
    check([1, 5, 40], [0, 1, 0], K, 136, 16, 2, seed=K)


@pytest.mark.parametrize("N", [1, 7, 8, 9, 31, 32, 33, 255, 256, 264, 1300, 5120])
@pytest.mark.parametrize("new", [[1, 2], [130]])
def test_output_sizes(N, new):
    check(new, [1, 0][:len(new)], 256, N, 32, 2, seed=N)


def test_requests_without_an_adapter():
    check([2, 3, 4, 1], [-1, 0, 7, -1], 256, 264, 16, 2)
    check([2, 3], [-1, -1], 256, 261, 16, 2)


def test_in_place():
    check([5, 70, 1], [0, -1, 1], 512, 200, 32, 2, alias=True)
    check([5, 70, 1], [0, -1, 1], 512, 203, 32, 2, alias=True)


def test_many_requests():
    check([1] * 300, [i % 41 - 1 for i in range(300)], 1024, 512, 16, 40)
    check([(i * 7) % 5 for i in range(300)], [i % 41 - 1 for i in range(300)], 1024, 512, 16, 40)


@pytest.mark.parametrize("R", [16, 64, 128])
def test_prompts(R):
    check([333, 700, 65], [1, 0, 1], 2560, 1288, R, 2)


def test_no_rows():
    import trellis_quantized_weight_gb300 as tq
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    got = tq.lora_add(z(0, 16), z(0, 8), z(1, 8, 8), z(1, 16, 8), torch.ones(1, device="cuda"),
                      torch.zeros(2, **i32), torch.zeros(1, **i32))
    assert got.shape == (0, 16)


def test_after_the_projection_on_its_workspace():
    """The product and its adapters in turn, through one workspace: both keep their results."""
    import trellis_quantized_weight_gb300 as tq
    from trellis_quantized_weight_gb300 import synth
    import helpers as H
    M, K, N, k = 5, 1024, 300, 3
    x, codes, scales = synth.small(M, K, N, k, seed=5).generate()
    dx, dc, ds = H.dev_bf16(x), H.dev_codes(codes), H.dev_bf16(scales)
    a = (torch.randn(2, 16, K, device="cuda") / 32).bfloat16()
    b = torch.randn(2, N, 16, device="cuda").bfloat16()
    s = torch.ones(2, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, which = torch.tensor([0, 2, 5], **i32), torch.tensor([1, 0], **i32)
    y = tq.gemm(dx, dc, ds, k)
    z = tq.lora_add(y, dx, a, b, s, starts, which)
    for _ in range(10):
        y2 = tq.gemm(dx, dc, ds, k)
        z2 = tq.lora_add(y2, dx, a, b, s, starts, which)
        assert torch.equal(y, y2) and torch.equal(z, z2)
