"""trellis_kv_attention: small weights of long contexts count.

One token's weight (or a few tokens' together) is 2^25.4 times that of each of the others, whose values
are 8 to 128 times as large: together the others have 2^(17 - 25.4) of the weight, or an eighth of that,
and some 5 per cent of the result.

Tolerance: 2^-8 |ref| + 2^-10 size as in test_gpu_kv_attention.py, and what a weight loses in f16, at most
2^-25 against a reference that is 2^6 or more below the largest: N 2^-31 max|v| in all.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu

N = 131072


def sharp(d, hot, seqs, hq, small, page=128, big=8.0):
    """One context of N tokens that every sequence reads; `hot` are the tokens of large weight.  Every row of every head
    is alike: (q, cache, starts, kv_len, pages, scale, the result in 64 bits, its size)."""
    pages = N // page
    dev = "cuda"
    k = torch.zeros(pages, 1, page, d, device=dev)
    v = torch.full((pages, 1, page, d), big, device=dev) * (1.0 - 0.25 * (torch.arange(d, device=dev) % 3))
    for t in hot:
        k[t // page, 0, t % page] = 1.5
        v[t // page, 0, t % page] = small
    one = torch.ones(pages, 1, page // 16, device=dev)
    cache = [k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), one, one.clone()]
    q = torch.ones(seqs, hq, d, device=dev).bfloat16()
    scale = 25.4 * math.log(2.0) / (1.5 * d)
    w = 2.0 ** -25.4 / len(hot)                     # of a token beside the hot ones' sum
    cold = big * (1.0 - 0.25 * (torch.arange(d, device=dev, dtype=torch.float64) % 3))
    ref = (small + (N - len(hot)) * w * cold) / (1.0 + (N - len(hot)) * w)
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.arange(pages, **i32).expand(seqs, pages).contiguous()
    return q, cache, torch.arange(seqs + 1, **i32), torch.full((seqs,), N, **i32), table, scale, ref


def check(d, hot, seqs, hq, small=0.5):
    import trellis_quantized_weight_gb300 as tq
    q, cache, starts, kv_len, pages, scale, ref = sharp(d, hot, seqs, hq, small)
    got = tq.kv_attention(q, cache, starts, kv_len, pages, scale=scale, max_q=1).double()
    tol = ref * (2.0 ** -8 + 2.0 ** -10) + N * 2.0 ** -31 * 8.0
    err = (got - ref).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max())}"


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_of_whole_units(d):
    """A sequence of 40 rows to a key head is one unit; as many as are not cut into parts."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check(d, [5], 4 * sms, 40)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_rows(d):
    """A token of large weight in each of the blocks that a CTA's warps begin with."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check(d, [16 * i + 3 for i in range(8)], 2 * sms, 8, small=0.0625)


@pytest.mark.parametrize("hq", [8, 40])
@pytest.mark.parametrize("seqs", [1, 3])
def test_units_in_parts(seqs, hq):
    check(128, [5], seqs, hq)


def test_the_reference_rises_late():
    """The largest score comes last and is 2^25.4 times the ones before: what was summed before is scaled down."""
    check(128, [N - 1], 1, 40)
    check(128, [N - 1], 1, 8)
