"""trellis_kv_attention, trellis_kv_append and trellis_lora_add in forms that the other files leave out.

Tolerances and references as in test_gpu_kv_attention.py and test_gpu_lora.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402
from test_gpu_kv_attention import check  # noqa: E402
from test_gpu_lora import check as check_lora  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 50])
@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_negative_and_zero_score_factors(d, new, scale):
    check(R.Step(d + new, [new, new], [333, 64], 8, 2, d, 16), scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 50])
@pytest.mark.parametrize("scale", [-0.5, -9.0])
def test_a_negative_factor_is_the_queries_sign(d, new, scale):
    """Bit for bit: the sign of a query is exact everywhere."""
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(d + new, [new, new], [333, 64], 8, 2, d, 16)
    cache = step.cache()
    q = step.randn(step.tokens, 8, d).bfloat16().to(step.dev)
    got = [tq.kv_attention(x, cache, step.starts, step.kv_len, step.pages, scale=f, max_q=new) for x, f in ((q, scale), (-q, -scale))]
    assert torch.equal(*got) and not torch.isnan(got[0]).any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 900])
def test_whole_units_of_long_contexts(d, window):
    """So many sequences and heads that no unit is cut: more units than CTAs, of lengths on both sides of 32 tiles."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    hk, group, unit_rows, new = 16, 3, 256 if d < 256 else 128, []
    while (sum(new) * group // unit_rows + len(new)) * hk < 4 * sms:
        new.append(60 - len(new) % 7)
    step = R.Step(d, new, [n + (i * 1237) % 4500 for i, n in enumerate(new)], hk * group, hk, d, 64)
    check(step, window=window)


def test_a_prompt_beside_single_tokens():
    lens = [1 + (i * 911) % 3000 for i in range(20)]
    for d in (64, 128, 256):
        check(R.Step(d, [1] * 10 + [300] + [1] * 10, lens[:10] + [700] + lens[10:], 8, 2, d, 64))


@pytest.mark.parametrize("R_", [16, 64, 128])
@pytest.mark.parametrize("alias", [False, True])
def test_adapters_of_prompts_with_odd_widths(R_, alias):
    check_lora([333, 700, 65], [1, -1, 0], 520, 1283, R_, 2, alias=alias)


@pytest.mark.parametrize("new", [[3, 2], [700, 800]])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_adapters_of_rows_that_are_not_finite(new, bad):
    """An infinite or NaN input reaches its own row, as infinities and NaN of the formula do; no other row changes."""
    import trellis_quantized_weight_gb300 as tq
    K, N, rank = 256, 264, 16
    g = torch.Generator().manual_seed(3)
    M = sum(new)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    y = torch.randn(M, N, generator=g).bfloat16().cuda()
    a = torch.zeros(2, rank, K)
    a[:, :, 7] = 0.5                                # every sum takes the bad element, with one sign
    a[:, :, 9] = 0.25
    b = torch.rand(2, N, rank, generator=g) + 0.5
    a, b, s = a.bfloat16().cuda(), b.bfloat16().cuda(), torch.ones(2, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, which = torch.tensor([0, new[0], M], **i32), torch.tensor([0, 1], **i32)
    ref = tq.lora_add(y, x, a, b, s, starts, which)
    x[new[0] + 1, 7] = bad
    y[0, 5] = bad
    got = tq.lora_add(y, x, a, b, s, starts, which)
    row = got[new[0] + 1].float()
    # (the columns of A that are zero leave 0 times the finite elements; the bad one is times 0.5)
    assert torch.isnan(row).all() if math.isnan(bad) else (row == bad).all()
    assert got[0, 5].isnan() if math.isnan(bad) else got[0, 5] == bad
    ref[new[0] + 1], got[new[0] + 1] = 0.0, 0.0
    ref[0, 5], got[0, 5] = 0.0, 0.0
    assert torch.equal(got, ref)


def test_adapterless_rows_pass_bit_by_bit():
    """NaN payloads, infinities and negative zeros of y included."""
    import trellis_quantized_weight_gb300 as tq
    i32 = dict(dtype=torch.int32, device="cuda")
    for M, N in ((70, 264), (70, 261), (1100, 264)):
        y = torch.arange(M * N, device="cuda").remainder(65536).to(torch.int32).to(torch.uint16).view(torch.bfloat16).view(M, N)
        x = torch.full((M, 64), math.nan, device="cuda").bfloat16()
        a, b = torch.ones(1, 8, 64, device="cuda").bfloat16(), torch.ones(1, N, 8, device="cuda").bfloat16()
        got = tq.lora_add(y, x, a, b, torch.ones(1, device="cuda"), torch.tensor([0, M], **i32), torch.tensor([-1], **i32))
        assert torch.equal(got.view(torch.int16), y.view(torch.int16))


def test_positions_past_the_table_take_its_last_row():
    import trellis_quantized_weight_gb300 as tq
    q, k, v = (torch.randn(5, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, kv_len, pages = torch.tensor([0, 5], **i32), torch.tensor([12], **i32), torch.tensor([[1]], **i32)
    short = tq.rope_table(9, 64)
    wide = torch.cat([short, short[-1:].expand(5, 64)]).contiguous()
    caches = [tq.kv_cache(2, 2, 16, 64) for _ in range(2)]
    outs = [tq.kv_append(c, k, v, starts, kv_len, pages, q=q, rope=t) for c, t in zip(caches, (short, wide))]
    assert torch.equal(*outs)
    for one, two in zip(*caches):
        assert torch.equal(one.view(torch.uint8), two.view(torch.uint8))
