"""trellis_kv_attention with many rows to a key head over long contexts: units cut into equal shares.

Tolerances and reference as in test_gpu_kv_attention.py.
"""
import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402
from test_gpu_kv_attention import check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[5000, 5, 2100, 2112, 9000], [2049, 2049], [64 * 40 + 1], [40000, 6, 30, 7]])
def test_drafts_over_long_contexts(d, lens):
    check(R.Step(d + len(lens), [5] * len(lens), lens, 16, 2, d, 64))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sequences_without_rows_or_tokens_between(d):
    check(R.Step(d, [0, 6, 0, 0, 40, 7, 0], [50, 3000, 0, 7000, 2500, 7, 100], 16, 2, d, 32))
    check(R.Step(d, [0] * 40 + [6] + [0] * 40 + [5], [3] * 40 + [2600] + [0] * 40 + [4000], 16, 2, d, 32))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_nothing_beside_long_ones(d):
    from trellis_quantized_weight_gb300 import binding
    step = R.Step(d, [8, 8, 8], [3000, 3, 2900], 16, 2, d, 64)     # 5 rows of the second come before its first token
    got = check(step)
    at = int(step.starts[1])
    assert (got[at:at + 5] == 0).all()
    assert binding.load().trellis_device_status(None) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_query_tiles_of_one_head(d):
    check(R.Step(d, [1500, 3], [4500, 2300], 8, 1, d, 128))


@pytest.mark.parametrize("window", [100, 2500, 6000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_over_long_contexts(window, d):
    check(R.Step(window + d, [40, 9], [9000, 3100], 8, 2, d, 16), window=window)


@pytest.mark.parametrize("lens", [[9000, 300, 2500], [150, 90, 33]])
def test_equal_calls_give_equal_bits(lens):
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(5, [6] * 3, lens, 16, 2, 256, 64)
    cache = step.cache()
    q = step.randn(step.tokens, 16, 256).bfloat16().to(step.dev)
    first = tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=6)
    for _ in range(5):
        assert torch.equal(tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=6), first)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_units_of_one_tile(d):
    from trellis_quantized_weight_gb300 import binding
    lens = [20 + (i * 7) % 45 for i in range(90)]
    step = R.Step(d, [20] * 90, lens, 32, 4, d, 64)
    check(step)
    assert binding.load().trellis_device_status(None) == 0
