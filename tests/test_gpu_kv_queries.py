"""trellis_kv_attention: a query row that is not finite, in both kernels."""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 50])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_is_nan_in_its_row_alone(d, new, bad):
    """A query with a NaN or an infinity has no softmax: its row is NaN, unless it sees no token; no other row changes."""
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(d, [new, new, 2], [200, 64, 1], 8, 2, d, 16)
    cache = step.cache()
    for c in (0, 1):                                # keys all positive: an infinity times them has one sign
        cache[c] = torch.where(cache[c].view(torch.uint8) == 0x7F, cache[c].view(torch.uint8),
                               (cache[c].view(torch.uint8) & 0x7F).clamp(min=8)).view(torch.float8_e4m3fn)
    q = step.randn(step.tokens, 8, d).bfloat16().to(step.dev)

    def run(x):
        return tq.kv_attention(x, cache, step.starts, step.kv_len, step.pages, max_q=new)
    ref = run(q)
    hit = q.clone()
    hit[new // 2, 3, d - 1] = bad
    hit[2 * new, 5, 0] = bad                        # stands before position 0: it sees nothing
    got = run(hit)
    assert torch.isnan(got[new // 2, 3]).all() and (got[2 * new] == 0).all()
    ref[new // 2, 3], got[new // 2, 3] = 0.0, 0.0
    assert torch.equal(got, ref)
