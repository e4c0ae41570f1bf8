"""trellis_kv_attention: a block that a row does not see leaves no trace in the row, NaN or not.

A block that took a NaN or an infinity has a NaN scale.  Rows that see it are NaN; rows that do not see
it, by causality or by their window, are what they are when the block is sound, whichever other rows
share their tile and their unit (tolerance and reference as in test_gpu_kv_attention.py); other
sequences keep their bits.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu


def poisoned(step, block, seq=0):
    """A sound cache, and copies in which the keys, the values or both of a block are NaN: scale and codes."""
    cache = step.cache()
    page, at = int(step.table[seq, block * 16 // step.page]), block * 16 % step.page
    out = []
    for which in ((0,), (1,), (0, 1)):
        bad = [t.clone() for t in cache]
        for w in which:
            bad[w].view(torch.uint8)[page, :, at:at + 16] = 0x7F
            bad[2 + w][page, :, at // 16] = math.nan
        out.append(bad)
    return cache, out


def check(step, block, window=0):
    import trellis_quantized_weight_gb300 as tq
    n, total = step.new[0], step.total[0]
    q = step.randn(step.tokens, step.hq, step.d).bfloat16().to(step.dev)

    def run(cache):
        return tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, window=window, max_q=max(step.new))
    sound, bad = poisoned(step, block)
    before = run(sound)
    ref, size = R.attention(step, q, sound, step.d ** -0.5, window)
    tol = ref.abs() * 2.0 ** -8 + size * 2.0 ** -10
    pos = torch.arange(total - n, total)
    low = (pos + 1 - window).clamp(min=0) if window else torch.zeros_like(pos)
    sees = ((pos >= 16 * block) & (low < 16 * block + 16)).to(step.dev)
    for cache in bad:
        got = run(cache)
        assert torch.isnan(got[:n][sees]).all()
        assert ((got[:n].double() - ref[:n]).abs() <= tol[:n])[~sees].all()
        assert torch.equal(got[n:], before[n:])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,total,hq,hk", [
    (4, 18, 8, 4), (4, 18, 4, 2), (8, 36, 2, 2), (8, 132, 4, 2),          # few rows: drafts that reach into a new block
    (40, 60, 8, 2), (100, 100, 6, 2), (300, 420, 8, 2), (40, 2300, 8, 2)])
def test_rows_before_a_bad_block(d, new, total, hq, hk):
    step = R.Step(d + new, [new, 3], [total, 40], hq, hk, d, 32)
    check(step, (total - 2) // 16)                  # seen by the last row or the last few
    if new > 40:
        check(step, (total - new // 2) // 16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,total,window", [
    (1, 200, 20), (1, 200, 33), (3, 300, 17), (8, 1000, 100), (40, 300, 50), (200, 700, 130), (40, 3000, 2500), (17, 257, 129)])
def test_rows_whose_window_has_left_a_bad_block(d, new, total, window):
    step = R.Step(d + new + window, [new, 1], [total, 9], 8, 2, d, 16)
    first_seen = max(0, total - new + 1 - window)   # by the first row
    if new > 1:
        check(step, first_seen // 16, window)       # seen by the first rows
    if first_seen >= 16:
        check(step, first_seen // 16 - 1, window)   # by none, in the 64 tokens that a tile starts with
    if first_seen >= 48:
        check(step, first_seen // 16 - 3, window)
