"""Compaction of tables that name what is not there, and of pages that something else holds, on a GB300."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [-1, -7, 12, 999, 1 << 30, 5])         # 5: a page of the pool that is free
@pytest.mark.parametrize("col", [0, 1, 2])
def test_a_sequence_that_names_no_page_of_the_pool_ends(bad, col):
    """Its entry became page 0 of the other cache, which is another sequence's: its appends went there, and giving it up
    counted that sequence's page down."""
    import trellis_quantized_weight_gb300 as tq
    cache, into = tq.kv_cache(12, 2, 16, 64), tq.kv_cache(12, 2, 16, 64)
    table = [[2, 7, 0, 0], [8, 9, 10, 0], [2, 11, 0, 0], [0, 0, 0, 0]]
    refs = [0, 0, 2, 0, 0, 0, 0, 1, 1, 1, 1, 1]
    table[1][col] = bad
    refs[8 + col] = 0
    refs2, lens2, table2 = tq.kv_compact(cache, ints(refs), ints([30, 40, 20, 0]), ints(table), into)
    assert lens2.tolist() == [30, 0, 20, 0]
    left = [p for p in range(12) if refs[p] > 0]
    assert table2.tolist() == [[left.index(2), left.index(7), 0, 0], [0] * 4, [left.index(2), left.index(11), 0, 0], [0] * 4]
    want = [refs[p] - (p in (8, 9, 10)) for p in left]
    assert refs2.tolist() == want + [0] * (12 - len(want))
    # all sequences give up what they have: nothing is left, and nothing is counted below that
    assert tq.kv_grow(into, refs2, lens2, table2, ints([-100] * 4)).all()
    assert refs2.tolist() == [0] * 12
