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


def test_pages_held_elsewhere_move_to_their_rank():
    """A page counted once more for its holder becomes the page of its rank among those in use."""
    import trellis_quantized_weight_gb300 as tq
    cache, into = tq.kv_cache(12, 2, 16, 64), tq.kv_cache(9, 2, 16, 64)
    for t in cache:
        t.view(torch.uint8)[:] = torch.randint(0, 256, t.view(torch.uint8).shape, device="cuda", dtype=torch.uint8)
    refs = ints([0, 3, 0, 0, 1, 1, 0, 0, 2, 0, 1, 0])
    held = torch.tensor([1, 5, 8, 10], device="cuda")                  # by no sequence, or by one more than their sequences
    refs2, lens2, table2 = tq.kv_compact(cache, refs, ints([40, 17]), ints([[1, 4, 8], [1, 8, 0]]), into)
    rank = (refs > 0).cumsum(0) - 1
    assert lens2.tolist() == [40, 17] and table2.tolist() == [[0, 1, 3], [0, 3, 0]]
    assert torch.equal(refs2[rank[held]], refs[held])
    for a, b in zip(cache, into):
        assert torch.equal(b.view(torch.uint8)[rank[held]], a.view(torch.uint8)[held])
