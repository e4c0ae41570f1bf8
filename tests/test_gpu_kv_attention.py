"""trellis_kv_attention against a plain 64-bit implementation on a GB300.

Tolerance, element by element: 2^-8 |ref| + 2^-10 size, size = sum p |v| / sum p.  The output's
rounding to bf16 is at most 2^-9 |ref|; a weight p is held in f16 against the fp32 denominators,
2^-11 of itself; score errors (fp32 sums of 64 to 256 products, fp32 exponents below 2^7) change
p by less than 2^-15 of itself; weights below 2^-14 of the largest lose at most 2^-25 of it each,
under 2^-12 for the few thousand tokens here.  Together below 2^-9 |ref| + 2^-10.4 size.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu


def check(step, window=0, scale=None, q=None, cache=None, max_q=None, sharp=1.0, **kw):
    import trellis_quantized_weight_gb300 as tq
    if q is None:
        q = (step.randn(step.tokens, step.hq, step.d) * sharp).bfloat16().to(step.dev)
    if cache is None:
        cache = step.cache()
    got = tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, scale=scale, window=window,
                          max_q=max(step.new) if max_q is None else max_q, **kw)
    ref, size = R.attention(step, q, cache, scale if scale is not None else step.d ** -0.5, window)
    err = (got.double() - ref).abs()
    tol = ref.abs() * 2.0 ** -8 + size * 2.0 ** -10
    bad = err > tol
    assert not torch.isnan(got).any()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((err / tol.clamp(min=1e-30)).max())}"
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens_of_ragged_lengths(d, page):
    lens = [1, 2, 15, 16, 17, 31, 127, 128, 129, 300, 1111]
    check(R.Step(d + page, [1] * len(lens), lens, 8, 2, d, page))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16, 24])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_head_groups(group, d):
    check(R.Step(group, [1, 1, 1], [40, 513, 129], 2 * group, 2, d, 32))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [2, 5, 8, 17])
def test_drafts_see_only_what_is_before_them(d, new):
    check(R.Step(new, [new, new, new], [new, new + 1, 260], 8, 4, d, 16))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_packed(d):
    check(R.Step(3, [70, 1, 0, 33, 129], [70, 200, 50, 33, 400], 6, 2, d, 64))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_window(window, new):
    check(R.Step(window + new, [new] * 4, [new, 77 + new, 300, 1025], 8, 2, 128, 32), window=window)


def test_rows_without_tokens_are_zero():
    step = R.Step(5, [1, 1, 3, 0, 1], [0, 20, 0, 9, 33], 8, 2, 128, 16)
    got = check(step)
    assert (got[0] == 0).all() and (got[2:5] == 0).all()
    # more rows than tokens: the first ones stand before position 0
    step = R.Step(6, [5, 1], [2, 33], 8, 2, 128, 16)
    assert (check(step)[:3] == 0).all()
    # nothing at all
    step = R.Step(7, [1, 2], [0, 0], 8, 2, 128, 16)
    assert (check(step) == 0).all()


def test_no_rows():
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(7, [0, 0], [3, 40], 8, 2, 128, 16)
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert tq.kv_attention(q, step.cache(), step.starts, step.kv_len, step.pages).shape == (0, 8, 128)


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("sharp", [0.0, 0.1, 8.0, 60.0])
def test_flat_and_sharp_rows(sharp, new):
    check(R.Step(11, [new, new], [700, 90], 8, 2, 128, 64), sharp=sharp)


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** 60])
def test_extreme_queries_and_scales(factor, new):
    """A query row times a power of two and the score factor over it give the same result."""
    step = R.Step(12, [new, new], [333, 64], 8, 2, 128, 16)
    q = step.randn(step.tokens, 8, 128).bfloat16().to(step.dev)
    check(step, q=q * factor, scale=step.d ** -0.5 / factor)


@pytest.mark.parametrize("new", [1, 50])
def test_value_scales_far_apart(new):
    step = R.Step(13, [new, new], [200, 517], 8, 2, 128, 16)
    cache = step.cache()
    e = torch.randint(-30, 30, cache[3].shape, generator=step.gen).float().to(step.dev)
    cache[3] = torch.where(torch.isnan(cache[3]), cache[3], torch.exp2(e))
    # one block as zero values leave it
    page = int(step.table[1, 3])
    cache[1].view(torch.uint8)[page] = 0
    cache[3][page] = 2.0 ** -60
    check(step, cache=cache)


@pytest.mark.parametrize("new", [1, 50])
def test_a_poisoned_block_reaches_the_rows_that_see_it(new):
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(14, [new, new], [200, 100], 4, 2, 128, 16)
    cache = step.cache()
    q = step.randn(step.tokens, 4, 128).bfloat16().to(step.dev)
    for which in (2, 3):
        bad = [t.clone() for t in cache]
        bad[which][int(step.table[0, 2]), 1] = math.nan       # tokens 32 .. 47 of sequence 0, key head 1
        got = tq.kv_attention(q, bad, step.starts, step.kv_len, step.pages, max_q=new)
        ref = tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=new)
        assert torch.isnan(got[:new, 2:]).all()
        assert torch.equal(got[:new, :2], ref[:new, :2]) and torch.equal(got[new:], ref[new:])


@pytest.mark.parametrize("new", [1, 60])
def test_strided_queries_and_given_output(new):
    step = R.Step(15, [new, new, new], [new, 200, 65], 8, 2, 64, 32)
    wide = step.randn(step.tokens, 12 * 64).bfloat16().to(step.dev)
    out = torch.full((step.tokens, 8, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    got = check(step, q=wide[:, 64:9 * 64].unflatten(1, (8, 64)), out=out)
    assert got.data_ptr() == out.data_ptr()


@pytest.mark.parametrize("new", [1, 4, 60])
def test_the_hint_changes_nothing_but_time(new):
    step = R.Step(16, [new, 1, new], [new, 200, 650], 8, 2, 128, 32)
    for hint in (1, 3, new, 10 * new + 1000):
        check(step, max_q=hint)


@pytest.mark.parametrize("new,lens", [(1, [20000, 3, 9000]), (1, [31, 60000]), (100, [3000, 101]), (700, [700])])
def test_equal_calls_give_equal_bits(new, lens):
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(17, [new] * len(lens), lens, 8, 2, 128, 64)
    cache = step.cache()
    q = step.randn(step.tokens, 8, 128).bfloat16().to(step.dev)
    first = tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=new)
    for _ in range(5):
        assert torch.equal(tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=new), first)


def test_long_sequence():
    check(R.Step(18, [1, 1], [33333, 1], 8, 2, 128, 64))


def test_many_sequences():
    lens = [(i * 37) % 150 for i in range(700)]
    check(R.Step(19, [1] * 700, lens, 4, 1, 64, 16))


@pytest.mark.parametrize("new", [1, 30])
def test_offsets_past_32_bits(new):
    """Pages near the end of a cache of more than 4 GiB of codes."""
    step = R.Step(20, [new, new], [300, 90], 8, 8, 128, 128)
    cache = step.cache()
    big = 34000
    at = big - step.num_pages
    wide = []
    for t in cache:
        w = torch.zeros((big,) + tuple(t.shape[1:]), dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype,
                        device="cuda")
        w[at:] = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        wide.append(w.view(torch.float8_e4m3fn) if t.dtype == torch.float8_e4m3fn else w)
    assert wide[0].numel() > 2 ** 32
    used = step.table < step.num_pages
    step.table = torch.where(used, step.table + at, step.table)
    step.pages = step.table.to(step.dev)
    check(step, cache=wide)


def test_on_another_stream():
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(21, [1, 1, 1], [5000, 800, 3], 8, 2, 128, 32)
    cache = step.cache()
    q = step.randn(3, 8, 128).bfloat16().to(step.dev)
    want = tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=1, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_in_a_graph():
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(22, [1, 1], [700, 90], 8, 2, 128, 32)
    cache = step.cache()
    q = step.randn(2, 8, 128).bfloat16().to(step.dev)
    out = torch.empty_like(q)
    call = lambda: tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=1, out=out)  # noqa: E731
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    q2 = step.randn(2, 8, 128).bfloat16().to(step.dev)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    assert torch.equal(got, tq.kv_attention(q2, cache, step.starts, step.kv_len, step.pages, max_q=1))
