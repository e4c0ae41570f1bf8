"""trellis_kv_grow, trellis_kv_fork and trellis_kv_compact against plain Python on a GB300: everything is equal."""
import random

import pytest

import pages_reference as plain

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def ints(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


class Pool:
    """A cache with sequences of these lengths; some pairs share whole pages, some free pages are held by others."""

    def __init__(self, lens, page, cols, spare, seed=0, heads=2, dim=64, share=False, held=0):
        import trellis_quantized_weight_gb300 as tq
        rng = random.Random(seed)
        self.page, self.lens = page, list(lens)
        need = [plain.pages_of(n, page) for n in lens]
        ids = list(range(sum(need) + spare))
        rng.shuffle(ids)
        self.pages = len(ids)
        self.refs, self.table = [0] * len(ids), []
        for s, n in enumerate(need):
            row = [ids.pop() for _ in range(n)]
            if share and s % 2:
                whole = min(self.lens[s], self.lens[s - 1]) // page
                back, row[:whole] = row[:whole], self.table[s - 1][:whole]
                ids += back
            for p in row:
                self.refs[p] += 1
            self.table.append(row + [rng.randrange(len(self.refs)) for _ in range(cols - n)])
        for p in ids[:held]:
            self.refs[p] += 1
        g = torch.Generator(device="cuda").manual_seed(seed)
        codes = [torch.randint(0, 256, (self.pages, heads, page, dim), generator=g, device="cuda", dtype=torch.uint8)
                 .view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.exp2(torch.randint(-9, 3, (self.pages, heads, page // 16), generator=g, device="cuda").float()) for _ in range(2)]
        self.cache = tq.KVCache(*codes, *scales)
        self.d_refs, self.d_lens, self.d_table = ints(self.refs), ints(self.lens), ints(self.table, (len(lens), cols))

    def arrays(self):
        return self.cache, self.d_refs, self.d_lens, self.d_table

    def check(self, refs, lens, table):
        assert self.d_refs.tolist() == refs
        assert self.d_lens.tolist() == lens
        assert self.d_table.tolist() == table
        self.refs, self.lens, self.table = refs, lens, table

    def grow(self, counts):
        import trellis_quantized_weight_gb300 as tq
        ok, *want = plain.grow(self.refs, self.lens, self.table, counts, self.page)
        got = tq.kv_grow(*self.arrays(), ints(counts))
        assert got.tolist() == ok
        self.check(*want)
        return ok

    def fork(self, parents):
        import trellis_quantized_weight_gb300 as tq
        ok, *want, copies = plain.fork(self.refs, self.lens, self.table, parents, self.page)
        before = [raw(t).clone() for t in self.cache]
        got = tq.kv_fork(*self.arrays(), ints(parents))
        assert got.tolist() == ok
        self.check(*want)
        for a, b, tokens in copies:
            blocks = -(-tokens // 16)
            for t in before[:2]:
                t[b, :, :blocks * 16] = t[a, :, :blocks * 16]
            for t in before[2:]:
                t[b, :, :blocks] = t[a, :, :blocks]
        for t, want in zip(self.cache, before):
            assert torch.equal(raw(t), want)
        return ok


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def lengths(seqs, most, seed):
    rng = random.Random(seed)
    return [rng.choice([0, 1, 15, 16, 17, 64, 128, most, rng.randint(0, most)]) for _ in range(seqs)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seqs", [1, 2, 33, 1030])
def test_grow_and_cut(page, seqs):
    p = Pool(lengths(seqs, 300, seqs), page, 40, spare=20 * seqs, seed=page, held=5, share=True)
    rng = random.Random(seqs)
    for _ in range(4):
        p.grow([rng.choice([0, 0, 1, 1, 5, page, 100, -1, -3, -page, -1000, 30 * page]) for _ in range(seqs)])


@pytest.mark.parametrize("spare", [0, 1, 2, 7, 40])
def test_grow_with_too_few_pages(spare):
    p = Pool([10, 16, 0, 31, 5, 40], 16, 6, spare=spare)
    p.grow([7, 1, 40, 1, 80, 1])
    p.grow([-30, -30, -30, 2, -30, 1])
    p.grow([16, 16, 16, 16, 16, 16])


def test_grow_past_the_table_and_past_32_bits():
    p = Pool([10, 60, 3], 16, 4, spare=30)
    assert p.grow([54, 5, 2 ** 31 - 1]) == [True, False, False]
    assert p.grow([1, 4, -(2 ** 31)]) == [False, True, True]


def test_a_sequence_is_not_cut_inside_a_page_that_it_shares():
    p = Pool([70, 100], 32, 8, spare=4, share=True)              # two whole pages in common
    assert p.grow([-30, -36]) == [False, True]                   # to 40: inside the second; to 64: between pages
    assert p.grow([-6, 1]) == [True, True]
    assert p.grow([-64, -65]) == [True, True]
    assert p.refs.count(0) == p.pages


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (8, 256)])
def test_fork(page, heads, dim):
    p = Pool([200, 0, 0, 96, 17, 128, 0, 1], page, 16, spare=40, heads=heads, dim=dim)
    p.fork([0, 0, 0, 3, 3, 3, 7, 7])
    p.fork([1, 2, 0, 4, 5, 3, 6, 6])                             # turned around
    p.grow([5, 6, 7, 40, 41, 42, 1, 1])
    p.fork([2, 2, 2, -1, 4, -5, 99, 8])                          # dropped, ended, past the last
    p.fork([-1] * 8)
    assert p.refs == [0] * p.pages


def test_fork_keeps_a_last_page_with_its_own_sequence_first():
    p = Pool([20, 20, 0, 0], 16, 4, spare=9)
    last = p.table[1][1]
    p.fork([1, 1, 1, -1])                                        # sequence 1 itself
    assert p.table[1][1] == last
    p.fork([2, 3, 1, 1])                                         # 1 ends: sequence 2 takes its place
    assert p.table[2][1] == last


@pytest.mark.parametrize("spare", [0, 1, 2, 3])
def test_fork_with_too_few_pages(spare):
    p = Pool([40, 0, 0, 20, 0, 32, 0], 16, 4, spare=spare)
    p.fork([0, 0, 0, 3, 3, 5, 5])
    p.fork([0, 0, 0, 0, 0, 0, 0])


@pytest.mark.parametrize("seqs", [64, 1500])
def test_fork_many(seqs):
    p = Pool(lengths(seqs, 200, 3), 32, 12, spare=seqs, seed=2, share=True, held=11)
    rng = random.Random(5)
    for _ in range(3):
        p.fork([rng.choice([s, s, rng.randrange(seqs), rng.randrange(seqs // 8), -1]) for s in range(seqs)])
        p.grow([rng.choice([0, 1, 2, 33]) for _ in range(seqs)])


def test_fork_of_the_longest_batch():
    seqs = 16384
    p = Pool([3 if s == 77 else 0 for s in range(seqs)], 16, 1, spare=seqs)
    p.fork([77] * seqs)
    p.fork([s if s == 100 else -1 for s in range(seqs)])


@pytest.mark.parametrize("page,heads,dim", [(16, 1, 64), (32, 3, 128), (64, 8, 64), (128, 2, 256)])
@pytest.mark.parametrize("seqs", [1, 9, 70])
def test_compact(page, heads, dim, seqs):
    import trellis_quantized_weight_gb300 as tq
    p = Pool(lengths(seqs, 500, 8), page, 32, spare=30, heads=heads, dim=dim, share=True, held=7)
    used = sum(n > 0 for n in p.refs)
    for room in sorted({max(1, used), used + 5, max(1, used // 2), 1}):
        into = [torch.full_like(raw(t), 3).view(t.dtype) for t in tq.kv_cache(room, heads, page, dim)]
        refs, lens, table, pages = plain.compact(p.refs, p.lens, p.table, page, room)
        got = tq.kv_compact(*p.arrays(), into)
        assert [t.tolist() for t in got] == [refs, lens, table]
        for a, b in zip(p.cache, into):
            assert torch.equal(raw(b)[:len(pages)], raw(a)[torch.tensor(pages, dtype=torch.long).cuda()])
            assert torch.all(raw(b)[len(pages):] == 3)
    p.check(p.refs, p.lens, p.table)


def test_compact_of_a_large_pool():
    import trellis_quantized_weight_gb300 as tq
    n = 300_001
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = tq.kv_cache(n, 1, 16, 64)
    raw(cache.k)[:, 0, 0, :4] = torch.arange(n, device="cuda", dtype=torch.int32).view(torch.uint8).view(n, 4)
    refs = (torch.rand(n, generator=g, device="cuda") < 0.3).int()
    used = refs.nonzero()[:, 0]
    table = used[torch.randperm(used.numel(), generator=g, device="cuda")].int()[None].contiguous()
    lens = ints([used.numel() * 16])
    into = tq.kv_cache(used.numel(), 1, 16, 64)
    out = tq.kv_compact(cache, refs, lens, table, into)
    assert torch.equal(raw(into.k)[:, 0, 0, :4].contiguous().view(torch.int32)[:, 0].long(), used)
    assert torch.equal(used[out[2][0].long()].int(), table[0]) and torch.all(out[0] == 1) and torch.equal(out[1], lens)


def test_grow_in_a_large_pool():
    n = 200_000
    import trellis_quantized_weight_gb300 as tq
    cache = tq.kv_cache(n, 1, 16, 64)
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    free = torch.randperm(n, device="cuda")[:70_000].sort().values
    refs[free] = 0
    lens, table = ints([0, 0, 0]), torch.zeros(3, 60_000, dtype=torch.int32, device="cuda")
    ok = tq.kv_grow(cache, refs, lens, table, ints([16 * 50_000, 16 * 30_000, 16 * 20_000]))
    assert ok.tolist() == [True, False, False] and lens.tolist() == [800_000, 0, 0]
    assert torch.equal(table[0, :50_000].long(), free[:50_000])
    ok = tq.kv_grow(cache, refs, lens, table, ints([0, 16 * 19_999 + 3, -1]))
    assert ok.tolist() == [True, True, True] and torch.equal(table[1, :20_000].long(), free[50_000:]) and refs.min() == 1


def test_entries_outside_the_pool_are_not_counted():
    import trellis_quantized_weight_gb300 as tq
    p = Pool([40, 10, 0, 0], 16, 4, spare=6)
    bad = p.d_table.clone()
    bad[0, 1], bad[0, 2], bad[1, 0] = 1 << 30, -7, 999
    refs = p.d_refs.clone()
    tq.kv_fork(p.cache, refs, p.d_lens.clone(), bad.clone(), ints([0, 0, 1, 1]))
    tq.kv_grow(p.cache, refs, p.d_lens.clone(), bad.clone(), ints([-40, -10, 0, 0]))
    into = tq.kv_cache(20, 2, 16, 64)
    out = tq.kv_compact(p.cache, p.d_refs, p.d_lens, bad, into)
    torch.cuda.synchronize()
    assert out[2].min() >= 0 and out[2].max() < 20


def test_captured_steps_and_another_stream():
    import trellis_quantized_weight_gb300 as tq
    p = Pool([20, 0, 0, 33], 16, 10, spare=30, seed=4)
    one, parents = ints([3, 0, 0, 5]), ints([0, 0, 3, 3])
    stream = torch.cuda.Stream(priority=-1)          # not of the pool whose streams other tests look into
    stream.wait_stream(torch.cuda.current_stream())
    p.grow([3, 0, 0, 5])
    p.fork([0, 0, 3, 3])
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            ok = tq.kv_grow(*p.arrays(), one)
            ok2 = tq.kv_fork(*p.arrays(), parents)
    for _ in range(3):
        a, *state = plain.grow(p.refs, p.lens, p.table, [3, 0, 0, 5], 16)
        b, *state, copies = plain.fork(*state, [0, 0, 3, 3], 16)
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        assert ok.tolist() == a and ok2.tolist() == b
        p.check(*state)
    got = tq.kv_grow(*p.arrays(), one, stream=stream)
    want, *state = plain.grow(p.refs, p.lens, p.table, [3, 0, 0, 5], 16)
    stream.synchronize()
    assert got.tolist() == want
    p.check(*state)


def test_no_sequences_and_refusals():
    import trellis_quantized_weight_gb300 as tq
    p = Pool([20, 5], 16, 4, spare=3)
    cache, refs, lens, table = p.arrays()
    assert tq.kv_grow(cache, refs, lens[:0], table[:0], ints([])).shape == (0,)
    assert tq.kv_fork(cache, refs, lens[:0], table[:0], ints([])).shape == (0,)
    two, other = ints([0, 1]), tq.kv_cache(5, 2, 32, 64)
    for bad in (lambda: tq.kv_grow(cache, refs[:-1], lens, table, two), lambda: tq.kv_grow(cache, refs, lens, table, two.long()),
                lambda: tq.kv_grow(cache, refs, lens, table, two[:1]), lambda: tq.kv_grow(cache, refs, lens[:1], table, two),
                lambda: tq.kv_grow(cache, refs, lens, table.T, two), lambda: tq.kv_grow(cache, refs.cpu(), lens, table, two),
                lambda: tq.kv_fork(cache, refs, lens, table, two.cpu()), lambda: tq.kv_fork(cache[:3] + (cache[2][:1],), refs, lens, table, two),
                lambda: tq.kv_compact(cache, refs, lens, table, other), lambda: tq.kv_compact(cache, refs, lens[:0], table[:0], cache)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tq.TrellisError):
        tq.kv_compact(cache, refs, lens, table, cache)
    with pytest.raises(tq.TrellisError):
        tq.kv_compact(cache, refs, lens, table, tuple(t[1:] for t in cache))
    with pytest.raises(tq.TrellisError):
        tq.kv_grow(cache, refs, lens, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), two)


def test_growth_looks_at_the_shape_of_the_keys():
    import trellis_quantized_weight_gb300 as tq
    p = Pool([20, 5], 16, 4, spare=3)
    cache, refs, lens, table = p.arrays()
    two = ints([0, 1])
    for bad in (cache[2], cache[0][0], cache[0].cpu(), cache[0].view(torch.uint8), cache[0][:, :, ::2], None):
        with pytest.raises(ValueError):
            tq.kv_grow((bad,) + tuple(cache[1:]), refs, lens, table, two)
    with pytest.raises(ValueError):
        tq.kv_grow((cache[0][1:],) + tuple(cache[1:]), refs, lens, table, two)
