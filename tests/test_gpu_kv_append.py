"""trellis_kv_append and trellis_rope_table against plain 64-bit implementations on a GB300.

Tolerances: a rotated value is two fp32 products and a sum, so within 2^-22 (|a| + |b|) of the
exact one; queries add one bf16 rounding (2^-9).  A stored value is the e4m3 nearest to x / s: within
2^-4 of itself, or 2^-10 s where e4m3 is subnormal; a block's earlier values round once more when
its scale grows, exactly unless they are subnormal then (2^-10 s each time).
"""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu


def table(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    a = torch.arange(rows).double()[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def run(step, rot=None, interleaved=False, with_q=True, cache=None, spread=3.0, max_q=None, shrink=1.0):
    """One append checked against the plain form; returns the cache."""
    import trellis_quantized_weight_gb300 as tq
    d, hk, hq = step.d, step.hk, step.hq
    x = (step.randn(step.tokens, (hq + 2 * hk) * d) * torch.exp(spread * step.randn(step.tokens, 1)) * shrink).bfloat16()
    q, k, v = (x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
               x[:, (hq + hk) * d:].unflatten(1, (hk, d)))
    xd = x.to(step.dev)
    dq, dk, dv = (xd[:, :hq * d].unflatten(1, (hq, d)), xd[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                  xd[:, (hq + hk) * d:].unflatten(1, (hk, d)))
    if cache is None:
        cache = step.cache()
    before = [t.cpu().clone() for t in cache]
    tab = table(max(step.total) + 1, rot) if rot else None
    got = tq.kv_append(cache, dk, dv, step.starts, step.kv_len, step.pages, q=dq if with_q else None,
                       rope=tab.to(step.dev) if rot else None, interleaved=interleaved,
                       max_q=max(step.new) if max_q is None else max_q)
    after = [t.cpu() for t in cache]
    touched = torch.zeros(step.num_pages, step.page, dtype=torch.bool)
    for i, (n, t) in enumerate(zip(step.new, step.total)):
        for r in range(n):
            pos = t - n + r
            row = step.start[i] + r
            if with_q:
                want = R.rotate(q[row].double(), pos, tab, rot, interleaved)
                err = (got[row].cpu().double() - want).abs()
                assert (err <= want.abs() * 2.0 ** -8 + q[row].double().abs().amax() * 2.0 ** -20).all()
        if t <= 0 or n == 0:
            continue
        p0 = max(0, t - n)
        for b in range(p0 // 16 * 16, t, 16):
            ph, off = int(step.table[i, b // step.page]), b % step.page
            lo, hi = max(p0, b), min(t, b + 16)
            touched[ph, off:off + hi - b] = True
            rows = slice(step.start[i] + lo - (t - n), step.start[i] + hi - (t - n))
            for which, src in ((0, k), (1, v)):
                val = src[rows].double()
                if which == 0 and rot:
                    val = torch.stack([R.rotate(val[j], lo + j, tab, rot, interleaved) for j in range(hi - lo)])
                for h in range(hk):
                    most = float(val[:, h].abs().max())
                    had = float(before[2 + which][ph, h, off // 16]) if lo > b else 0.0
                    s = float(after[2 + which][ph, h, off // 16])
                    near = abs(most / (448.0 * R.power(most)) - 1.0) < 1e-6 or abs(most / (224.0 * R.power(most)) - 1.0) < 1e-6
                    assert s == max(had, R.power(most)) or near
                    new = after[which][ph, h, off + lo - b:off + hi - b].double() * s
                    assert ((new - val[:, h]).abs() <= val[:, h].abs() * (2.0 ** -4 + 1e-6) + s * 2.0 ** -10 + most * 1e-6).all()
                    if lo > b:
                        old = before[which][ph, h, off:off + lo - b].double() * had
                        again = after[which][ph, h, off:off + lo - b].double() * s
                        assert ((old - again).abs() <= (s * 2.0 ** -10 if s > had else 0.0)).all()
    # nothing else changed
    for which in (0, 1):
        a, b = before[which].view(torch.uint8), after[which].view(torch.uint8)
        same = (a == b).all(-1).transpose(1, 2)                 # [pages, page, heads]
        assert same[~touched].all()
    return cache


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_single_tokens(d, page, interleaved):
    run(R.Step(d + page, [1] * 9, [1, 2, 15, 16, 17, 32, 33, 64, 129], 6, 2, d, page), rot=d, interleaved=interleaved)


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(rot, interleaved):
    run(R.Step(rot, [3, 20], [9, 41], 3, 1, 128, 32), rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts(d):
    run(R.Step(d, [1, 16, 0, 17, 70, 33], [1, 16, 5, 40, 75, 33], 4, 2, d, 32), rot=d)


def test_without_rotation_and_without_queries():
    run(R.Step(1, [5, 1], [20, 9], 4, 2, 128, 16))
    run(R.Step(2, [5, 1], [20, 9], 4, 2, 128, 16), rot=64, with_q=False)


def test_idle_slots_and_rows_before_position_zero():
    run(R.Step(3, [1, 3, 0, 1], [0, 1, 7, 18], 4, 2, 128, 16), rot=128)


@pytest.mark.parametrize("hint", [1, 2, 100000])
def test_the_hint_changes_nothing_but_time(hint):
    run(R.Step(4, [70, 1, 20], [90, 4, 20], 4, 2, 64, 32), rot=64, max_q=hint)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (7, 1), (40, 8)])
def test_head_counts(hq, hk):
    run(R.Step(5, [2, 1], [20, 9], hq, hk, 64, 16), rot=32)


@pytest.mark.parametrize("shrink", [2.0 ** -70, 2.0 ** -55, 0.0, 2.0 ** 40])
def test_tiny_zero_and_large_values(shrink):
    run(R.Step(6, [2, 20], [20, 20], 4, 2, 64, 16), rot=64, shrink=shrink)


def test_token_by_token_equals_at_once():
    """With scales that are powers of two, growing blocks lose nothing but subnormals."""
    import trellis_quantized_weight_gb300 as tq
    d, hk, page, n = 128, 2, 32, 50
    x = (torch.randn(n, 2 * hk, d, generator=torch.Generator().manual_seed(1)) *
         torch.exp(torch.randn(n, 1, 1, generator=torch.Generator().manual_seed(2)))).bfloat16().cuda()
    rope = tq.rope_table(n, d)
    made = []
    for steps in ([n], [1] * n, [7] * 7 + [1]):
        cache = tq.kv_cache(2, hk, page, d)
        pages = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
        at = 0
        for m in steps:
            tq.kv_append(cache, x[at:at + m, :hk], x[at:at + m, hk:], torch.tensor([0, m], dtype=torch.int32, device="cuda"),
                         torch.tensor([at + m], dtype=torch.int32, device="cuda"), pages, rope=rope, max_q=m)
            at += m
        made.append([t.clone() for t in cache])
    used = (slice(None), slice(None))
    for other in made[1:]:
        for s in (2, 3):
            assert torch.equal(made[0][s].flatten()[:], other[s].flatten())
        for c, s in ((0, 2), (1, 3)):
            sc = made[0][s].double().repeat_interleave(16, -1)[..., None]
            a, b = made[0][c][used].double() * sc, other[c].double() * sc
            big = a.abs() >= sc * 2.0 ** -6                     # normal in e4m3 at the block's last scale
            assert torch.equal(a[big], b[big])
            assert ((a - b).abs() <= sc * 2.0 ** -9).all()


def test_going_back_drops_drafted_tokens():
    step = R.Step(8, [4], [40], 4, 2, 64, 16)
    cache = run(step, rot=64)
    back = R.Step(8, [2], [38], 4, 2, 64, 16, spare=step.num_pages - 3)
    back.table, back.pages, back.num_pages = step.table, step.pages, step.num_pages
    run(back, rot=64, cache=cache)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_bad_value_poisons_its_block_only(bad):
    import trellis_quantized_weight_gb300 as tq
    cache = tq.kv_cache(3, 2, 16, 64)
    k = torch.randn(40, 2, 64, device="cuda").bfloat16()
    v = torch.randn(40, 2, 64, device="cuda").bfloat16()
    k[20, 1, 3] = bad
    v[39, 0, 0] = bad
    i32 = dict(dtype=torch.int32, device="cuda")
    tq.kv_append(cache, k, v, torch.tensor([0, 40], **i32), torch.tensor([40], **i32), torch.tensor([[0, 1, 2]], **i32))
    assert torch.isnan(cache.k_scale).flatten().nonzero().flatten().tolist() == [3]
    assert torch.isnan(cache.v_scale).flatten().nonzero().flatten().tolist() == [4]


def test_offsets_past_32_bits():
    import trellis_quantized_weight_gb300 as tq
    big = 34000
    cache = tq.kv_cache(big, 8, 128, 128)
    assert cache.k.numel() > 2 ** 32
    k = torch.randn(20, 8, 128, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    tq.kv_append(cache, k, k, torch.tensor([0, 20], **i32), torch.tensor([20], **i32),
                 torch.tensor([[big - 1]], **i32))
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert not codes[:1000].view(torch.uint8).any() and not codes[big - 2].view(torch.uint8).any()
        got = codes[big - 1, :, :20].double() * scale[big - 1, :, :2].double().repeat_interleave(16, -1)[:, :20, None]
        want = k.transpose(0, 1).double()
        assert ((got - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -16).all()


def test_on_another_stream_then_attention():
    """Append and attention in order on a stream of their own."""
    import trellis_quantized_weight_gb300 as tq
    step = R.Step(9, [1, 1], [500, 90], 8, 2, 128, 32)
    cache = step.cache()
    k, v, q = (step.randn(2, h, 128).bfloat16().to(step.dev) for h in (2, 2, 8))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            tq.kv_append(cache, k, v, step.starts, step.kv_len, step.pages, max_q=1)
            got = tq.kv_attention(q, cache, step.starts, step.kv_len, step.pages, max_q=1)
    s.synchronize()
    ref, size = R.attention(step, q, cache, 128 ** -0.5)
    assert ((got.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * 2.0 ** -10).all()


# ---- the table -------------------------------------------------------------------------------
@pytest.mark.parametrize("rows,rot,base,stretch,original", [
    (1, 16, 10000.0, 1.0, 0), (777, 64, 10000.0, 1.0, 0), (300, 128, 1e6, 4.0, 0), (5000, 128, 5e5, 8.0, 512),
    (200000, 32, 10000.0, 2.5, 4096)])
def test_rope_table(rows, rot, base, stretch, original):
    """Within one fp32 rounding of the 64-bit formula (and 2^-40 for its angle)."""
    import trellis_quantized_weight_gb300 as tq
    got = tq.rope_table(rows, rot, base, stretch, original, low=1.0, high=4.0, gain=1.25).cpu().double()
    i = torch.arange(rot // 2).double()
    f = base ** (-2.0 * i / rot)
    slow = torch.full_like(f, 1.0 / stretch)
    if original:
        turns = original * f / (2.0 * math.pi)
        w = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
        slow = w + (1.0 - w) / stretch
    a = torch.arange(rows).double()[:, None] * (f * slow)
    want = 1.25 * torch.cat([a.cos(), a.sin()], 1)
    assert ((got - want).abs() <= want.abs() * 2.0 ** -24 + 2.0 ** -30).all()
