"""Operators of a decoding step around the cache and the packed projections, as cases to measure and compare.

Three that touch the pages of the 8-bit cache, so that a program need not wait for the host to hand them out, and two
that carry a row from one projection to the next:

  grow      the pages that a step's new tokens need are taken from the pool, or those of dropped tokens given back
  fork      sequences go on as continuations of others (samples of one prompt, reordered beams, ended requests): whole
            pages are shared, a last page that is not full is copied
  compact   the pages in use go to another cache, close together, and the table with them
  norm      the residual's addition and the root-mean-square norm, to bf16 or to 8 bits with a scale a row
  product   x W^T with 4-bit weights in groups, x in bf16 or as norm leaves it in 8 bits

The cache is the one of the append and attention operators: codes float8_e4m3fn [pages, kv_heads, page_size, head_dim],
scales float32 [pages, kv_heads, page_size / 16], twice; `table` int32 [S, columns] holds the pages of a sequence's tokens
0 .. len - 1.  `refs` int32 [pages] counts the places of the table that name a page: 0 is free.  Pages are handed out
lowest first, to sequences in their order; one that a call gives back is free from the next call on.

The 4-bit weights: codes int32 [N, K / 8], eight a word, the lowest bits first; scales (and biases) bf16 [N, K / group].
A weight is scale * code + bias, or scale * (code - 8) without biases.

`own` false: the operators in elementary torch operations, in 32 bits; true: the package's calls.
"""
import math

import torch

own = False

BLOCK = 16          # tokens of a page that share a scale, per head
E4M3_MAX = 448.0
EPS = 1e-6
LEAST = 2.0 ** -100  # of a row's scale


# ---- the cases --------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one user's drafted tokens get their pages and, all refused, give them back: latency alone
        dict(name="grow 1 draft", op="grow", seqs=1, new_lo=5, new_hi=5, past_lo=781, past_hi=781, page=16),
        # a batch of prompts is admitted and, answered, ends: pools of a long-running server
        dict(name="grow 64 prompts", op="grow", seqs=64, new_lo=130, new_hi=16384, past_lo=0, past_hi=0, page=32),
        # one prompt, eight answers sampled from it
        dict(name="fork 1 x 8", op="fork", kind="samples", groups=1, wide=8, len_lo=777, len_hi=777, kv_heads=8, dim=128,
             page=64, spare=64),
        # beam search: 24 requests of four beams, each step keeps some and drops some
        dict(name="fork 24 x 4 beams", op="fork", kind="beams", groups=24, wide=4, len_lo=300, len_hi=9000, kv_heads=8,
             dim=128, page=128, spare=300),
        # a handful of short conversations moves to a cache of its own
        dict(name="compact short", op="compact", groups=8, wide=1, len_lo=40, len_hi=777, kv_heads=8, dim=128, page=16, spare=500),
        # a full server's cache, with prefixes shared by two answers each, pulled together
        dict(name="compact ragged", op="compact", groups=32, wide=2, len_lo=1000, len_hi=16384, kv_heads=8, dim=128, page=64,
             spare=5000),
        # one user's next token
        dict(name="norm 1 row", op="norm", rows=1, width=5120, heads=0, resid=True, eight=False),
        # packed prompts, to 8 bits for the product that follows
        dict(name="norm prompts 8k", op="norm", rows=8165, width=5120, heads=0, resid=True, eight=True),
        # one user's next token through an up projection
        dict(name="product 1 row", op="product", m=1, k=5120, n=17408, group=64, affine=True, eight=False),
        # a small batch through a down projection, activations in 8 bits
        dict(name="product 11 rows", op="product", m=11, k=17408, n=5120, group=128, affine=False, eight=True),
        # a larger batch of single tokens
        dict(name="product 64 rows", op="product", m=64, k=5120, n=17408, group=32, affine=True, eight=False),
        # packed prompts
        dict(name="product prompts 2k", op="product", m=1999, k=5120, n=17408, group=128, affine=False, eight=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grow", "fork", "compact", "norm", "norm", "product", "product", "product"])
    if op == "product":
        group = rng.choice([32, 64, 128])
        c = dict(op=op, k=group * _log(rng, 1, 17408 // group), n=_log(rng, 1, 17408), group=group, affine=rng.random() < 0.5,
                 eight=rng.random() < 0.5)
        c["m"] = rng.choice([_log(rng, 1, 16), _log(rng, 1, max(1, min(2048, 1999 * 5120 * 17408 // (c["k"] * c["n"]))))])
        return c
    if op == "norm":
        heads = rng.choice([0, 0, 0, 8, 40])
        width = rng.choice([64, 128, 256]) if heads else rng.choice([8 * _log(rng, 1, 2176), _log(rng, 1, 17408)])
        most = max(1, min(8165, 8165 * 5120 // (width * max(1, heads))))
        return dict(op=op, rows=_log(rng, 1, most), width=width, heads=heads, resid=not heads and rng.random() < 0.7,
                    eight=not heads and rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "grow":
        seqs = _log(rng, 1, 512)
        c = dict(op=op, seqs=seqs, new_hi=_log(rng, 1, max(1, min(16384, 524288 // seqs))),
                 past_hi=_log(rng, 1, max(1, min(16384, 524288 // seqs))), page=page)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["past_lo"] = rng.randint(0, c["past_hi"])
        return c
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    c = dict(op=op, groups=_log(rng, 1, 32), wide=rng.choice([1, 2, 3, 4, 8]), kv_heads=kv_heads, dim=dim, page=page)
    room = 32 * 8192 * 8 * 128 // (c["groups"] * kv_heads * dim)
    if op == "fork":
        c["kind"] = rng.choice(["samples", "beams"])
        room = min(room, 9000)
        c["spare"] = _log(rng, 1, 512)              # now and then too few for every copy
    else:
        c["spare"] = _log(rng, 1, 5000 * 64 // page)
    c["len_hi"] = _log(rng, 16, max(17, min(16384, room // (1 if op == "fork" else c["wide"]))))
    c["len_lo"] = rng.randint(1, c["len_hi"])
    return c


def _spread(count, lo, hi):
    """`count` whole numbers from lo to hi, spread evenly and out of order."""
    return [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(count)]


def _grow_sizes(c):
    return _spread(c["seqs"], c["new_lo"], c["new_hi"]), _spread(c["seqs"] + 1, c["past_lo"], c["past_hi"])[1:]


def _groups(c):
    """Each group's shared prefix in whole pages, and the length of each of its sequences (0: an empty slot)."""
    shared, lens = [], []
    for i, n in enumerate(_spread(c["groups"], c["len_lo"], c["len_hi"])):
        if c.get("kind") == "samples":
            shared.append(0)
            lens.append([n] + [0] * (c["wide"] - 1))
        else:
            shared.append(n * 3 // 4 // c["page"] if c["wide"] > 1 else 0)
            # beams are of one length, other answers are not
            lens.append([n if c["op"] == "fork" else n - (j * 5 + i) % (1 + n // 8) for j in range(c["wide"])])
    return shared, lens


# ---- inputs -----------------------------------------------------------------------------------------------------------
def _codes(shape, gen, dev):
    """e4m3 codes, any but NaN."""
    return torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8).bitwise_and_(0xFB).view(torch.float8_e4m3fn)


def _cache(c, pages, gen, dev):
    shape = (pages, c["kv_heads"], c["page"], c["dim"])
    scales = [torch.exp2(torch.randint(-9, -5, shape[:2] + (c["page"] // BLOCK,), generator=gen, device=dev).float()) for _ in range(2)]
    return (_codes(shape, gen, dev), _codes(shape, gen, dev), *scales)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = case
    s = dict(case=c)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == "product":
        m, k, n, per = c["m"], c["k"], c["n"], c["k"] // c["group"]
        s["codes"] = torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=gen, device=dev, dtype=torch.int64).int()
        s["scales"] = ((torch.rand(n, per, generator=gen, device=dev) + 0.5) * (0.2 / k ** 0.5)).bfloat16()
        # the least value of a group is somewhat below 7.5 steps under its middle
        s["biases"] = (s["scales"].float() * -(6.5 + 2 * torch.rand(n, per, generator=gen, device=dev))).bfloat16() if c["affine"] else None
        x = normal(m, k)
        s["x_scales"] = None
        if c["eight"]:
            top = x.abs().amax(1, keepdim=True)
            x = (x * (E4M3_MAX / top)).to(torch.float8_e4m3fn)
            s["x_scales"] = (top[:, 0] / E4M3_MAX * (0.5 + torch.rand(m, generator=gen, device=dev))).contiguous()
        s["x"] = x if c["eight"] else x.bfloat16()
        return s
    if c["op"] == "norm":
        rows, width = c["rows"], c["width"]
        if c["heads"]:
            # the queries' heads of a projection to queries, keys and values
            s["x"] = normal(rows, (c["heads"] + 16) * width).bfloat16()[:, :c["heads"] * width].unflatten(1, (c["heads"], width))
        else:
            s["x"] = normal(rows, width).bfloat16()
        s["weight"] = (1.0 + 0.3 * normal(width)).bfloat16()
        s["residual"] = None
        if c["resid"]:
            h = normal(rows, width) * 4.0
            h[:, ::37] *= 12.0                                  # the stream's few large channels
            s["residual"] = h.bfloat16()
        return s
    if c["op"] == "grow":
        new, lens = _grow_sizes(c)
        need = [-(-t // c["page"]) for t in lens]
        more = [-(-(t + g) // c["page"]) for t, g in zip(lens, new)]
        spare = (sum(more) - sum(need)) * 3 // 2 + 8         # a third of it is held by others
        rows, width = need, max(more)
        s["grow"] = ints(new)
        s["back"] = -s["grow"]
    else:
        shared, by_group = _groups(c)
        lens = [n for g in by_group for n in g]
        rows, width, spare = [-(-t // c["page"]) for t in lens], max(-(-t // c["page"]) for t in lens), c["spare"]
    ids, at, first = [], 0, {}
    for i, need in enumerate(rows):
        row = []
        for j in range(need):
            g = i // c["wide"] if c["op"] != "grow" else i
            if c["op"] != "grow" and j < min(shared[g], lens[i] // c["page"]):
                p = first.get((g, j), at)
                first[g, j] = p
                at += p == at
            else:
                p, at = at, at + 1
            row.append(p)
        ids.append(row + [0] * (width - need))
    pages = at + spare
    order = torch.randperm(pages, generator=gen, device=dev).int()
    s["kv_len"] = ints(lens)
    used = torch.arange(width, device=dev)[None] < ints(rows)[:, None]
    s["table"] = torch.where(used, order[ints(ids).long()], 0).int().contiguous()
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev).index_add_(0, s["table"].flatten().long(), used.flatten().int())
    if c["op"] == "grow":
        s["refs"][order[at:at + spare // 3].long()] = 1
        s["cache"] = _cache(dict(c, kv_heads=1, dim=64), pages, gen, dev)
        return s
    s["cache"] = _cache(c, pages, gen, dev)
    if c["op"] == "compact":
        s["into"] = tuple(torch.zeros_like(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).view(t.dtype) for t in s["cache"])
        return s
    seqs = len(lens)
    slot = torch.arange(seqs, device=dev)
    lead = slot // c["wide"] * c["wide"]
    if c["kind"] == "samples":
        s["parents"] = lead.int()
    else:
        # each beam goes on from one of its request's; some requests end, all their beams
        pick = lead + torch.randint(0, c["wide"], (seqs,), generator=gen, device=dev)
        ends = (torch.rand(c["groups"], generator=gen, device=dev) < 0.1)[slot // c["wide"]]
        s["parents"] = torch.where(ends, -1, pick).int()
    return s


# ---- the operators ----------------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        import trellis_quantized_weight_gb300 as tq
        if c["op"] == "product":
            return tq.gemm_q4(s["x"], s["codes"], s["scales"], s["biases"], x_scales=s["x_scales"])
        if c["op"] == "norm":
            if c["eight"]:
                got = tq.rms_norm_q8(s["x"], s["weight"], EPS, residual=s["residual"])
                return dict(zip(("codes", "scales", "h"), got))
            got = tq.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
            return dict(zip(("y", "h"), got)) if c["resid"] else dict(y=got)
        if c["op"] == "grow":
            took = tq.kv_grow(s["cache"], s["refs"], s["kv_len"], s["table"], s["grow"])
            gave = tq.kv_grow(s["cache"], s["refs"], s["kv_len"], s["table"], s["back"])
            return dict(took=took, gave=gave, refs=s["refs"], kv_len=s["kv_len"], table=s["table"])
        if c["op"] == "fork":
            ok = tq.kv_fork(s["cache"], s["refs"], s["kv_len"], s["table"], s["parents"])
            return dict(ok=ok, refs=s["refs"], kv_len=s["kv_len"], table=s["table"], cache=s["cache"])
        refs, kv_len, table = tq.kv_compact(s["cache"], s["refs"], s["kv_len"], s["table"], s["into"])
        return dict(refs=refs, kv_len=kv_len, table=table, cache=s["into"])
    if c["op"] == "product":
        return _plain_product(s)
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "grow":
        took = _plain_grow(s, s["grow"])
        gave = _plain_grow(s, s["back"])
        return dict(took=took, gave=gave, refs=s["refs"], kv_len=s["kv_len"], table=s["table"])
    if c["op"] == "fork":
        return dict(ok=_plain_fork(s), refs=s["refs"], kv_len=s["kv_len"], table=s["table"], cache=s["cache"])
    return _plain_compact(s)


def _plain_product(s):
    codes, group = s["codes"], s["case"]["group"]
    shift = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    q = ((codes[..., None] >> shift) & 15).flatten(1).float().unflatten(1, (-1, group))
    scale = s["scales"].float()[..., None]
    w = scale * q + s["biases"].float()[..., None] if s["biases"] is not None else scale * (q - 8.0)
    y = s["x"].float() @ w.flatten(1).T
    return (y if s["x_scales"] is None else y * s["x_scales"][:, None]).bfloat16()


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {}
    if s["case"]["eight"]:
        top = y.abs().amax(-1, keepdim=True)
        scale = torch.where(torch.isfinite(top), (top / E4M3_MAX).clamp(min=LEAST), torch.nan)
        out["codes"] = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        out["scales"] = scale[:, 0]
    else:
        out["y"] = y.bfloat16()
    if s["residual"] is not None:
        out["h"] = h.bfloat16()
    return out


def _free_page(refs, rank):
    """The free pages of these ranks, lowest first (the pool's size where there are not so many)."""
    return torch.searchsorted((refs == 0).long().cumsum(0), rank + 1)


def _plain_grow(s, grow):
    refs, kv_len, table, page = s["refs"], s["kv_len"], s["table"], s["case"]["page"]
    old, g, cols = kv_len.long(), grow.long(), table.shape[1]
    new = (old + g).clamp(min=0)
    have, want = (old + page - 1) // page, (new + page - 1) // page
    left = (refs == 0).sum()
    need = torch.where((g > 0) & (want <= cols), want - have, 0)
    upto = need.cumsum(0)
    fits = (want <= cols) & ((need == 0) | (upto <= left))
    last = table.gather(1, (want - 1).clamp(0, cols - 1)[:, None])[:, 0].long()
    tied = (new % page != 0) & (refs[last] > 1)             # it would write to a page that it shares
    ok = torch.where(g > 0, fits, (g == 0) | ~tied)
    col = torch.arange(cols, device=refs.device)[None]
    take = (ok & (g > 0))[:, None] & (col >= have[:, None]) & (col < want[:, None])
    give = (ok & (g < 0))[:, None] & (col >= want[:, None]) & (col < have[:, None])
    fresh = _free_page(refs, ((upto - need - have)[:, None] + col).clamp(min=0)).clamp(max=refs.numel() - 1)
    gone = table.long()
    table.copy_(torch.where(take, fresh, gone))
    refs.index_add_(0, fresh.flatten(), take.flatten().int())
    refs.index_add_(0, gone.flatten(), -give.flatten().int())
    kv_len.copy_(torch.where(ok, new, old))
    return ok


def _plain_fork(s):
    refs, kv_len, table, page = s["refs"], s["kv_len"], s["table"], s["case"]["page"]
    parents, old, rows = s["parents"].long(), kv_len.long(), table.long()
    seqs, cols = table.shape
    slot = torch.arange(seqs, device=refs.device)
    valid = (parents >= 0) & (parents < seqs)
    src = torch.where(valid, parents, slot)
    new = torch.where(valid, old[src], 0)
    whole, part = new // page, new % page
    # the sequence itself, or the first that goes on from it, keeps the page in place
    first = torch.full((seqs,), seqs, device=refs.device).scatter_reduce_(0, src, torch.where(valid, slot, seqs), "amin")
    first = torch.where(parents == slot, slot, first)
    copy = valid & (part > 0) & (first[src] != slot)
    rank = copy.long().cumsum(0) - 1
    lost = copy & (rank >= (refs == 0).sum())
    got = copy & ~lost
    new = torch.where(lost, 0, new)
    fresh = _free_page(refs, rank.clamp(min=0))
    col = torch.arange(cols, device=refs.device)[None]
    had, has = (old + page - 1) // page, (new + page - 1) // page
    taken = rows[src]
    here = torch.where(got[:, None] & (col == whole[:, None]), fresh[:, None], taken)
    now = torch.where(col < has[:, None], here, rows)
    refs.index_add_(0, rows.flatten(), -(col < had[:, None]).flatten().int())
    refs.index_add_(0, now.clamp(max=refs.numel() - 1).flatten(), (col < has[:, None]).flatten().int())
    table.copy_(now)
    kv_len.copy_(new)
    who = got.nonzero()[:, 0]
    to, of, tokens = fresh[who], taken[who, whole[who]], part[who]
    used = torch.arange(0, page, BLOCK, device=refs.device)[None] < tokens[:, None]            # [copies, blocks]
    for t in s["cache"]:
        x = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        x = x.unflatten(2, (page // BLOCK, -1))                                                  # [pages, heads, blocks, ...]
        keep = used[:, None].view(-1, 1, used.shape[1], *[1] * (x.dim() - 3))
        x[to] = torch.where(keep, x[of], x[to])
    return (valid & ~lost) | (parents < 0)


def _plain_compact(s):
    refs, kv_len, table, page = s["refs"], s["kv_len"], s["table"], s["case"]["page"]
    room = s["into"][0].shape[0]
    used = refs > 0
    rank = used.long().cumsum(0) - 1
    ids = used.nonzero()[:, 0][:room]
    for t, u in zip(s["cache"], s["into"]):
        a, b = (t.view(torch.uint8), u.view(torch.uint8)) if t.dtype == torch.float8_e4m3fn else (t, u)
        b[:ids.numel()] = a[ids]
    col = torch.arange(table.shape[1], device=refs.device)[None]
    live = col < ((kv_len.long() + page - 1) // page)[:, None]
    to = rank[table.long()]
    kept = ~(live & (to >= room)).any(1)
    out = torch.zeros(room, dtype=torch.int32, device=refs.device)
    out[:ids.numel()] = refs[ids]
    drop = live & ~kept[:, None] & (to < room)
    out.index_add_(0, to.clamp(0, room - 1).flatten(), -drop.flatten().int())
    return dict(refs=out, kv_len=torch.where(kept, kv_len, 0), table=torch.where(live & kept[:, None], to, 0).int(), cache=s["into"])


# ---- what a pass cannot do without ------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "product":
        m, k, n, per = c["m"], c["k"], c["n"], c["k"] // c["group"]
        x = m * k + 4 * m if c["eight"] else 2 * m * k
        return dict(bytes=n * k // 2 + n * per * (4 if c["affine"] else 2) + x + 2 * m * n, flops=2 * m * k * n)
    if c["op"] == "norm":
        values = c["rows"] * c["width"] * max(1, c["heads"])
        per = 2 + (4 if c["resid"] else 0) + (1 if c["eight"] else 2)
        return dict(bytes=values * per + 2 * c["width"] + (4 * c["rows"] if c["eight"] else 0), flops=values * (5 + c["resid"]))
    if c["op"] == "grow":
        new, lens = _grow_sizes(c)
        took = sum(-(-(t + g) // c["page"]) - -(-t // c["page"]) for t, g in zip(lens, new))
        # both calls: lengths read and written, the change read, a flag; each page's count and its place in the table
        return dict(bytes=2 * c["seqs"] * 13 + took * (4 + 4 + 4 + 8), flops=2 * c["seqs"] + took)
    shared, by_group = _groups(c)
    token = 2 * c["kv_heads"] * c["dim"]
    block = BLOCK * token + 8 * c["kv_heads"]
    if c["op"] == "fork":
        # in earnest: all but one of a request's sequences copy the last page's used blocks; every sequence's row is read
        # and written, and its pages counted
        move = entries = 0
        for g in by_group:
            n = max(g)
            move += (c["wide"] - 1) * -(-(n % c["page"]) // BLOCK) * block
            entries += c["wide"] * -(-n // c["page"])
        copies = min(1.0, c["spare"] / max(1, c["groups"] * (c["wide"] - 1)))
        return dict(bytes=int(2 * move * copies) + entries * 16 + c["groups"] * c["wide"] * 13, flops=entries)
    pages = entries = 0
    for k, g in zip(shared, by_group):
        need = [-(-n // c["page"]) for n in g]
        alike = min(k, *[n // c["page"] for n in g]) if len(g) > 1 else 0
        pages += sum(need) - (len(g) - 1) * alike
        entries += sum(need)
    return dict(bytes=2 * pages * (c["page"] // BLOCK) * block + entries * 8 + (2 * pages + c["spare"]) * 4, flops=pages + entries)


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------------
def exact(case, seed):
    """Pages are copied and counted, not computed: they have no other value than the plain form's."""
    c = case
    if c["op"] not in ("product", "norm"):
        return None
    s = prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if c["resid"]:
            h = h + s["residual"].double()
        size = torch.linalg.vector_norm(h, dim=-1, keepdim=True)
        y = s["weight"].double() * h / torch.sqrt(size ** 2 / c["width"] + EPS)
        out = dict(y=y)
        if c["eight"]:
            scale = torch.maximum(torch.linalg.vector_norm(y, ord=math.inf, dim=-1) / 448, torch.full_like(y[:, 0], LEAST))
            out = dict(codes=y / scale[:, None], scales=scale)
        return dict(out, h=h) if c["resid"] else out
    low = torch.stack([(s["codes"].long() // 16 ** i) % 16 for i in range(8)], -1).double()       # floor division: the sign bit is bit 31
    low = low.view(c["n"], -1, c["group"])
    y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device=low.device)
    x = s["x"].double().view(c["m"], -1, c["group"])
    for g in range(low.shape[1]):
        part = x[:, g] @ (low[:, g].T if c["affine"] else low[:, g].T - 8)
        y += part * s["scales"][:, g].double()
        if c["affine"]:
            y += torch.outer(x[:, g].sum(1), s["biases"][:, g].double())
    return y * s["x_scales"].double()[:, None] if c["eight"] else y
