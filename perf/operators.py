"""Operators around the packed-weight projections of an attention block, as cases to measure and compare.

Three operators that a program calls between and beside the quantized projections when it serves a model:

  append   the step's keys and values go into a paged cache of 8-bit values, with the rotary rotation applied on the way
           (queries are rotated by the same call)
  attend   attention of the step's queries over that cache, from one token a sequence to whole prompt chunks
  adapt    the low-rank adapters of many requests, added to the output of a projection that they share

The cache.  keys and values: float8_e4m3fn [pages, kv_heads, page_size, head_dim]; scales: float32 [pages, kv_heads,
page_size / 16], a power of two for each block of 16 tokens of a page and head.  A stored value is code * scale.  Token t
of sequence s lies in page table[s, t // page_size], at t % page_size.  `starts` [S + 1] says which rows of the step's
packed tokens are sequence s's, `kv_len` [S] how many tokens it has with them, so that its last row is token kv_len - 1.
The scale of a block of values with largest magnitude a is the smallest power of two s >= 2^-100 with a <= 448 s; a block
that had tokens before keeps its scale unless the new tokens need a larger one, and then its old codes are rounded again.

`own` false: the operators in elementary torch operations, in 32 bits; true: the package's calls.
"""
import math

import torch

own = False

BLOCK = 16          # tokens of a page that share a scale, per head
E4M3_MAX = 448.0


# ---- the cases --------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: latency alone.  40 query heads of 128 are a hidden size of 5120
        dict(name="append 1 token", op="append", seqs=1, new_lo=1, new_hi=1, past_lo=1000, past_hi=1000, q_heads=40, kv_heads=8,
             dim=128, page=16, rot=128, inter=False, stretch=1.0),
        # a full serving batch, a token each; half of each head rotated, neighbouring pairs
        dict(name="append 128 tokens", op="append", seqs=128, new_lo=1, new_hi=1, past_lo=3, past_hi=500, q_heads=32, kv_heads=8,
             dim=128, page=32, rot=64, inter=True, stretch=1.0),
        # prompts of different lengths packed, positions stretched four times for a long context
        dict(name="append prompts 8k", op="append", seqs=5, new_lo=77, new_hi=3300, past_lo=0, past_hi=90, q_heads=32, kv_heads=8,
             dim=128, page=64, rot=128, inter=False, stretch=4.0),
        # one user's next token after a short conversation
        dict(name="attend 1 x 777", op="attend", seqs=1, new_lo=1, new_hi=1, len_lo=777, len_hi=777, idle=0, q_heads=40, kv_heads=8,
             dim=128, page=16, window=0),
        # one user's next token at the end of a very long document
        dict(name="attend 1 x 131k", op="attend", seqs=1, new_lo=1, new_hi=1, len_lo=131071, len_hi=131071, idle=0, q_heads=32,
             kv_heads=8, dim=128, page=64, window=0),
        # a full serving batch of very different lengths, some slots of it idle
        dict(name="attend 64 x ragged", op="attend", seqs=64, new_lo=1, new_hi=1, len_lo=1, len_hi=16384, idle=3, q_heads=64,
             kv_heads=8, dim=128, page=64, window=0),
        # five drafted tokens a sequence, checked at once; wide heads
        dict(name="attend 16 x 5 drafts", op="attend", seqs=16, new_lo=5, new_hi=5, len_lo=300, len_hi=9000, idle=0, q_heads=32,
             kv_heads=4, dim=256, page=32, window=0),
        # chunks of long prompts on top of what is cached already
        dict(name="attend 4 x 2k chunk", op="attend", seqs=4, new_lo=2048, new_hi=2048, len_lo=4100, len_hi=9001, idle=0, q_heads=32,
             kv_heads=8, dim=128, page=64, window=0),
        # whole prompts, packed, each token seeing the last 1024; narrow heads
        dict(name="attend prompts window", op="attend", seqs=6, new_lo=130, new_hi=4099, len_lo=0, len_hi=0, idle=0, q_heads=24,
             kv_heads=8, dim=64, page=128, window=1024),
        # one request's next token through its adapter, beside the gate projection
        dict(name="adapt 1 row", op="adapt", seqs=1, new_lo=1, new_hi=1, adapters=4, rank=16, k=5120, n=17408),
        # a serving batch in which the requests use many adapters, some none
        dict(name="adapt 64 rows", op="adapt", seqs=64, new_lo=1, new_hi=1, adapters=24, rank=32, k=17408, n=5120),
        # prompts of a few requests
        dict(name="adapt prompts 4k", op="adapt", seqs=4, new_lo=333, new_hi=1701, adapters=3, rank=64, k=5120, n=17408),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "adapt"])
    if op == "adapt":
        c = dict(op=op, seqs=_log(rng, 1, 96), adapters=_log(rng, 1, 32), rank=rng.choice([8, 16, 24, 32, 64, 128]),
                 k=256 * _log(rng, 1, 68), n=_log(rng, 100, 17408))
        most = max(1, 4096 // c["seqs"])
        c["new_hi"] = _log(rng, 1, most)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        return c
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(op=op, seqs=_log(rng, 1, 96), q_heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16]), kv_heads=kv_heads, dim=dim,
             page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        c["new_hi"] = _log(rng, 1, max(1, min(3300, 8000 // c["seqs"])))
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["past_hi"] = _log(rng, 1, 500)
        c["past_lo"] = rng.randint(0, c["past_hi"])
        c["rot"] = rng.choice([16, 32, dim // 2, dim])
        c["inter"] = rng.random() < 0.5
        c["stretch"] = rng.choice([1.0, 1.0, 2.5, 8.0])
        return c
    room = 64 * 8192 * 8 * 128 // (c["seqs"] * kv_heads * dim)       # cached tokens a sequence, on average
    kind = rng.choice(["token", "token", "drafts", "chunk"])
    if kind == "chunk":
        c["seqs"] = min(c["seqs"], 8)
        c["new_hi"] = _log(rng, 9, max(9, min(2048, 8192 // c["seqs"])))
        c["new_lo"] = rng.randint(1, c["new_hi"])
        room = min(room, 9001, max(16, 2 * 4 * 2048 * 6500 * 32 * 128 // (c["seqs"] * c["new_hi"] * c["q_heads"] * dim)))
    else:
        c["new_lo"] = c["new_hi"] = 1 if kind == "token" else rng.randint(2, 8)
    c["len_hi"] = _log(rng, 16, max(17, min(131071, room)))
    c["len_lo"] = rng.randint(0, c["len_hi"])
    c["idle"] = rng.choice([0, 0, 1, 2]) if c["seqs"] > 4 else 0
    c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
    return c


def _spread(count, lo, hi):
    """`count` whole numbers from lo to hi, spread evenly and out of order."""
    return [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(count)]


def _sizes(c):
    """(new tokens, cached tokens with them) of each sequence; an idle slot has a row and nothing in the cache."""
    new = _spread(c["seqs"], c["new_lo"], c["new_hi"])
    if c["op"] == "adapt":
        return new, None
    if c["op"] == "append":
        return new, [p + n for p, n in zip(_spread(c["seqs"] + 1, c["past_lo"], c["past_hi"])[1:], new)]
    total = [max(n, t) for n, t in zip(new, _spread(c["seqs"] + 1, c["len_lo"], c["len_hi"])[1:])]
    for i in range(min(c["idle"], c["seqs"])):
        total[(i * 7) % c["seqs"]] = 0
    return new, total


# ---- inputs -----------------------------------------------------------------------------------------------------------
def _rope_table(positions, rot, stretch, device):
    """cos and sin of position / stretch * 10000^(-2 i / rot): float32 [positions, rot], the cosines first."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot) / stretch
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq[None]
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _page_table(c, total, gen, dev):
    need = [-(-t // c["page"]) for t in total]
    width = max(1, max(need))
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    at = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    table = at[:, None] + torch.arange(width, device=dev)[None]
    used = torch.arange(width, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    return torch.where(used, order[table.clamp(max=pages - 1)], 0).to(torch.int32).contiguous(), pages


def _cache(c, pages, gen, dev):
    """Pages as earlier steps left them: every slot holds something, used or not."""
    shape = (pages, c["kv_heads"], c["page"], c["dim"])
    made = []
    for _ in range(2):
        made.append((torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16) * 110.0).clamp(-E4M3_MAX, E4M3_MAX)
                    .to(torch.float8_e4m3fn))
    for _ in range(2):
        e = torch.randint(-9, -5, shape[:2] + (c["page"] // BLOCK,), generator=gen, device=dev)
        made.append(torch.exp2(e.float()))
    return tuple(made)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = case
    new, total = _sizes(c)
    tokens = sum(new)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = dict(case=c, starts=torch.tensor(starts, dtype=torch.int32, device=dev), tokens=tokens, most=max(new))
    if c["op"] == "adapt":
        s["x"] = torch.randn(tokens, c["k"], generator=gen, device=dev).bfloat16()
        s["y"] = torch.randn(tokens, c["n"], generator=gen, device=dev).bfloat16()
        s["a"] = (torch.randn(c["adapters"], c["rank"], c["k"], generator=gen, device=dev) / c["k"] ** 0.5).bfloat16()
        s["b"] = (torch.randn(c["adapters"], c["n"], c["rank"], generator=gen, device=dev) * 0.5 / c["rank"] ** 0.5).bfloat16()
        s["scales"] = torch.rand(c["adapters"], generator=gen, device=dev) + 0.5
        # -1: a request without an adapter
        s["which"] = torch.randint(-1 if c["seqs"] > 4 else 0, c["adapters"], (c["seqs"],), generator=gen, device=dev).to(torch.int32)
        return s
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    s["longest"] = max(total)
    s["pages"], pool = _page_table(c, total, gen, dev)
    s["cache"] = _cache(c, pool, gen, dev)
    if c["op"] == "append":
        # the output of one projection to queries, keys and values; a few channels of the keys are large, as they are in use
        qkv = torch.randn(tokens, (hq + 2 * hk) * d, generator=gen, device=dev)
        qkv[:, hq * d:(hq + hk) * d:37] *= 8.0
        qkv = qkv.bfloat16()
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["rope"] = _rope_table(max(total), c["rot"], c["stretch"], dev)
    else:
        # queries of mixed sharpness: some rows attend to a few tokens, some to nearly all
        sharp = torch.exp(torch.randn(tokens, hq, 1, generator=gen, device=dev) * 0.7)
        s["q"] = (torch.randn(tokens, hq, d, generator=gen, device=dev) * sharp).bfloat16()
    return s


# ---- the operators ----------------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        import trellis_quantized_weight_gb300 as tq
        if c["op"] == "adapt":
            return tq.lora_add(s["y"], s["x"], s["a"], s["b"], s["scales"], s["starts"], s["which"])
        if c["op"] == "attend":
            return tq.kv_attention(s["q"], s["cache"], s["starts"], s["kv_len"], s["pages"], window=c["window"], max_q=s["most"])
        q = tq.kv_append(s["cache"], s["k"], s["v"], s["starts"], s["kv_len"], s["pages"], q=s["q"], rope=s["rope"],
                         interleaved=c["inter"], max_q=s["most"])
        return dict(q=q, k=s["cache"][0], v=s["cache"][1], k_scale=s["cache"][2], v_scale=s["cache"][3])
    return {"append": _plain_append, "attend": _plain_attend, "adapt": _plain_adapt}[c["op"]](s)


def _token_sequence(s):
    """For each packed token its sequence and its position there."""
    at = torch.arange(s["tokens"], device=s["starts"].device)
    seq = torch.searchsorted(s["starts"][1:].long().contiguous(), at, right=True)
    return seq, (s["kv_len"][seq] - s["starts"][seq + 1] + at).long()


def _rotate(x, table, rot, inter):
    """x [tokens, heads, dim] in float32 with its first `rot` values rotated by the table's rows [tokens, rot]."""
    half = rot // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _power(a):
    """The smallest power of two s >= 2^-100 with a <= 448 s, from a's own bits."""
    m, e = torch.frexp(a)
    e = (e - 9 + (m > 0.875).int()).clamp(min=-100)
    e = torch.where(a > 0, e, -100)
    s = ((e + 127) << 23).view(torch.float32)
    return torch.where(torch.isfinite(a), s, torch.nan)


def _plain_append(s):
    c = s["case"]
    page, hk = c["page"], c["kv_heads"]
    seq, pos = _token_sequence(s)
    row = s["rope"][pos]
    phys = s["pages"][seq, pos // page].long()
    slot = pos % page
    blk = slot // BLOCK
    # the block of each sequence's first new token may hold earlier ones
    first = s["starts"][:-1].long()
    live = s["starts"][1:] > s["starts"][:-1]
    seq0 = torch.arange(first.numel(), device=first.device)[live]
    p0 = pos[first[live]]
    page0, blk0, kept = s["pages"][seq0, p0 // page].long(), p0 % page // BLOCK, p0 % BLOCK
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    for x, codes, scale in ((_rotate(s["k"].float(), row, c["rot"], c["inter"]), k_codes, k_scale), (s["v"].float(), v_codes, v_scale)):
        flat = (phys * (page // BLOCK) + blk)
        most = torch.zeros(scale.shape[0] * (page // BLOCK), hk, device=x.device)
        most.scatter_reduce_(0, flat[:, None].expand(-1, hk), x.abs().amax(-1), "amax")
        want = _power(most[flat])                                       # of each token's block, from the new tokens
        had = torch.where(kept[:, None] > 0, scale[page0, :, blk0], 0.0)
        scale[phys, :, blk] = want
        need = scale[page0, :, blk0]
        kept_scale = torch.maximum(had, need)
        scale[page0, :, blk0] = kept_scale
        # earlier tokens of that block, at the scale it has now
        lane = torch.arange(BLOCK, device=x.device)
        at = (page0[:, None], slice(None), blk0[:, None] * BLOCK + lane[None])
        old = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn)      # [sequences, 16, heads, dim]
        again = (old.float() * (had / kept_scale)[:, None, :, None]).to(torch.float8_e4m3fn)
        keep = (lane[None] < kept[:, None])[:, :, None, None]
        codes.view(torch.uint8)[at] = torch.where(keep, again.view(torch.uint8), old.view(torch.uint8))
        new = (x / scale[phys, :, blk][:, :, None]).to(torch.float8_e4m3fn)
        codes.view(torch.uint8)[phys, :, slot] = new.view(torch.uint8)
    return dict(q=_rotate(s["q"].float(), row, c["rot"], c["inter"]).bfloat16(), k=k_codes, v=v_codes, k_scale=k_scale, v_scale=v_scale)


def _plain_attend(s):
    c = s["case"]
    hk, d, page = c["kv_heads"], c["dim"], c["page"]
    g = c["q_heads"] // hk
    seqs, most, longest = c["seqs"], s["most"], max(1, s["longest"])
    used = s["pages"][:, :-(-longest // page)].long()
    dense = []
    for codes, scale in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        x = codes.view(torch.uint8)[used].view(torch.float8_e4m3fn).float()          # [seqs, pages, heads, page, dim]
        x = x * scale[used].repeat_interleave(BLOCK, -1)[..., None]
        dense.append(x.transpose(1, 2).reshape(seqs, hk, -1, d))
    k, v = dense
    lane = torch.arange(most, device=k.device)
    count = s["starts"][1:] - s["starts"][:-1]
    row = (s["starts"][:-1, None] + torch.minimum(lane[None], (count - 1).clamp(min=0)[:, None])).long()
    q = s["q"][row].float().view(seqs, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(seqs, hk, g * most, d)
    score = (q @ k.transpose(-1, -2)).view(seqs, hk, g, most, -1) * (1.0 / math.sqrt(d))
    pos = (s["kv_len"] - count)[:, None] + lane[None]                                # of each row
    key = torch.arange(k.shape[2], device=k.device)
    seen = key[None, None] <= pos[:, :, None]
    if c["window"]:
        seen &= key[None, None] > pos[:, :, None] - c["window"]
    seen = seen[:, None, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(seqs, hk, g * most, -1) @ v).view(seqs, hk, g, most, d)
    o = torch.where(total > 0, o / total, 0.0)                                       # a row that sees nothing is zero
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, most, hk * g, d)
    seq, at = _token_sequence(s)
    return o[seq, at - (s["kv_len"] - count)[seq]].bfloat16()


def _plain_adapt(s):
    count = s["starts"][1:] - s["starts"][:-1]
    lane = torch.arange(s["most"], device=count.device)
    row = (s["starts"][:-1, None] + torch.minimum(lane[None], (count - 1).clamp(min=0)[:, None])).long()
    which = s["which"].clamp(min=0).long()
    h = s["x"][row].float() @ s["a"][which].float().transpose(-1, -2)
    delta = (h @ s["b"][which].float().transpose(-1, -2)) * torch.where(s["which"] < 0, 0.0, s["scales"][which])[:, None, None]
    at = torch.arange(s["tokens"], device=count.device)
    seq = torch.searchsorted(s["starts"][1:].long().contiguous(), at, right=True)
    return (s["y"].float() + delta[seq, at - s["starts"][seq]]).bfloat16()


# ---- what a pass cannot do without ------------------------------------------------------------------------------------
def work(case):
    c = case
    new, total = _sizes(c)
    tokens = sum(new)
    if c["op"] == "adapt":
        seen = min(c["adapters"], c["seqs"])
        return dict(bytes=2 * tokens * (c["k"] + 2 * c["n"]) + 2 * seen * c["rank"] * (c["k"] + c["n"]),
                    flops=2 * tokens * c["rank"] * (c["k"] + c["n"]))
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        blocks = sum((t - 1) // BLOCK - (t - n) // BLOCK + 1 for n, t in zip(new, total))
        return dict(bytes=tokens * (4 * hq * d + 2 * hk * d * 3 + 4 * c["rot"]) + 8 * hk * blocks,
                    flops=tokens * (3 * (hq + hk) * c["rot"] + 4 * hk * d))
    read = pairs = 0
    for n, t in zip(new, total):
        if t == 0:
            continue
        w = c["window"] or t
        read += t - max(0, t - n - w + 1)
        full = max(0, min(n, w - (t - n)))                       # rows that see everything before them
        pairs += full * (t - n) + full * (full + 1) // 2 + (n - full) * w
    return dict(bytes=read * hk * (2 * d + 8 / BLOCK) + 4 * tokens * hq * d, flops=4 * pairs * hq * d)


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------------
def exact(case, seed):
    s, c = prepare(case, seed), case
    new, total = _sizes(c)
    start = [sum(new[:i]) for i in range(len(new))]
    if c["op"] == "adapt":
        out = s["y"].double()
        for i, n in enumerate(new):
            w = int(s["which"][i])
            if w >= 0:
                rows = slice(start[i], start[i] + n)
                out[rows] += float(s["scales"][w]) * torch.einsum("mr,nr->mn", torch.einsum("mk,rk->mr", s["x"][rows].double(), s["a"][w].double()),
                                                                  s["b"][w].double())
        return out
    return _exact_attend(s, c, new, total, start) if c["op"] == "attend" else _exact_append(s, c, new, total, start)


def _exact_attend(s, c, new, total, start):
    page, g = c["page"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["tokens"], c["q_heads"], c["dim"], dtype=torch.float64, device=s["q"].device)
    for i, (n, t) in enumerate(zip(new, total)):
        if t == 0:
            continue
        ids = s["pages"][i, :-(-t // page)].long()
        k, v = [(codes[ids].double().unflatten(2, (-1, BLOCK)) * scale[ids].double()[..., None, None]).flatten(2, 3).transpose(0, 1).flatten(1, 2)[:, :t]
                for codes, scale in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3]))]
        for r in range(0, n, 512):
            rows = torch.arange(r, min(n, r + 512), device=k.device)
            q = s["q"][start[i] + rows].double().unflatten(1, (-1, g))                  # [rows, kv heads, group, dim]
            x = torch.einsum("rhgd,hkd->hgrk", q, k) / c["dim"] ** 0.5
            ahead = torch.arange(t, device=k.device)[None] - (t - n + rows)[:, None]    # > 0: not there yet
            hidden = (ahead > 0) | ((ahead <= -c["window"]) if c["window"] else False)
            x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[start[i] + rows] = torch.einsum("hgrk,hkd->rhgd", x, v).flatten(1, 2)
    return out


def _exact_append(s, c, new, total, start):
    """The codes as the quotients that they are rounded from."""
    page, rot = c["page"], c["rot"]
    codes = [s["cache"][0].double(), s["cache"][1].double()]
    scales = [s["cache"][2].double(), s["cache"][3].double()]
    q = s["q"].double().clone()
    for i, (n, t) in enumerate(zip(new, total)):
        rows = slice(start[i], start[i] + n)
        pos = torch.arange(t - n, t, device=q.device)
        angle = s["rope"][pos].double()
        turn = torch.complex(angle[:, :rot // 2], angle[:, rot // 2:])[:, None]
        pair = (slice(0, rot, 2), slice(1, rot, 2)) if c["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
        kv = [s["k"][rows].double().clone(), s["v"][rows].double()]
        for x in (q[rows], kv[0]):
            z = torch.complex(x[..., pair[0]], x[..., pair[1]]) * turn
            x[..., pair[0]], x[..., pair[1]] = z.real, z.imag
        for b in range((t - n) // BLOCK, (t - 1) // BLOCK + 1):
            lo, hi = max(b * BLOCK, t - n), min(b * BLOCK + BLOCK, t)
            ph, off = int(s["pages"][i, b * BLOCK // page]), b * BLOCK % page
            for x, code, scale in zip(kv, codes, scales):
                y = x[lo - (t - n):hi - (t - n)].transpose(0, 1)                        # [heads, tokens, dim]
                most = y.abs().amax((1, 2))
                m, e = torch.frexp(most / E4M3_MAX)                                     # most = 448 m 2^e, 0.5 <= m < 1
                want = torch.ldexp(torch.ones_like(m), (e - (m == 0.5).int()).clamp(min=-100))
                had = scale[ph, :, off // BLOCK].clone()
                kept = lo - b * BLOCK
                now = torch.maximum(want, had) if kept else want
                code[ph, :, off:off + kept] *= (had / now)[:, None, None]
                code[ph, :, off + kept:off + kept + hi - lo] = y / now[:, None, None]
                scale[ph, :, off // BLOCK] = now
    return dict(q=q, k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1])
