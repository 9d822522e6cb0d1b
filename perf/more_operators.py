"""Workloads of the serving operators around a cache in 8 bits: page tables and
slot maps built from request lengths, appending rotated keys and values to a
cache of E4M3 codes with a power-of-two scale for each block of tokens and
head, reading tokens back in 16 bits, and attention of one new token per
sequence over that cache or a 16-bit one, with a window and first tokens that
stay visible.

``listed()`` names cases over the real range, ``draw(rng)`` makes more of the
same ranges, ``prepare`` makes a case's inputs on the GPU, ``run`` makes one
pass and returns its outputs, ``exact`` gives the same outputs from the
definitions in 64 bits, ``work`` counts the bytes and operations that a pass
cannot do without.  With ``own`` set ``run`` calls the library; without it the
operators are written out in elementary torch operations in 32 bits (64 for
values that are rounded to 8), rounded once at the end.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
CACHE_ELEMENTS = 64 * 16384 * 8 * 128  # keys (or values) of the largest cache below


def listed():
    return [
        # A decoding step of 256 users: their places in the cache, a page for the few that begin one; a draft token given back first.
        dict(name="plan-step", op="plan", seqs=256, longest=8192, new=1, page=16, spare=64),
        # A batch of 96 prompts admitted at once where earlier requests have just ended: tables and slots of a quarter million tokens.
        dict(name="plan-prompts", op="plan", seqs=96, longest=5500, new=0, page=16, spare=100),
        # One user's new token: nothing but latency.
        dict(name="append8-token", op="append", tokens=1, seqs=0, start=700, heads=32, kv_heads=8, dim=128, rot=128, page=16, block=16, type="bf16", interleaved=False, order="nhd"),
        # A batch of users, each one token at a place of its own, most of them in blocks that hold earlier tokens; half of each head rotated.
        dict(name="append8-batch", op="append", tokens=192, seqs=0, start=4000, heads=16, kv_heads=16, dim=64, rot=32, page=32, block=8, type="f16", interleaved=True, order="hnd"),
        # Prompts of three users in one call, an odd count of tokens, a scale for each page and head.
        dict(name="append8-prompts", op="append", tokens=8191, seqs=3, start=0, heads=32, kv_heads=8, dim=128, rot=128, page=64, block=64, type="bf16", interleaved=False, order="nhd"),
        # A short context back in 16 bits, for a prompt's next part to attend to.
        dict(name="read-short", op="read", tokens=300, seqs=1, kv_heads=8, dim=128, page=16, block=16, cache="e4m3", type="bf16", order="nhd"),
        # Long contexts of five users back in 16 bits.
        dict(name="read-long", op="read", tokens=100003, seqs=5, kv_heads=8, dim=128, page=64, block=32, cache="e4m3", type="bf16", order="hnd"),
        # One user early in a conversation: latency again.
        dict(name="attention8-short", op="attention", seqs=1, longest=300, ragged=False, heads=32, kv_heads=8, dim=128, page=16, block=16, window=0, sinks=0, cache="e4m3", type="bf16", order="nhd"),
        # One user with a very long context: few rows, a long axis.
        dict(name="attention8-long", op="attention", seqs=1, longest=131071, ragged=False, heads=32, kv_heads=8, dim=128, page=64, block=64, window=0, sinks=0, cache="e4m3", type="bf16", order="hnd"),
        # A serving batch with lengths from none to 16384.
        dict(name="attention8-batch", op="attention", seqs=64, longest=16384, ragged=True, heads=32, kv_heads=8, dim=128, page=16, block=16, window=0, sinks=0, cache="e4m3", type="bf16", order="nhd"),
        # Small heads of their own, 16-bit cache: the newest 1000 tokens and the first four.
        dict(name="sinks-window", op="attention", seqs=96, longest=5000, ragged=True, heads=16, kv_heads=16, dim=64, page=32, block=32, window=1000, sinks=4, cache="f16", type="f16", order="nhd"),
        # Long conversations in 8 bits of which the newest 4096 tokens and the first 20 are seen.
        dict(name="sinks-window8", op="attention", seqs=40, longest=60000, ragged=False, heads=32, kv_heads=8, dim=128, page=64, block=16, window=4096, sinks=20, cache="e4m3", type="bf16", order="nhd"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "read", "attention", "attention", "attention"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "plan":
        seqs = _log(rng, 1, 2000)
        longest = min(_log(rng, 1, 131071), 260000 // seqs)
        new = rng.choice([0, 1, min(longest, rng.choice([2, 5, 40]))])
        return dict(op=op, seqs=seqs, longest=longest, new=new, page=page, spare=rng.randrange(0, 200))
    block = rng.choice([b for b in (1, 4, 8, 12, 16, 24, 32, 64, 128) if page % b == 0])
    kind = rng.choice(["bf16", "f16"])
    order = rng.choice(["nhd", "hnd"])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 16])
    if op == "append":
        tokens = _log(rng, 1, 8191)
        tokens = max(1, min(tokens, 8191 * 48 * 128 // (dim * (heads + 2 * kv_heads))))
        seqs = rng.choice([0, min(tokens, rng.choice([1, 2, 5]))]) if tokens <= 256 else rng.choice([1, 2, 5])
        return dict(op=op, tokens=tokens, seqs=seqs, start=rng.randrange(0, 5000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), page=page, block=block, type=kind, interleaved=rng.choice([False, True]), order=order)
    cache = rng.choice(["e4m3", "e4m3", kind])
    if op == "read":
        tokens = min(_log(rng, 1, 100003), 100003 * 1024 // (kv_heads * dim))
        return dict(op=op, tokens=tokens, seqs=min(tokens, rng.choice([1, 2, 5, 9])), kv_heads=kv_heads, dim=dim, page=page, block=block,
                    cache=cache, type=kind, order=order)
    seqs = _log(rng, 1, 96)
    longest = min(_log(rng, 1, 131071), CACHE_ELEMENTS * 49 // 100 // (seqs * kv_heads * dim))
    few = rng.choice([0, 0, 1]) if cache == "e4m3" else 1  # a 16-bit cache: with sinks
    return dict(op=op, seqs=seqs, longest=max(1, longest), ragged=rng.choice([False, True]), heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                block=block, window=_log(rng, 1, 8192) if few else 0, sinks=_log(rng, 1, 200) if few else 0, cache=cache, type=kind, order=order)


def _spread(n, longest):
    """Lengths of n sequences, spread from none to the longest."""
    return [longest * ((17 * i + n - 1) % n) // (n - 1) if n > 1 else longest for i in range(n)]


def _lengths(case):
    return _spread(case["seqs"], case["longest"]) if case["ragged"] else [case["longest"]] * case["seqs"]


def _seen(case, length):
    """Positions that are seen: the first `sinks` and the newest `window`."""
    return min(length, case["sinks"] + case["window"]) if case["window"] else length


def _plan_new(case):
    """(lengths, new tokens among them) of a plan's sequences; new = 0: all of them are."""
    lengths = _spread(case["seqs"], case["longest"])
    return lengths, [min(n, case["new"]) if case["new"] else n for n in lengths]


def _split(case):
    """(first new position, new tokens) of each sequence of prompts."""
    t, n = case["tokens"], case["seqs"]
    each = -(-t // n)
    return [(case["start"], max(0, min(t - i * each, each))) for i in range(n)]


def work(case):
    page = case["page"]
    if case["op"] == "plan":
        lengths, new = _plan_new(case)
        pages = sum(-(-a // page) - -(-(a - n) // page) for a, n in zip(lengths, new))
        # back and forth: per sequence count, length, room in and length, room out; a page's table entry and its number; a token's three indexes
        return {"bytes": 2 * (20 * case["seqs"] + 8 * pages) + 16 * sum(new), "flops": 0}
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        t, h, r = case["tokens"], case["heads"], case["rot"]
        b = case["block"]
        if case["seqs"]:  # places whose block is touched: read back
            look = sum(max(0, s + n - s // b * b) for s, n in _split(case) if n)
            places = max(n for _, n in _split(case))
        else:
            look, places = t * (1 + (b - 1) / 2), t
        look *= hk * d
        return {"bytes": int(2 * 2 * t * d * h + 2 * (2 + 1) * t * d * hk + 4 * places * r + 8 * t + 2 * (1 + 2) * look), "flops": 3 * t * r * (h + hk)}
    width = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "read":
        return {"bytes": 2 * (width + 2) * case["tokens"] * hk * d + 8 * case["tokens"], "flops": 0}
    h = case["heads"]
    seen = sum(_seen(case, n) for n in _lengths(case))
    scales = 2 * seen * hk // case["block"] if width == 1 else 0
    return {"bytes": 2 * width * seen * hk * d + scales + 2 * 2 * case["seqs"] * h * d + 4 * seen // page, "flops": 4 * seen * h * d}


# ------------------------------------------------------------------ inputs

def _scales(top):
    """E8M0 codes: the smallest power of two that brings magnitudes up to `top` to 448 or less."""
    f, x = torch.frexp(top)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    return torch.where(top > 0, (e + 127).clamp(0, 254), 0)


def _pages(case, cache, count, gen, dev):
    """Keys and values of `count` pages, indexed [page][place][head][dim] whatever their order in memory, and their scales: heads of
    different size, as projections make them."""
    p, h, d = case["page"], case["kv_heads"], case["dim"]
    made = []
    for _ in range(2):
        gain = torch.exp2(torch.randint(-3, 3, (h, 1), generator=gen, device=dev).float())
        x = torch.randn((count, p, h, d), generator=gen, device=dev, dtype=torch.float32)
        if cache != "e4m3":
            x = x.to(TYPES[cache])
            made += [x.transpose(1, 2).contiguous().transpose(1, 2) if case["order"] == "hnd" else x, None]
            continue
        x = x.mul_(gain).view(count, p // case["block"], case["block"], h, d)
        code = _scales(x.abs().amax(-1).amax(2))
        x = x.mul_(torch.exp2(127.0 - code)[:, :, None, :, None]).to(E4M3).view(count, p, h, d)
        made += [x.transpose(1, 2).contiguous().transpose(1, 2) if case["order"] == "hnd" else x, code.to(torch.uint8)]
    return made


def _table(need, gen, dev):
    """A page table for `need` pages per sequence: pages of the pool in random order."""
    wide = max(1, max(need))
    order = torch.randperm(sum(need) + 1, generator=gen, device=dev).to(torch.int32)
    need = torch.tensor(need, device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(wide, device=dev)
    at = torch.where(col < need[:, None], first[:, None] + col, 0)
    return torch.where(col < need[:, None], order[at], 0).to(torch.int32)


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    s = {"case": case}
    page = case["page"]
    if case["op"] == "plan":
        lengths, new = (torch.tensor(v, device=dev) for v in _plan_new(case))
        order = torch.randperm(case["seqs"], generator=gen, device=dev)
        lengths, new = lengths[order], new[order]
        need = (-(-lengths // page)).tolist()
        used, wide = sum(need), max(need) + 3
        table = torch.full((case["seqs"], wide), -1, dtype=torch.int32, device=dev)
        pages = torch.randperm(used + case["spare"], generator=gen, device=dev).to(torch.int32)
        table.masked_scatter_(torch.arange(wide, device=dev) < torch.tensor(need, device=dev)[:, None], pages[case["spare"]:])
        s["table"] = table
        s["lengths"], s["new"] = lengths.to(torch.int32), new.to(torch.int32)
        s["back"] = -s["new"]
        s["room"] = _ints(need, dev) * page
        s["tokens"] = sum(new.tolist()) + 7  # a batch of fixed size: some rows hold no token
        # the free pages: how many, a word that is zero, the stack
        s["pool"] = torch.cat([_ints([case["spare"], 0], dev), pages[:case["spare"]], torch.zeros(used, dtype=torch.int32, device=dev)])
        return s
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        dt = TYPES[case["type"]]
        t, h, b = case["tokens"], case["heads"], case["block"]
        if case["seqs"]:  # prompts: each sequence's tokens in a row
            parts = _split(case)
            s["seq"] = _ints([i for i, (_, n) in enumerate(parts) for _ in range(n)], dev)
            s["pos"] = _ints([a + j for a, n in parts for j in range(n)], dev)
            look = [(i, j) for i, (a, n) in enumerate(parts) if n for j in range(a // b * b, a + n)]
            s["look_seq"], s["look_pos"] = (_ints(v, dev) for v in zip(*look))
            last, n = case["start"] + max(m for _, m in parts), case["seqs"]
            need = -(-last // page)
            s["table"], count = _table([need] * n, gen, dev), need * n + 1
        else:             # one token of each sequence
            s["seq"], n = None, t
            pos = torch.randint(case["start"] // 2, case["start"] + 1, (t,), generator=gen, device=dev)
            s["pos"] = pos.to(torch.int32)
            last = case["start"] + 1
            j = torch.arange(b, device=dev)
            look = pos[:, None] // b * b + j
            s["look_pos"] = torch.where(look <= pos[:, None], look, -1).to(torch.int32).view(-1)
            s["look_seq"] = torch.arange(t, device=dev, dtype=torch.int32)[:, None].repeat(1, b).view(-1)
            # only the last pages of each sequence are at hand: earlier ones hold nothing that is looked at
            s["table"] = torch.randperm(2 * n, generator=gen, device=dev)[:n, None].expand(n, -(-last // page)).to(torch.int32).contiguous()
            count = 2 * n
        s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"] = _pages(case, "e4m3", count, gen, dev)
        fused = torch.randn((t, h + 2 * hk, d), generator=gen, device=dev).to(dt)  # one projection gives all three
        s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
        half = case["rot"] // 2
        turn = torch.exp(torch.arange(half, device=dev, dtype=torch.float64) * (-math.log(10000.0) / half))
        angle = torch.arange(last, device=dev, dtype=torch.float64)[:, None] * turn
        s["rope"] = torch.cat([torch.cos(angle), torch.sin(angle)], -1).float()
        return s
    if case["op"] == "read":
        each = -(-case["tokens"] // case["seqs"])
        i = torch.arange(case["tokens"], device=dev)
        s["seq"], s["pos"] = (i // each).to(torch.int32), (i % each).to(torch.int32)
        need = -(-each // page)
        s["table"] = _table([need] * case["seqs"], gen, dev)
        s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"] = _pages(case, case["cache"], need * case["seqs"] + 1, gen, dev)
        return s
    lengths = _ints(_lengths(case), dev)
    s["lengths"] = lengths[torch.randperm(case["seqs"], generator=gen, device=dev)]
    need = [-(-int(n) // page) for n in s["lengths"].tolist()]
    s["table"] = _table(need, gen, dev)
    s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"] = _pages(case, case["cache"], sum(need) + 1, gen, dev)
    s["q"] = torch.randn((case["seqs"], case["heads"], d), generator=gen, device=dev).to(TYPES[case["type"]])
    return s


# -------------------------------------------------------------- plain forms

def _plan_plain(s, new, tokens):
    """One plan: the new state is written into s; the maps of `tokens` tokens, or None."""
    page, table, pool = s["case"]["page"], s["table"], s["pool"]
    seqs, wide = table.shape
    n, length, held = new.long(), s["lengths"].long(), s["room"].long() // page
    after = (length + n).clamp(min=0)
    want = (after + page - 1) // page
    adds = n.clamp(min=0)
    ends = torch.cumsum(adds, 0)
    fits = after <= wide * page
    if tokens is not None:
        fits = fits & (ends <= tokens)
    grow = torch.where(fits & (n >= 0), (want - held).clamp(min=0), 0)
    upto = torch.cumsum(grow, 0)
    free = pool[0].long()
    ok = (n < 0) | (fits & ((grow == 0) | (upto <= free)))
    grow = torch.where(ok, grow, 0)
    given = torch.where(n < 0, (held - want).clamp(min=0), 0)
    before = torch.cumsum(given, 0) - given
    left, total = free - grow.sum(), given.sum()
    col = torch.arange(wide, device=table.device)
    first, size = held[:, None], grow[:, None]
    gets = (col >= first) & (col < first + size)
    at = free - 1 - ((upto - grow)[:, None] + col - first)
    gives = (col >= want[:, None]) & (col < first) & (n < 0)[:, None]
    to = left + total - 1 - (before[:, None] + col - want[:, None])
    stack = torch.cat([pool[2:], pool[:1]])  # the last takes what is not given
    got = stack[torch.where(gets, at, 0)]
    stack.scatter_(0, torch.where(gives, to, stack.shape[0] - 1).view(-1), table.view(-1))
    pool[2:] = stack[:-1]
    pool[0] = (left + total).to(torch.int32)
    table.copy_(torch.where(gets, got, torch.where(gives, -1, table)))
    s["room"].copy_(torch.where(n < 0, torch.minimum(want, held), held + grow) * page)
    s["lengths"].copy_(torch.where(ok, after, length))
    if tokens is None:
        return None
    t = torch.arange(tokens, device=table.device)
    seq = torch.searchsorted(ends, t, right=True)
    there = seq < seqs
    i = seq.clamp(max=seqs - 1)
    pos = torch.where(there & ok[i], length[i] + t - (ends - adds)[i], -1)
    p = pos.clamp(min=0)
    slot = torch.where(pos >= 0, table[i, p // page].long() * page + p % page, -1)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
    return torch.where(there, seq, -1).to(torch.int32), pos.to(torch.int32), slot, offsets


def _rotated_plain(x, cos, sin, case):
    r = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _store_plain(pages, scale, x, page, place, block):
    """Values x [tokens, heads, dim] in 64 bits into places of a cache in 8 bits."""
    n, blocks, h = scale.shape
    where = page * blocks + place // block
    ones = torch.zeros(n * blocks, device=x.device)
    touched = ones.index_reduce(0, where, torch.ones_like(where, dtype=torch.float32), "amax")[:, None] > 0
    fresh = ones.index_reduce(0, where, (place % block == 0).float(), "amax")[:, None] > 0
    top = torch.zeros((n * blocks, h), device=x.device, dtype=torch.float64).index_reduce(0, where, x.abs().amax(-1), "amax")
    need, old = _scales(top), scale.view(-1, h).long()
    code = torch.where(touched, torch.where(fresh, need, torch.maximum(need, old)), old)
    down = torch.where(fresh, 0, old - code).view(n, blocks, 1, h, 1)
    kept = pages.float().unflatten(1, (blocks, block)) * torch.exp2(down.float())
    pages.copy_(kept.to(E4M3).flatten(1, 2))
    scale.copy_(code.view(n, blocks, h).to(torch.uint8))
    shift = torch.exp2(127.0 - code[where].double())[:, :, None]
    pages.view(torch.uint8)[page, place] = (x * shift).float().to(E4M3).view(torch.uint8)


def _read_plain(s, which, page, place, keep):
    case = s["case"]
    x = s[which + "_pages"]
    if x.dtype == E4M3:
        x = x.view(torch.uint8)[page, place].view(E4M3).float()
        x = x * torch.exp2(s[which + "_scale"][page, place // case["block"]].float() - 127)[..., None]
    else:
        x = x[page, place].float()
    return torch.where(keep[:, None, None], x, 0.0).to(TYPES[case["type"]])


def _append_plain(s):
    case = s["case"]
    pos, half = s["pos"].long(), case["rot"] // 2
    angle = s["rope"][pos]
    cos, sin = angle[:, None, :half], angle[:, None, half:]
    seq = torch.arange(case["tokens"], device=pos.device) if s["seq"] is None else s["seq"].long()
    page, place = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
    k = _rotated_plain(s["k"].double(), cos.double(), sin.double(), case)
    _store_plain(s["k_pages"], s["k_scale"], k, page, place, case["block"])
    _store_plain(s["v_pages"], s["v_scale"], s["v"].double(), page, place, case["block"])
    q = _rotated_plain(s["q"].float(), cos, sin, case).to(TYPES[case["type"]])
    look = s["look_pos"].long()
    p = look.clamp(min=0)
    page, place = s["table"][s["look_seq"].long(), p // case["page"]].long(), p % case["page"]
    return [q] + [_read_plain(s, which, page, place, look >= 0) for which in "kv"]


def _attention_plain(s):
    case = s["case"]
    b, h, hk, d = case["seqs"], case["heads"], case["kv_heads"], case["dim"]
    table = s["table"].long()

    def whole(which):
        x = s[which + "_pages"]
        if x.dtype != E4M3:
            return x[table].float().reshape(b, -1, hk, d)
        x = x.view(torch.uint8)[table].view(E4M3).float().unflatten(2, (-1, case["block"]))
        return x.mul_(torch.exp2(s[which + "_scale"][table].float() - 127)[:, :, :, None, :, None]).reshape(b, -1, hk, d)

    keys = whole("k")
    q = s["q"].float().view(b, hk, h // hk, d)
    score = torch.einsum("bkgd,blkd->bkgl", q, keys) * d ** -0.5
    del keys
    at, length = torch.arange(score.shape[-1], device=q.device), s["lengths"].long()[:, None]
    seen = at < length
    if case["window"]:
        seen = seen & ((at >= length - case["window"]) | (at < case["sinks"]))
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = torch.einsum("bkgl,blkd->bkgd", weight, whole("v")) / torch.where(total > 0, total, 1.0)
    return out.view(b, h, d).to(TYPES[case["type"]])


def run(state):
    s = state
    case = s["case"]
    if own:
        import fp4_block_scaled_quantize_gb300 as fq
    if case["op"] == "plan":  # tokens given back, then taken again: the state is as before
        if own:
            fq.page_plan(s["back"], s["lengths"], s["table"], s["room"], s["pool"], case["page"])
            maps = fq.page_plan(s["new"], s["lengths"], s["table"], s["room"], s["pool"], case["page"], tokens=s["tokens"])
        else:
            _plan_plain(s, s["back"], None)
            maps = _plan_plain(s, s["new"], s["tokens"])
        return list(maps) + [s["lengths"], s["table"], s["room"], s["pool"]]
    if case["op"] == "append":
        if not own:
            return _append_plain(s)
        q = fq.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["pos"], seq=s["seq"], q=s["q"], rope=s["rope"],
                         interleaved=case["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        # the blocks that it wrote into, as the values that they stand for
        k, v = fq.kv_read(s["k_pages"], s["v_pages"], s["table"], s["look_pos"], seq=s["look_seq"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"], dtype=TYPES[case["type"]])
        return [q, k, v]
    if case["op"] == "read":
        if own:
            return list(fq.kv_read(s["k_pages"], s["v_pages"], s["table"], s["pos"], seq=s["seq"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"], dtype=TYPES[case["type"]]))
        pos = s["pos"].long()
        page, place = s["table"][s["seq"].long(), pos // case["page"]].long(), pos % case["page"]
        return [_read_plain(s, which, page, place, pos >= 0) for which in "kv"]
    if own:
        return fq.decode_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], window=case["window"],
                                   sinks=case["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _attention_plain(s)


# ------------------------------------------------------- definitions, 64 bits

def _e4m3(x):
    """The nearest E4M3 value, ties to the even one, of numbers up to 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _held(s, which):
    """What a cache's places stand for, [page][place][head][dim]."""
    x = s[which + "_pages"].double()
    if s[which + "_scale"] is not None:
        x = x * torch.exp2(s[which + "_scale"].double() - 127).repeat_interleave(s["case"]["block"], 1)[..., None]
    return x


def _exact_store(s, which, x, page, place):
    """The values of all places after the tokens' x have been stored, block by block of those touched."""
    b, blocks = s["case"]["block"], s["case"]["page"] // s["case"]["block"]
    value = _held(s, which)
    value = value.reshape(-1, b, *value.shape[2:])  # [block][place][head][dim]
    old = torch.exp2(s[which + "_scale"].double() - 127).reshape(value.shape[0], -1)
    where = page * blocks + place // b
    touched, of = torch.unique(where, return_inverse=True)
    now, had = value[touched], old[touched]
    new = torch.zeros(now.shape[:2], dtype=torch.bool, device=x.device)
    new[of, place % b] = True
    now[of, place % b] = x
    top = torch.where(new[:, :, None, None], now, 0.0).abs().amax((1, 3))
    least = torch.exp2(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -127))))
    least = torch.where(least / 2 * 448 >= top, (least / 2).clamp(min=2.0 ** -127), torch.where(least * 448 < top, least * 2, least))
    unit = torch.where(new[:, :1], least, torch.maximum(least, had))[:, None, :, None]
    value[touched] = _e4m3(now / unit) * unit
    return value.view(-1, s["case"]["page"], *value.shape[2:])


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "read":
        pos = s["pos"].long()
        page, place = s["table"][s["seq"].long(), pos // case["page"]].long(), pos % case["page"]
        return [_held(s, which)[page, place] for which in "kv"]
    if case["op"] == "append":
        pos, half = s["pos"].long(), case["rot"] // 2
        z = torch.complex(s["rope"][pos, :half].double(), s["rope"][pos, half:].double())[:, None]

        def turned(x):
            x = x.double()
            y = x.clone()
            a = slice(0, case["rot"], 2) if case["interleaved"] else slice(0, half)
            b = slice(1, case["rot"], 2) if case["interleaved"] else slice(half, case["rot"])
            w = torch.complex(x[..., a], x[..., b]) * z
            y[..., a], y[..., b] = w.real, w.imag
            return y

        seq = torch.arange(case["tokens"], device=pos.device) if s["seq"] is None else s["seq"].long()
        page, place = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
        look = s["look_pos"].long()
        at = s["table"][s["look_seq"].long(), look.clamp(min=0) // case["page"]].long(), look.clamp(min=0) % case["page"]
        out = [turned(s["q"])]
        for which, x in (("k", turned(s["k"])), ("v", s["v"].double())):
            held = _exact_store(s, which, x, page, place)[at]
            held[look < 0] = 0
            out.append(held)
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    group = case["heads"] // case["kv_heads"]
    for i, length in enumerate(s["lengths"].tolist()):
        if length == 0:
            continue
        at = torch.arange(length, device=out.device)
        if case["window"]:
            at = at[(at < case["sinks"]) | (at >= length - case["window"])]
        page, place = s["table"][i, at // case["page"]].long(), at % case["page"]
        for j in range(case["kv_heads"]):
            keys, values = (s[w + "_pages"].view(torch.uint8)[page, place, j].view(E4M3).double() *
                            torch.exp2(s[w + "_scale"][page, place // case["block"], j].double() - 127)[:, None]
                            if s[w + "_scale"] is not None else s[w + "_pages"][page, place, j].double() for w in "kv")
            w = torch.softmax(s["q"][i, j * group:(j + 1) * group].double() @ keys.t() / math.sqrt(case["dim"]), -1)
            out[i, j * group:(j + 1) * group] = w @ values
    return out
