"""Workloads of the token-by-token serving operators: products with 4-bit
weights for a few tokens, appending rotated keys and values to a paged cache,
and attention of one new token per sequence over that cache.

``listed()`` names cases over the real range, ``draw(rng)`` makes more of the
same ranges, ``prepare`` makes a case's inputs on the GPU, ``run`` makes one
pass and returns its outputs, ``exact`` gives the same outputs from the
definitions in 64 bits, ``work`` counts the bytes and operations that a pass
cannot do without.  With ``own`` set ``run`` calls the library; without it the
operators are written out in elementary torch operations in 32 bits, rounded
once at the end.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "ue5m3": 16, "mxfp4": 32, "ue5m3_b32": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CACHE_ELEMENTS = 64 * 16384 * 8 * 128  # keys (or values) of the largest cache below


def listed():
    return [
        # One token through a 4096 x 4096 projection: a single user's reply, where latency counts.
        dict(name="matvec-token-4096", op="matvec", tokens=1, n=4096, k=4096, fmt="nvfp4", layout="plain", x="bf16", y="bf16"),
        # The same token through the 8B down_proj, weights as the training GEMM holds them.
        dict(name="matvec-token-down", op="matvec", tokens=1, n=4096, k=14336, fmt="ue5m3", layout="mma", x="bf16", y="bf16"),
        # A small batch of eight users through the 8B up projection, MXFP4 weights.
        dict(name="matvec-batch8-up", op="matvec", tokens=8, n=14336, k=4096, fmt="mxfp4", layout="plain", x="bf16", y="bf16"),
        # Sixteen tokens through an output head: the largest weight of a model, scores in 32 bits.
        dict(name="matvec-batch16-head", op="matvec", tokens=16, n=131072, k=4096, fmt="nvfp4", layout="plain", x="f16", y="f32"),
        # Odd sizes: three tokens, a row count that fills no tile, a width that ends inside one.
        dict(name="matvec-odd", op="matvec", tokens=3, n=1001, k=2064, fmt="ue5m3", layout="plain", x="f16", y="f16"),
        # One user's new token appended: nothing but latency.
        dict(name="append-token", op="append", tokens=1, seqs=0, start=700, heads=32, kv_heads=8, dim=128, rot=128, page=16, type="bf16", interleaved=False, order="nhd"),
        # A batch of users, each one token at a place of its own; half of each head rotated, pairs side by side.
        dict(name="append-batch", op="append", tokens=192, seqs=0, start=4000, heads=16, kv_heads=16, dim=64, rot=32, page=32, type="f16", interleaved=True, order="hnd"),
        # Prompts of three users written in one call, an odd count of tokens.
        dict(name="append-prompts", op="append", tokens=8191, seqs=3, start=0, heads=32, kv_heads=8, dim=128, rot=128, page=64, type="bf16", interleaved=False, order="nhd"),
        # One user early in a conversation: latency again.
        dict(name="attention-short", op="attention", seqs=1, longest=300, ragged=False, heads=32, kv_heads=8, dim=128, page=16, window=0, type="bf16", order="nhd"),
        # One user with a very long context: few rows, a long axis.
        dict(name="attention-long", op="attention", seqs=1, longest=131071, ragged=False, heads=32, kv_heads=8, dim=128, page=64, window=0, type="bf16", order="hnd"),
        # A serving batch with lengths from none to 16384.
        dict(name="attention-batch", op="attention", seqs=64, longest=16384, ragged=True, heads=32, kv_heads=8, dim=128, page=16, window=0, type="bf16", order="nhd"),
        # As many key heads as query heads, small heads, and only the newest 1000 tokens seen.
        dict(name="attention-window", op="attention", seqs=96, longest=5000, ragged=True, heads=16, kv_heads=16, dim=64, page=32, window=1000, type="f16", order="nhd"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["matvec", "append", "attention"])
    if op == "matvec":
        fmt, layout = rng.choice([("nvfp4", "plain"), ("nvfp4", "mma"), ("ue5m3", "plain"), ("ue5m3", "mma"),
                                  ("mxfp4", "plain"), ("mxfp4", "mma"), ("ue5m3_b32", "plain")])
        unit = BLOCK[fmt] if layout == "plain" else 64
        k = _log(rng, 256, 16384) // unit * unit
        x = rng.choice(["bf16", "f16"])
        return dict(op=op, tokens=_log(rng, 1, 24), n=_log(rng, 100, 32768), k=k, fmt=fmt, layout=layout, x=x,
                    y=rng.choice([x, "f32"]))
    kind = rng.choice(["bf16", "f16"])
    order = rng.choice(["nhd", "hnd"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 16])
    if op == "append":
        tokens = _log(rng, 1, 8191)
        tokens = max(1, min(tokens, 8191 * 48 * 128 // (dim * (heads + 2 * kv_heads))))
        seqs = rng.choice([0, min(tokens, rng.choice([1, 2, 5]))]) if tokens <= 256 else rng.choice([1, 2, 5])
        return dict(op=op, tokens=tokens, seqs=seqs, start=rng.randrange(0, 5000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), page=page, type=kind, interleaved=rng.choice([False, True]), order=order)
    seqs = _log(rng, 1, 96)
    longest = min(_log(rng, 1, 131071), CACHE_ELEMENTS * 49 // 100 // (seqs * kv_heads * dim))
    return dict(op=op, seqs=seqs, longest=max(1, longest), ragged=rng.choice([False, True]), heads=heads, kv_heads=kv_heads,
                dim=dim, page=page, window=rng.choice([0, 0, _log(rng, 1, 8192)]), type=kind, order=order)


def _lengths(case):
    """Lengths of the sequences: all the same, or spread from none to the longest."""
    n, longest = case["seqs"], case["longest"]
    if not case["ragged"]:
        return [longest] * n
    return [longest * ((17 * i + n - 1) % n) // max(n - 1, 1) if n > 1 else longest for i in range(n)]


def _seen(case, length):
    return min(length, case["window"]) if case["window"] else length


def work(case):
    if case["op"] == "matvec":
        m, n, k = case["tokens"], case["n"], case["k"]
        out = 4 if case["y"] == "f32" else 2
        return {"bytes": n * k // 2 + n * k // BLOCK[case["fmt"]] + 2 * m * k + out * m * n, "flops": 2 * m * n * k}
    if case["op"] == "append":
        t, h, hk, d, r = (case[a] for a in ("tokens", "heads", "kv_heads", "dim", "rot"))
        places = t if not case["seqs"] else -(-t // case["seqs"])
        return {"bytes": 2 * 2 * t * d * (h + 2 * hk) + 4 * places * r + 8 * t, "flops": 3 * t * r * (h + hk)}
    d, h, hk = case["dim"], case["heads"], case["kv_heads"]
    seen = sum(_seen(case, n) for n in _lengths(case))
    return {"bytes": 2 * 2 * seen * hk * d + 2 * 2 * case["seqs"] * h * d + 4 * seen // case["page"], "flops": 4 * seen * h * d}


# ------------------------------------------------------------------ inputs

def _scale_values(fmt, remapped):
    """The value of each of the 256 scale codes, in 64 bits."""
    c = torch.arange(256, dtype=torch.float64)
    e, m = torch.div(c, 8, rounding_mode="floor"), torch.remainder(c, 8)
    if fmt == "mxfp4":
        return torch.exp2(c - 127)
    if fmt == "nvfp4" or remapped:
        e = torch.remainder(e, 16)
        return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    return torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2(e - 18))


def _tiled(sf):
    """Scale codes [rows][columns] in tiles of 128 rows and 4 columns, line r % 32, word r / 32 of a line."""
    n, c = sf.shape
    full = torch.zeros((-(-n // 128) * 128, -(-c // 4) * 4), dtype=torch.uint8, device=sf.device)
    full[:n, :c] = sf
    return full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _weights(case, gen, dev):
    """A weight ~ N(0, 0.02) in 4 bits with a scale per block, as a checkpoint holds it."""
    n, k, fmt, block = case["n"], case["k"], case["fmt"], BLOCK[case["fmt"]]
    w = torch.randn((n, k), generator=gen, device=dev).mul_(0.02).view(n, k // block, block)
    top = w.abs().amax(-1)
    shift = None
    remapped = fmt.startswith("ue5m3") and case["layout"] == "mma"
    if fmt == "mxfp4":
        s_dec = torch.ones(1, device=dev)
        code = (torch.floor(torch.log2(top)) - 2 + 127).clamp_(0, 254).to(torch.uint8)
    else:
        s_dec = (top.max() / (6 * 448)).reshape(1)
        raw = top / (6 * s_dec)
        if remapped:
            shift = torch.floor(torch.log2(raw.amax(-1))) - 7
            raw = raw * torch.exp2(-shift)[:, None]
        if fmt == "nvfp4" or remapped:
            code = raw.clamp(2.0 ** -6, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            bits = raw.clamp(2.0 ** -14, 61440).half().view(torch.int16).int()
            code = ((bits + 63 + ((bits >> 7) & 1)) >> 7).clamp_(1, 0xF7).to(torch.uint8)
    value = _scale_values(fmt, remapped).float().to(dev)[code.int()] * s_dec
    if shift is not None:
        value = value * torch.exp2(shift)[:, None]
    w /= value[:, :, None]
    q = torch.bucketize(w.abs(), torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev), out_int32=True).to(torch.uint8)
    q |= (w < 0).to(torch.uint8) << 3
    q = q.view(n, k // 2, 2)
    q = q[:, :, 0] | (q[:, :, 1] << 4)
    sf = _tiled(code) if case["layout"] == "mma" else code.contiguous().view(-1)
    return q.contiguous(), sf, s_dec, None if shift is None else shift.to(torch.int8)


def _pages(case, count, gen, dev):
    """Keys and values of `count` pages, indexed [page][place][head][dim] whatever their order in memory."""
    shape = (count, case["page"], case["kv_heads"], case["dim"])
    if case["order"] == "hnd":
        shape = (shape[0], shape[2], shape[1], shape[3])
    made = [torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(TYPES[case["type"]]) for _ in range(2)]
    return [t.transpose(1, 2) for t in made] if case["order"] == "hnd" else made


def _table(need, page, gen, dev):
    """A page table for `need` pages per sequence: pages of the pool in random order."""
    wide = max(1, max(need))
    order = torch.randperm(sum(need) + 1, generator=gen, device=dev).to(torch.int32)
    need = torch.tensor(need, device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(wide, device=dev)
    at = torch.where(col < need[:, None], first[:, None] + col, 0)
    return torch.where(col < need[:, None], order[at], 0).to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "matvec":
        remapped = case["fmt"].startswith("ue5m3") and case["layout"] == "mma"
        s["q"], s["sf"], s["s_dec"], s["shift"] = _weights(case, gen, dev)
        s["x"] = torch.randn((case["tokens"], case["k"]), generator=gen, device=dev).to(TYPES[case["x"]])
        # tables of the plain form: the two values of a byte, the value of a scale code
        one = torch.tensor(E2M1 + tuple(-v for v in E2M1))
        s["pairs"] = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1).to(dev)
        s["scales"] = _scale_values(case["fmt"], remapped).float().to(dev)
        return s
    page, dt = case["page"], TYPES[case["type"]]
    if case["op"] == "append":
        t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        if case["seqs"]:  # prompts: each sequence's tokens in a row
            each = -(-t // case["seqs"])
            i = torch.arange(t, device=dev)
            s["seq"], pos = (i // each).to(torch.int32), case["start"] + i % each
            last, n = case["start"] + each, case["seqs"]
        else:             # one token of each sequence
            s["seq"], n = None, t
            pos = torch.randint(case["start"] // 2, case["start"] + 1, (t,), generator=gen, device=dev)
            last = case["start"] + 1
        s["pos"] = pos.to(torch.int32)
        need = -(-last // page)
        if s["seq"] is None:  # only the last pages of each sequence are at hand: earlier ones hold nothing that is looked at
            s["table"] = torch.randperm(2 * n, generator=gen, device=dev)[:n, None].expand(n, need).to(torch.int32).contiguous()
            count = 2 * n
        else:
            s["table"], count = _table([need] * n, page, gen, dev), need * n + 1
        s["k_pages"], s["v_pages"] = _pages(case, count, gen, dev)
        fused = torch.randn((t, h + 2 * hk, d), generator=gen, device=dev).to(dt)  # one projection gives all three
        s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
        half = case["rot"] // 2
        turn = torch.exp(torch.arange(half, device=dev, dtype=torch.float64) * (-math.log(10000.0) / half))
        angle = torch.arange(last, device=dev, dtype=torch.float64)[:, None] * turn
        s["rope"] = torch.cat([torch.cos(angle), torch.sin(angle)], -1).float()
        return s
    lengths = torch.tensor(_lengths(case), device=dev, dtype=torch.int32)
    s["lengths"] = lengths[torch.randperm(case["seqs"], generator=gen, device=dev)]
    need = [-(-int(n) // page) for n in s["lengths"].tolist()]
    s["table"] = _table(need, page, gen, dev)
    s["k_pages"], s["v_pages"] = _pages(case, sum(need) + 1, gen, dev)
    s["q"] = torch.randn((case["seqs"], case["heads"], case["dim"]), generator=gen, device=dev).to(dt)
    return s


# -------------------------------------------------------------- plain forms

def _matvec_plain(s):
    case, block = s["case"], BLOCK[s["case"]["fmt"]]
    n, k = case["n"], case["k"]
    sf = s["sf"]
    if case["layout"] == "mma":
        c = -(-(k // block) // 4)
        sf = sf.view(-1, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, c * 4)[:n, :k // block]
    scale = s["scales"][sf.reshape(n, k // block, 1).int()]
    if s["shift"] is not None:
        scale = scale * torch.exp2(s["shift"].float())[:, None, None]
    w = (s["pairs"][s["q"].int()].view(n, k // block, block) * scale).view(n, k)
    y = torch.matmul(s["x"].float(), w.t()) * s["s_dec"]
    return y.to(TYPES[case["y"]])


def _rotated_plain(x, cos, sin, case):
    r = case["rot"]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1).to(TYPES[case["type"]])


def _append_plain(s):
    case = s["case"]
    pos, half = s["pos"].long(), case["rot"] // 2
    angle = s["rope"][pos]
    cos, sin = angle[:, None, :half], angle[:, None, half:]
    seq = torch.arange(case["tokens"], device=pos.device) if s["seq"] is None else s["seq"].long()
    page = s["table"][seq, pos // case["page"]].long()
    place = pos % case["page"]
    s["k_pages"][page, place] = _rotated_plain(s["k"], cos, sin, case)
    s["v_pages"][page, place] = s["v"]
    return [_rotated_plain(s["q"], cos, sin, case), s["k_pages"], s["v_pages"]]


def _attention_plain(s):
    case = s["case"]
    b, h, hk, d = case["seqs"], case["heads"], case["kv_heads"], case["dim"]
    table = s["table"].long()
    keys = s["k_pages"][table].reshape(b, -1, hk, d).float()
    values = s["v_pages"][table].reshape(b, -1, hk, d).float()
    q = s["q"].float().view(b, hk, h // hk, d)
    score = torch.einsum("bkgd,blkd->bkgl", q, keys) * d ** -0.5
    at, length = torch.arange(keys.shape[1], device=q.device), s["lengths"].long()[:, None]
    seen = at < length
    if case["window"]:
        seen = seen & (at >= length - case["window"])
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = torch.einsum("bkgl,blkd->bkgd", weight, values) / torch.where(total > 0, total, 1.0)
    return out.view(b, h, d).to(TYPES[case["type"]])


def run(state):
    s = state
    case = s["case"]
    if not own:
        return {"matvec": _matvec_plain, "append": _append_plain, "attention": _attention_plain}[case["op"]](s)
    import fp4_block_scaled_quantize_gb300 as fq
    if case["op"] == "matvec":
        fmt = {"nvfp4": fq.FP4_FMT_NVFP4_B16, "ue5m3": fq.FP4_FMT_UE5M3_B16, "mxfp4": fq.FP4_FMT_MXFP4_B32,
               "ue5m3_b32": fq.FP4_FMT_UE5M3_B32}[case["fmt"]]
        w = fq.Quantized(s["q"], s["sf"], s["s_dec"], s["shift"], fmt,
                         fq.FP4_SF_MMA if case["layout"] == "mma" else fq.FP4_SF_PLAIN)
        return fq.matvec(s["x"], w, out_dtype=TYPES[case["y"]])
    if case["op"] == "append":
        q = fq.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["pos"], seq=s["seq"], q=s["q"],
                         rope=s["rope"], interleaved=case["interleaved"])
        return [q, s["k_pages"], s["v_pages"]]
    return fq.decode_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], window=case["window"])


# ------------------------------------------------------- definitions, 64 bits

def _exact_scales(s, rows):
    """Scales of some rows of a weight by the formats' definitions, in 64 bits."""
    case = s["case"]
    cols = case["k"] // BLOCK[case["fmt"]]
    r, c = rows[:, None], torch.arange(cols, device=rows.device)
    if case["layout"] == "mma":
        at = ((r // 128) * (-(-cols // 4)) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    else:
        at = r * cols + c
    code = s["sf"][at].double()
    if case["fmt"] == "mxfp4":
        return torch.exp2(code - 127)
    e5 = case["fmt"].startswith("ue5m3") and case["layout"] == "plain"
    e, m = torch.floor(code / 8), code % 8
    bias = 15 if e5 else 7
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - bias), m / 8 * 2.0 ** (1 - bias))
    if s["shift"] is not None:
        v = v * torch.exp2(s["shift"][rows].double())[:, None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        n, k, block = case["n"], case["k"], BLOCK[case["fmt"]]
        x, parts = s["x"].double(), []
        for i in range(0, n, 4096):
            rows = torch.arange(i, min(n, i + 4096), device=x.device)
            byte = s["q"][rows]
            code = torch.stack([byte & 15, byte >> 4], -1).view(len(rows), k).double()
            mag = code % 8
            e, m = torch.floor(mag / 2), mag % 2
            v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
            w = torch.where(code >= 8, -v, v).view(len(rows), -1, block) * _exact_scales(s, rows)[:, :, None]
            parts.append(x @ w.view(len(rows), k).t())
        return torch.cat(parts, 1) * s["s_dec"].double()
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

        keys, values = s["k_pages"].double(), s["v_pages"].double()
        seq = torch.arange(case["tokens"], device=pos.device) if s["seq"] is None else s["seq"].long()
        page = s["table"][seq, pos // case["page"]].long()
        keys[page, pos % case["page"]] = turned(s["k"])
        values[page, pos % case["page"]] = s["v"].double()
        return [turned(s["q"]), keys, values]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    group = case["heads"] // case["kv_heads"]
    for i, length in enumerate(s["lengths"].tolist()):
        if length == 0:
            continue
        at = torch.arange(length - _seen(case, length), length, device=out.device)
        page, place = s["table"][i, at // case["page"]].long(), at % case["page"]
        for j in range(case["kv_heads"]):
            keys, values = s["k_pages"][page, place, j].double(), s["v_pages"][page, place, j].double()
            w = torch.softmax(s["q"][i, j * group:(j + 1) * group].double() @ keys.t() / math.sqrt(case["dim"]), -1)
            out[i, j * group:(j + 1) * group] = w @ values
    return out
