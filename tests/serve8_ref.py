"""Plain 64-bit definitions of the operators around a cache in 8 bits, for
their tests (torch and Python on the CPU; none of the library's code)."""
import math

import torch

from serve_ref import rotate

E4M3 = torch.float8_e4m3fn


def nearest_e4m3(x):
    """The nearest E4M3 value of 64-bit numbers up to 448 in magnitude, ties to
    the even one; NaN and infinities give NaN."""
    finite = torch.isfinite(x)
    y = torch.where(finite, x, 0.0)
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    y = torch.round(y / step) * step
    return torch.where(finite, y, torch.nan)


def need_code(top):
    """E8M0 code of the smallest power of two u >= 2^-127 with top <= 448 u."""
    if top == 0:
        return 0
    e = max(-127, math.frexp(top / 448)[1] - 1)
    while math.ldexp(448.0, e) < top:
        e += 1
    return e + 127


class Cache8:
    """Codes (as their E4M3 values) and scale codes of a cache, as tensors
    k, v [pages, page, heads, dim] (64 bits) and ks, vs [pages, blocks, heads]."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v = (t.cpu().float().double() for t in (k, v))
        self.ks, self.vs = (t.cpu().long() for t in (ks, vs))
        self.page, self.block = k.shape[1], k.shape[1] // ks.shape[1]

    def append(self, k, v, table, pos, seq, rope, interleaved):
        """The definition of fp4_kv_append8; returns what of the bounds
        |a cos| + |b sin| belongs to each stored key."""
        table = table.cpu()
        x, mag = rotate(k, rope, pos, interleaved)
        v = v.cpu().double()
        T = len(pos)
        seq = list(range(T)) if seq is None else seq.tolist()
        pos = pos.tolist()
        groups = {}
        for t in range(T):
            s, p = seq[t], pos[t]
            if p < 0 or not 0 <= s < table.shape[0] or p >= table.shape[1] * self.page:
                continue
            if rope is not None and p >= rope.shape[0]:
                continue
            n = int(table[s, p // self.page])
            if not 0 <= n < self.k.shape[0]:
                continue
            groups.setdefault((n, p % self.page // self.block), []).append((t, p % self.page))
        for (n, b), places in groups.items():
            for codes, scales, src in ((self.k, self.ks, x), (self.v, self.vs, v)):
                for h in range(codes.shape[2]):
                    new = torch.stack([src[t, h] for t, _ in places])
                    top = torch.where(torch.isfinite(new), new.abs(), 0.0).max().item()
                    old, code = int(scales[n, b, h]), need_code(top)
                    at = [p for _, p in places]
                    if b * self.block not in at:
                        code = max(code, old)
                        rest = [p for p in range(b * self.block, (b + 1) * self.block) if p not in at]
                        if code > old and rest:
                            codes[n, rest, h] = nearest_e4m3(codes[n, rest, h] * 2.0 ** (old - code))
                    codes[n, at, h] = nearest_e4m3(new * 2.0 ** (127 - code))
                    scales[n, b, h] = code
        return mag

    def units(self, which):
        scales = self.ks if which == "k" else self.vs
        return torch.where(scales == 255, math.nan, torch.exp2((scales - 127).double())).repeat_interleave(self.block, 1)

    def values(self, which):
        return (self.k if which == "k" else self.v) * self.units(which)[..., None]


def seen_positions(length, window, sinks):
    return [j for j in range(length) if not window or j >= length - window or j < sinks]


def attention(q, k, v, table, lengths, scale, window, sinks, units=None):
    """(out, sum of weighted |v|, lse, largest sum |q k| scale per row) over
    caches of 64-bit values k, v [pages, page, heads, dim].  With the values'
    units [pages, page, heads] also the sum of |code| times the largest of
    weight times unit."""
    q, table = q.cpu().double(), table.cpu().long()
    S, H, D = q.shape
    P, Hk = k.shape[1], k.shape[2]
    G = H // Hk
    out, wv = torch.zeros_like(q), torch.zeros_like(q)
    floor = torch.zeros_like(q)
    lse, mag = torch.full((S, H), -math.inf, dtype=torch.float64), torch.zeros(S, H, dtype=torch.float64)
    for s, n in enumerate(lengths.tolist()):
        at = torch.tensor(seen_positions(n, window, sinks), dtype=torch.long)
        if not len(at):
            continue
        page, place = table[s, at // P], at % P
        ks, vs = k[page, place], v[page, place]
        qs = q[s].view(Hk, G, D)
        score = torch.einsum("kgd,nkd->kgn", qs, ks) * scale
        lse[s] = torch.logsumexp(score, -1).reshape(H)
        lse[s][~torch.isfinite(q[s]).all(-1)] = math.nan  # as the header has it
        w = torch.softmax(score, -1)
        out[s] = torch.einsum("kgn,nkd->kgd", w, vs).reshape(H, D)
        wv[s] = torch.einsum("kgn,nkd->kgd", w, vs.abs()).reshape(H, D)
        mag[s] = (torch.einsum("kgd,nkd->kgn", qs.abs(), ks.abs()).amax(-1) * abs(scale)).reshape(H)
        if units is not None:
            u = units[page, place]
            most = torch.nan_to_num(w * u.t()[:, None]).amax(-1)
            floor[s] = (most[..., None] * torch.nan_to_num(vs / u[..., None]).abs().sum(0)[:, None]).reshape(H, D)
    return (out, wv, lse, mag) if units is None else (out, wv, lse, mag, floor)


class Pages:
    """The definition of fp4_page_plan on lists."""

    def __init__(self, lengths, table, room, pool, page):
        self.lengths, self.room = lengths.tolist(), room.tolist()
        self.table = table.tolist()
        pool = pool.tolist()
        self.free, self.page, self.pages = pool[2:2 + pool[0]], page, len(pool) - 2
        self.wide = table.shape[1]

    def plan(self, new, tokens=None):
        """(seq, pos, slot, offsets) or None, and whether a sequence was refused."""
        P, seqs = self.page, len(new)
        pages, back, refused = 0, [], False
        seq, pos, slot, offsets = [], [], [], [0]
        given = []
        for s, n in enumerate(new):
            L, held = self.lengths[s], self.room[s] // P
            after = max(L + n, 0)
            want = -(-after // P)
            offsets.append(offsets[-1] + max(n, 0))
            if n < 0:
                back += [self.table[s][e] for e in range(want, held)]
                for e in range(want, held):
                    self.table[s][e] = -1
                self.lengths[s], self.room[s] = after, min(want, held) * P
                continue
            ok = want <= self.wide and (tokens is None or offsets[-1] <= tokens)
            grow = max(want - held, 0) if ok else 0
            pages += grow
            ok = ok and (grow == 0 or pages <= len(self.free))
            refused |= not ok
            if ok:
                for e in range(grow):
                    self.table[s][held + e] = self.free[len(self.free) - 1 - (pages - grow + e)]
                    given.append(self.table[s][held + e])
                self.lengths[s], self.room[s] = after, (held + grow) * P
            for j in range(n if tokens is not None else 0):
                seq.append(s)
                pos.append(L + j if ok else -1)
                slot.append(self.table[s][(L + j) // P] * P + (L + j) % P if ok else -1)
        self.free = self.free[:len(self.free) - len(given)] + back[::-1]
        if tokens is None:
            return None, refused
        pad = lambda v: (v + [-1] * tokens)[:tokens]  # noqa: E731
        return (pad(seq), pad(pos), pad(slot), offsets), refused
