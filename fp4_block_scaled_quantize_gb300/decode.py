"""Token-by-token attention layer on FP4 weights: the path from a hidden state
to the layer's output through the serving operators.

    qkv  = x W_qkv^T               matvec (4-bit weight, 16-bit activations)
    cache <- rotate(k), v          kv_append (queries rotated on the way)
    a    = softmax(q k^T) v        decode_attention over the paged cache
    y    = a W_o^T                 matvec

``PagedCache`` owns the pages, hands them out to sequences and keeps the page
table and the lengths on the device; ``FP4DecodeAttention`` holds the two
weights as the FP4 copies that training's GEMMs read (tensor-core scale
layout, 2D tiles), so a weight trained with ``FP4Linear`` serves as it was
trained.  A step waits for nothing on the host and allocates its results, the
tensors between the calls and attention's workspace from torch's pool alone, so
it can be captured in a CUDA graph once the pages it needs are reserved.
"""
import torch

from . import (FP4_FMT_UE5M3_B16, FP4_SF_MMA, Quantized, amax, decode_attention, kv_append, matvec,
               params, quantize, rope_table)


class PagedCache:
    """Keys and values of up to `seqs` sequences in `pages` pages of
    `page_size` places.  Pages are taken from a list on the host by
    ``reserve`` and given back by ``release``; ``table`` [seqs, max_pages]
    (-1 where a sequence has no page), ``room`` [seqs] (the positions its pages
    hold) and ``lengths`` [seqs], all int32, live on the device."""

    def __init__(self, seqs, max_len, kv_heads, head_dim, pages=None, page_size=64,
                 dtype=torch.bfloat16, device="cuda"):
        if min(seqs, max_len, kv_heads, head_dim, page_size) < 1:
            raise ValueError("PagedCache: sizes must be positive")
        wide = -(-max_len // page_size)
        pages = seqs * wide if pages is None else int(pages)
        shape = (pages, page_size, kv_heads, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        self.table = torch.full((seqs, wide), -1, dtype=torch.int32, device=device)
        self.room = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.page_size, self.max_len = page_size, max_len
        self.places = wide * page_size  # that a sequence's row of the table can name
        self._free = list(range(pages - 1, -1, -1))
        self._owned = [[] for _ in range(seqs)]

    def reserve(self, lengths):
        """Pages for sequence s up to lengths[s] positions (those it has
        stay); raises without a change if there are too few."""
        if len(lengths) != len(self._owned):
            raise ValueError("PagedCache.reserve: one length per sequence")
        if any(n > self.max_len for n in lengths):
            raise ValueError(f"PagedCache.reserve: at most {self.max_len} positions a sequence")
        need = [max(0, -(-n // self.page_size) - len(o)) for n, o in zip(lengths, self._owned)]
        if sum(need) > len(self._free):
            raise RuntimeError(f"PagedCache: {sum(need)} pages needed, {len(self._free)} free")
        for s, n in enumerate(need):
            if not n:
                continue
            new = [self._free.pop() for _ in range(n)]
            at = len(self._owned[s])
            self._owned[s] += new
            self.table[s, at:at + n] = torch.tensor(new, dtype=torch.int32)
            self.room[s] = (at + n) * self.page_size

    def release(self, seq):
        """Gives the pages of a sequence back, takes them out of the table and
        sets its length to zero."""
        self._free += reversed(self._owned[seq])
        self._owned[seq] = []
        self.table[seq] = -1
        self.room[seq] = 0
        self.lengths[seq] = 0


_PARTS = ("q", "sf", "s_dec", "row_shift")


def _weight(name):
    """A Quantized copy whose parts are buffers of the module, so that they
    are saved, loaded and moved with it."""
    def get(self):
        b = self._buffers
        return Quantized(*(b[f"{name}_{part}"] for part in _PARTS), *self._forms[name])

    def put(self, w):
        for part in _PARTS:
            self.register_buffer(f"{name}_{part}", getattr(w, part))
        self._forms[name] = (w.format, w.sf_layout)

    return property(get, put)


class FP4DecodeAttention(torch.nn.Module):
    """Attention layer for decoding: heads query heads over kv_heads key heads
    of head_dim, rotated over rot_dim elements (default: all; 0: none) by
    positions up to max_len.  w_qkv [(heads + 2 kv_heads) head_dim, hidden] and w_o [hidden,
    heads head_dim] are bfloat16 weights, quantised once, or Quantized
    copies."""

    w_qkv, w_o = _weight("w_qkv"), _weight("w_o")

    def __init__(self, w_qkv, w_o, heads, kv_heads, head_dim, max_len, rot_dim=None, base=10000.0,
                 window=0, interleaved=False, format=FP4_FMT_UE5M3_B16):
        super().__init__()
        if heads % kv_heads:
            raise ValueError("FP4DecodeAttention: heads must be a multiple of kv_heads")
        p = params(format=format, block2d=True, sf_layout=FP4_SF_MMA)  # as a linear layer's weight
        self._forms = {}
        self.w_qkv, self.w_o = (w if isinstance(w, Quantized) else self.quantized(w, p)
                                for w in (w_qkv, w_o))
        if self.w_qkv.rows != (heads + 2 * kv_heads) * head_dim or self.w_o.k != heads * head_dim:
            raise ValueError("FP4DecodeAttention: the weights do not fit the heads")
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.window, self.interleaved = window, interleaved
        rot_dim = head_dim if rot_dim is None else rot_dim
        rope = rope_table(max_len, rot_dim, base, self.w_qkv.q.device) if rot_dim else None
        self.register_buffer("rope", rope, persistent=False)

    def get_extra_state(self):
        """Format and scale layout of the two weights."""
        return torch.tensor([self._forms["w_qkv"], self._forms["w_o"]])

    def set_extra_state(self, state):
        self._forms = dict(zip(("w_qkv", "w_o"), map(tuple, state.tolist())))

    @staticmethod
    def quantized(w, p):
        """The copy of a weight with producer options p, by its current amax."""
        w = w.detach().to(torch.bfloat16).contiguous()
        return quantize(w, amax(w)[0], p)

    @classmethod
    def from_linear(cls, qkv, o, heads, kv_heads, head_dim, max_len, **kw):
        """From two FP4Linear layers: the copies their GEMMs multiply."""
        return cls(cls.quantized(qkv.weight, qkv.p_w), cls.quantized(o.weight, o.p_w), heads, kv_heads,
                   head_dim, max_len, **kw)

    def forward(self, x, cache, pos=None):
        """One new token of every sequence: x [seqs, hidden] at positions pos
        (default: the cache's lengths).  Returns [seqs, hidden] and advances the
        cache's lengths.  A sequence at position -1 is left out of the step: it
        keeps its length, and its row of the result is zero.  Where a sequence
        has no page for its position, or the rotation ends before it, nothing is
        stored, its length stays (at most the room of its pages), its row of the
        result means nothing and fp4_status_sync reports FP4_ERR_INVALID_ARG."""
        n, rope, given = len(cache._owned), self.rope, pos is not None
        if x.dim() != 2 or x.shape[0] != n:
            raise ValueError(f"FP4DecodeAttention: x must be [{n}, hidden], a token of every sequence of the cache")
        if not given:
            pos = cache.lengths
        elif pos.shape != (n,) or pos.dtype != torch.int32 or pos.device != cache.lengths.device:
            raise ValueError(f"FP4DecodeAttention: pos must be {n} int32 positions beside the cache")
        after = pos + 1
        qkv = matvec(x, self.w_qkv).view(n, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = kv_append(k, v, cache.k, cache.v, cache.table, pos, q=q, rope=rope, interleaved=self.interleaved)
        seen = torch.minimum(after, cache.room, out=None if given else cache.lengths)
        if rope is not None and cache.places > rope.shape[0]:
            seen.clamp_(max=rope.shape[0])
        if given:  # what is left out sees nothing and keeps its length
            seen.clamp_(min=0)
            cache.lengths.copy_(torch.where(pos < 0, cache.lengths, seen))
        a = decode_attention(q, cache.k, cache.v, cache.table, seen, window=self.window)
        return matvec(a.view(n, -1), self.w_o)

    def prefill(self, x, cache, seq, pos):
        """Prompt tokens x [tokens, hidden] of sequences seq at positions pos:
        their keys and values into the cache (queries and outputs of prompts
        belong to another kernel).  The caller sets the lengths."""
        qkv = matvec(x, self.w_qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.head_dim)
        k, v = qkv[:, self.heads:self.heads + self.kv_heads], qkv[:, self.heads + self.kv_heads:]
        kv_append(k, v, cache.k, cache.v, cache.table, pos, seq=seq, rope=self.rope,
                  interleaved=self.interleaved)


__all__ = ["FP4DecodeAttention", "PagedCache"]
