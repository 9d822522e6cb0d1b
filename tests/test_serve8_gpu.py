"""The operators around a cache in 8 bits on the GPU against their definitions
in 64 bits (serve8_ref.py).

Values and their keys' rotations by cosines and sines of few bits are exact in
binary32, so codes and scales have to be those of the definition, and so do
indexes.  Tolerances elsewhere, derived from the arithmetic (u: half a unit in
the last place of the output type, binary32 sums throughout):
  rotation   r = 2^-22 (|a cos| + |b sin|): three binary32 roundings.  Stored in
             8 bits: half a step of E4M3, 2^-4 of the value or 2^-10 of the unit
             (the scale), on top; where the largest is within r of a power of
             two times 448 the unit may be the next one
  attention  a score is off by d = (D/16 + 8) 2^-23 max sum |q k| scale (sums of
             exact products; powers of two cost nothing, three roundings of the
             factors are in the 8), which changes a weight and the sum by the
             factor 1 +- d each; exponentials, weights as two 16-bit parts and
             exponents up to 2^7 added to scores 2^-14 together; the sum over L
             positions a rounding per 16 products and per join:
             (4 d + 2^-14 + (L/16 + 32) 2^-23) sum w |v| + 2 u |out|
             A weight times its value's unit is held, 2^7 or more times as large
             relative to the row's largest, as two f16 parts, of which the second
             is off by half of f16's smallest, 2^-25: 2^-32 of the largest, for
             each position.  Where only small weights meet values that are not
             zero this is what counts: + 2^-32 max(w unit) sum |code|
"""
import math

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from serve8_ref import E4M3, Cache8, Pages, attention
from serve_ref import HALF_ULP, TINY, rotate

pytestmark = pytest.mark.gpu

BF, HF, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


@pytest.fixture(autouse=True)
def _clean_status():
    need_gpu()
    fq.fp4_status_sync()
    yield


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol) & ~(torch.isnan(got) & torch.isnan(want))
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                             f"{got[i]} for {want[i]}, tolerance {tol[i]}")


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def ordered(t, hnd):
    """The same [pages, page, heads, ...] tensor with heads outermost in memory."""
    return t.transpose(1, 2).contiguous().transpose(1, 2) if hnd else t


def cache8(pages, page, block, heads, dim, seed=0, hnd=False, lo=118, hi=132):
    """Random codes (no NaN) and scales over some binades."""
    g = gen(seed)
    out = []
    for _ in range(2):
        code = torch.randint(0, 256, (pages, page, heads, dim), generator=g, dtype=I32)
        code = torch.where(code & 127 == 127, code - 1, code).to(torch.uint8)
        out.append(ordered(code.cuda(), hnd).view(E4M3))
    for _ in range(2):
        s = torch.randint(lo, hi, (pages, page // block, heads), generator=g, dtype=I32).to(torch.uint8)
        out.append(ordered(s.cuda(), hnd))
    return out  # k, v, k_scale, v_scale


def tables(need, pages, seed=0, wide=0):
    """Tables of `need` pages a sequence, distinct pages in random order; -1 behind."""
    order = torch.randperm(pages, generator=gen(seed)).tolist()
    wide = max(wide, *need, 1)
    return ints([[order.pop() for _ in range(n)] + [-1] * (wide - n) for n in need])


def check_cache(got, ref, what=""):
    """Codes and scales equal the reference's (NaN codes by being NaN)."""
    k, v, ks, vs = got
    for name, t, want in (("k", k, ref.k), ("v", v, ref.v)):
        t = t.cpu().float().double()
        assert torch.equal(torch.isnan(t), torch.isnan(want)), (what, name)
        t, want = torch.nan_to_num(t), torch.nan_to_num(want)
        if not torch.equal(t, want):
            i = tuple(torch.nonzero(t != want)[0].tolist())
            raise AssertionError(f"{what} {name}: {int((t != want).sum())} codes differ, first at {i}: {t[i]} for {want[i]}")
    assert torch.equal(ks.cpu().long(), ref.ks), (what, "key scales")
    assert torch.equal(vs.cpu().long(), ref.vs), (what, "value scales")


def exact_rope(positions, rot):
    """Cosines and sines of few bits: rotations by them are exact in binary32."""
    c = torch.randint(-4, 5, (positions, rot), generator=gen(99)).float() / 4
    return c.cuda()


def few_bits(shape, dtype, seed, scale=1.0):
    """Values of 6 bits over a dozen binades (exact in products with 1/4ths)."""
    g = gen(seed)
    m = torch.randint(-63, 64, shape, generator=g).float()
    e = torch.randint(-8, 3, shape, generator=g).float()
    return (m * torch.exp2(e) * scale).to(dtype).cuda()


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,dim,rot,inter", [(2, 64, 64, False), (1, 80, 32, False), (8, 128, 128, True), (3, 16, 16, False),
                                                 (2, 256, 128, False), (2, 192, 24, True), (2, 48, 0, False)])
@pytest.mark.parametrize("page,block,hnd", [(16, 16, False), (24, 8, True), (8, 1, False), (64, 64, True), (12, 4, False)])
def test_append_prompts_then_tokens(dtype, heads, dim, rot, inter, page, block, hnd):
    """Ragged prompts in one call, more of them that begin inside blocks, then
    single tokens whose sizes rise: codes and scales of every place."""
    need = [-(-n // page) for n in (70, 3, 41)]
    k, v, ks, vs = cache8(sum(need) + 2, page, block, heads, dim, seed=dim, hnd=hnd)
    table = tables(need, sum(need) + 2, seed=page)
    ref = Cache8(k, v, ks, vs)
    rope = exact_rope(80, rot) if rot else None
    done = [0, 0, 0]
    for call, n in enumerate(([33, 1, 9], [21, 0, 32], [5, 1, 0], [1, 1, 0], [1, 0, 0], [1, 0, 0])):
        seq = ints([s for s in range(3) for _ in range(n[s])])
        pos = ints([done[s] + j for s in range(3) for j in range(n[s])])
        done = [a + b for a, b in zip(done, n)]
        T = len(seq)
        x = few_bits((T, heads * 3, dim), dtype, seed=call, scale=2.0 ** call)
        q, kn, vn = x[:, :heads], x[:, heads:2 * heads], x[:, 2 * heads:]
        qo = fq.kv_append(kn, vn, k, v, table, pos, seq=seq, q=q, rope=rope, interleaved=inter, k_scale=ks, v_scale=vs)
        ref.append(kn, vn, table, pos.cpu(), seq.cpu(), rope, inter)
        check_cache((k, v, ks, vs), ref, f"call {call}")
        want, mag = rotate(q, rope, pos, inter)
        close(qo, want, 2.0 ** -22 * mag + 2 * HALF_ULP[dtype] * want.abs() + 2 * TINY[dtype], "queries")
    assert fq.fp4_status_sync() == fq.FP4_OK


def test_append_one_token_of_each_sequence():
    """Without seq: 300 sequences, a token each, some left out."""
    k, v, ks, vs = cache8(301, 16, 8, 2, 64)
    table = tables([1] * 300, 301)
    ref = Cache8(k, v, ks, vs)
    pos = torch.randint(-1, 16, (300,), generator=gen(1)).to(I32).cuda()
    x = few_bits((300, 4, 64), BF, 2, 16.0)
    rope = exact_rope(16, 64)
    fq.kv_append(x[:, :2], x[:, 2:], k, v, table, pos, rope=rope, k_scale=ks, v_scale=vs)
    ref.append(x[:, :2], x[:, 2:], table, pos.cpu(), None, rope, False)
    check_cache((k, v, ks, vs), ref)
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("page,block", [(16, 16), (128, 128), (96, 32), (40, 20)])
def test_append_many_prompt_tokens(page, block):
    """Blocks that begin and end anywhere in the lists that warps look at."""
    n = [1000, 37, 0, 511, 64]
    need = [-(-(a + 5) // page) for a in n]
    k, v, ks, vs = cache8(sum(need), page, block, 2, 32, seed=page)
    table = tables(need, sum(need), seed=3)
    ref = Cache8(k, v, ks, vs)
    seq = ints([s for s in range(5) for _ in range(n[s])])
    pos = ints([5 + j for s in range(5) for j in range(n[s])])
    x = few_bits((len(seq), 4, 32), HF, 4)
    fq.kv_append(x[:, :2], x[:, 2:], k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
    ref.append(x[:, :2], x[:, 2:], table, pos.cpu(), seq.cpu(), None, False)
    check_cache((k, v, ks, vs), ref)
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("rot,inter", [(64, False), (34, False), (6, True), (20, True), (16, False)])
def test_append_odd_rows(rot, inter):
    """Rows at odd addresses and strides, rotations that fill no piece."""
    k, v, ks, vs = cache8(6, 16, 16, 2, 64)
    table = tables([3, 3], 6)
    ref = Cache8(k, v, ks, vs)
    seq, pos = ints([0] * 20 + [1] * 13), ints(list(range(20)) + list(range(30, 43)))
    flat = few_bits((33 * 525 + 3,), BF, 5)
    x = flat[3:].as_strided((33, 8, 64), (525, 65, 1))
    rope = exact_rope(48, rot)
    qo = fq.kv_append(x[:, :2], x[:, 2:4], k, v, table, pos, seq=seq, q=x[:, 4:], rope=rope, interleaved=inter, k_scale=ks,
                      v_scale=vs)
    ref.append(x[:, :2], x[:, 2:4], table, pos.cpu(), seq.cpu(), rope, inter)
    check_cache((k, v, ks, vs), ref)
    want, mag = rotate(x[:, 4:], rope, pos, inter)
    close(qo, want, 2.0 ** -22 * mag + 2 * HALF_ULP[BF] * want.abs() + 2 * TINY[BF], "queries")


def test_append_extremes():
    """Zeros, BF16's largest and smallest, infinities and NaN: they stay where
    they are, and the rest keeps its accuracy."""
    k, v, ks, vs = cache8(2, 16, 4, 1, 16)
    table = ints([[0, 1]])
    ref = Cache8(k, v, ks, vs)
    x = few_bits((16, 2, 16), BF, 6)
    x[0:4] = 0
    x[4, 0, 0], x[5, 1, 3], x[6, 0, 7] = math.inf, -math.inf, math.nan
    x[8, 0, 1], x[9, 1, 2] = 3.3e38, -3.3e38
    x[12:16] *= 2.0 ** -130
    seq, pos = ints([0] * 16), ints(list(range(16)))
    fq.kv_append(x[:, :1], x[:, 1:], k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
    ref.append(x[:, :1], x[:, 1:], table, pos.cpu(), seq.cpu(), None, False)
    check_cache((k, v, ks, vs), ref)
    for p, scale in ((2, 1e-30), (3, 1e30), (1, 1.0), (0, 1.0)):  # rises, and a block begun anew
        y = few_bits((1, 2, 16), BF, p) * scale
        fq.kv_append(y[:, :1], y[:, 1:], k, v, table, ints([p]), seq=ints([0]), k_scale=ks, v_scale=vs)
        ref.append(y[:, :1], y[:, 1:], table, torch.tensor([p]), torch.tensor([0]), None, False)
        check_cache((k, v, ks, vs), ref, f"place {p}")


def test_append_by_angles():
    """Ordinary rotations: half a step of the codes on top of binary32's."""
    k, v, ks, vs = cache8(40, 16, 16, 4, 128)
    table = tables([40], 40)
    ref = Cache8(k, v, ks, vs)
    T = 600
    x = torch.randn(T, 8, 128, generator=gen(7)).to(BF).cuda()
    rope = fq.rope_table(700, 128)
    seq, pos = ints([0] * T), ints(list(range(16, T + 16)))
    fq.kv_append(x[:, :4], x[:, 4:], k, v, table, pos, seq=seq, rope=rope, k_scale=ks, v_scale=vs)
    mag = ref.append(x[:, :4], x[:, 4:], table, pos.cpu(), seq.cpu(), rope, False)
    want, _ = rotate(x[:, :4], rope, pos, False)
    kk, vv = fq.kv_read(k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
    unit = torch.exp2(ks.cpu().double() - 127)[table[0].cpu().long()[pos.cpu().long() // 16], 0][:, :, None]
    close(kk, want, (2.0 ** -22 * mag) * 1.1 + torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * unit), "keys")
    assert torch.equal(vs.cpu().long(), ref.vs)
    close(vv, ref.values("v")[table[0].cpu().long()[pos.cpu().long() // 16], pos.cpu().long() % 16], torch.zeros(T, 4, 128), "values")


def test_append_leaves_out_what_has_no_place():
    k, v, ks, vs = cache8(4, 16, 8, 1, 32)
    before = [t.clone() for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
    table = ints([[0, 9], [-1, 2]])  # page 9 does not exist
    x = few_bits((6, 3, 32), BF, 8)
    seq, pos = ints([0, 1, 2, -1, 0, 1]), ints([16, 3, 0, 0, 32, 31])
    rope = exact_rope(31, 32)  # ends before position 31
    qo = fq.kv_append(x[:, :1], x[:, 1:2], k, v, table, pos, seq=seq, q=x[:, 2:], rope=rope, k_scale=ks, v_scale=vs)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, (k.view(torch.uint8), v.view(torch.uint8), ks, vs)))
    assert not qo.any()
    fq.kv_append(x[:, :1], x[:, 1:2], k, v, table, ints([-1] * 6), seq=seq, k_scale=ks, v_scale=vs)
    assert fq.fp4_status_sync() == fq.FP4_OK
    assert all(torch.equal(a, b) for a, b in zip(before, (k.view(torch.uint8), v.view(torch.uint8), ks, vs)))


def test_append_general_way_gives_the_same_bits():
    """A given stream and output, queries turned in place."""
    a, b = cache8(5, 16, 16, 2, 64), cache8(5, 16, 16, 2, 64)
    table = tables([2, 2], 5)
    x = torch.randn(20, 8, 64, generator=gen(9)).to(HF).cuda()
    seq, pos = ints([0] * 12 + [1] * 8), ints(list(range(3, 15)) + list(range(8)))
    rope = fq.rope_table(32, 64)
    q1 = fq.kv_append(x[:, :2], x[:, 2:4], a[0], a[1], table, pos, seq=seq, q=x[:, 4:], rope=rope, k_scale=a[2], v_scale=a[3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fq.kv_append(x[:, :2], x[:, 2:4], b[0], b[1], table, pos, seq=seq, q=x[:, 4:], rope=rope, q_out=x[:, 4:], stream=s,
                 k_scale=b[2], v_scale=b[3])
    s.synchronize()
    assert torch.equal(q1, x[:, 4:])
    assert all(torch.equal(m.view(torch.uint8), n.view(torch.uint8)) for m, n in zip(a, b))


# --------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page,block,hnd", [(16, 16, False), (24, 8, True), (5, 1, False)])
@pytest.mark.parametrize("heads,dim", [(1, 16), (3, 80), (8, 128), (2, 256)])
def test_read(dtype, page, block, hnd, heads, dim):
    k, v, ks, vs = cache8(9, page, block, heads, dim, hnd=hnd)
    table = tables([4, 4], 9)
    ref = Cache8(k, v, ks, vs)
    seq = torch.randint(0, 2, (77,), generator=gen(1)).to(I32)
    pos = torch.randint(-1, 4 * page, (77,), generator=gen(2)).to(I32)
    got = fq.kv_read(k, v, table, pos.cuda(), seq=seq.cuda(), k_scale=ks, v_scale=vs, dtype=dtype)
    at = pos.clamp(min=0).long()
    page_of = table.cpu().long()[seq.long(), at // page]
    for t, which in zip(got, "kv"):
        want = ref.values(which)[page_of, at % page] * (pos >= 0)[:, None, None]
        assert t.dtype == dtype
        close(t, want, torch.zeros_like(want) if dtype == BF else 2.0 ** -11 * want.abs() + 2.0 ** -25, which)
    # a cache in 16 bits: its own rows
    kp, vp = (ordered(torch.randn(9, page, heads, dim, generator=gen(i)).to(dtype).cuda(), hnd) for i in (3, 4))
    for t, p in zip(fq.kv_read(kp, vp, table, pos.cuda(), seq=seq.cuda()), (kp, vp)):
        assert torch.equal(t.cpu(), p.cpu()[page_of, at % page] * (pos >= 0)[:, None, None])
    assert fq.fp4_status_sync() == fq.FP4_OK


def test_read_what_has_no_place():
    k, v, ks, vs = cache8(4, 16, 16, 2, 32)
    k.view(torch.uint8)[1, 3, 0, 5], ks[2, 0, 1] = 0x7F, 255
    table = ints([[0, 9], [1, 2]])
    seq, pos = ints([0, 1, 2, -1, 0, 1, 1]), ints([16, 99, 0, 0, 0, 3, 16])
    s = torch.cuda.Stream()
    a = fq.kv_read(k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    s.wait_stream(torch.cuda.current_stream())
    b = fq.kv_read(k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs, stream=s)
    s.synchronize()
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))
    assert not a[0][:4].any() and not a[1][:4].any() and a[0][4].any()
    nan = torch.isnan(a[0])
    assert nan[5].sum() == 1 and nan[5, 0, 5] and nan[6, 1].all() and not nan[6, 0].any()
    fq.fp4_status_sync()


# ---------------------------------------------------------------- attention

def check_attention(q, cache, table, lengths, window=0, sinks=0, scale=None, **kw):
    k, v, ks, vs = cache
    units = None
    if ks is None:
        kk, vv = k.cpu().double(), v.cpu().double()
    else:
        ref = Cache8(k, v, ks, vs)
        kk, vv, units = ref.values("k"), ref.values("v"), ref.units("v")
    S, H, D = q.shape
    scale_ = D ** -0.5 if scale is None else scale
    want, wv, lse, mag, *floor = attention(q, kk, vv, table, lengths.cpu(), scale_, window, sinks, units)
    if "stream" not in kw:  # the ordinary way, then the general one: the same bits
        first = fq.decode_attention(q, k, v, table, lengths, scale=scale, window=window, sinks=sinks, k_scale=ks, v_scale=vs)
    out, got_lse = fq.decode_attention(q, k, v, table, lengths, scale=scale, window=window, sinks=sinks, k_scale=ks, v_scale=vs,
                                       return_lse=True, **kw)
    if "stream" not in kw:
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    d = ((D / 16 + 8) * 2.0 ** -23 * mag)[:, :, None]
    L = max([1] + lengths.tolist())
    tol = (4 * d + 2.0 ** -14 + (L / 16 + 32) * 2.0 ** -23) * wv + 2 * HALF_ULP[q.dtype] * want.abs() + 2 * TINY[q.dtype]
    close(out, want, tol + 2.0 ** -32 * floor[0] if floor else tol, f"attention {tuple(q.shape)}")
    ltol = 2 * d[:, :, 0] + 2.0 ** -14 + (L / 16 + 32) * 2.0 ** -23 + 2.0 ** -22 * torch.nan_to_num(lse, neginf=0.0).abs()
    none = torch.isinf(lse)
    assert torch.equal(torch.isinf(got_lse.cpu()), none) and torch.equal(torch.isnan(got_lse.cpu()), torch.isnan(lse))
    close(torch.where(none, 0.0, got_lse.cpu().double()), torch.where(none, 0.0, lse), ltol, "lse")
    return out


def queries(S, H, D, dtype, seed=0):
    return torch.randn(S, H, D, generator=gen(seed)).to(dtype).cuda()


def narrow(pages, page, block, heads, dim, seed=0, hnd=False):
    """A cache of standard-normal values, as a model has it: heads of different size."""
    g = gen(seed)
    out, scales = [], []
    for _ in range(2):
        x = torch.randn(pages, page // block, block, heads, dim, generator=g) * torch.exp2(torch.randint(-2, 3, (heads, 1), generator=g))
        e = torch.ceil(torch.log2(x.abs().amax((2, 4)) / 448))
        x = (x * torch.exp2(-e)[:, :, None, :, None]).to(E4M3).view(pages, page, heads, dim)
        out.append(ordered(x.cuda().view(torch.uint8), hnd).view(E4M3))
        scales.append(ordered((e + 127).to(torch.uint8).cuda(), hnd))
    return out + scales


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (4, 4, 64), (40, 2, 64), (24, 1, 128), (5, 1, 80), (16, 2, 192), (9, 1, 256),
                                    (2, 1, 16), (32, 2, 96)])
@pytest.mark.parametrize("page,block,hnd", [(16, 16, False), (24, 8, True), (64, 32, True), (7, 7, False), (48, 1, False)])
def test_attention8(dtype, H, Hk, D, page, block, hnd):
    lengths = [0, 1, 2, 15, 16, 17, 33, 100, 257]
    need = [-(-n // page) for n in lengths]
    cache = narrow(sum(need) + 1, page, block, Hk, D, seed=H, hnd=hnd)
    table = tables(need, sum(need) + 1)
    check_attention(queries(len(lengths), H, D, dtype), cache, table, ints(lengths))
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 128, 16), (4, 4, 64, 24), (20, 1, 64, 32), (3, 1, 192, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 0), (16, 4), (50, 16), (37, 33), (100, 200), (128, 7), (0, 9), (2 ** 31 - 1, 2 ** 31 - 1),
                                          (3, 2 ** 31 - 1)])
def test_attention_window_and_sinks(codes, H, Hk, D, page, window, sinks):
    lengths = [0, 1, 5, 16, 40, 41, 71, 150, 300, 517]
    need = [-(-n // page) for n in lengths]
    if codes:
        cache = narrow(sum(need), page, page // 2, Hk, D, seed=window % 1000)
    else:
        g = gen(window % 1000)
        cache = [torch.randn(sum(need), page, Hk, D, generator=g).to(BF).cuda() for _ in range(2)] + [None, None]
    table = tables(need, sum(need))
    check_attention(queries(len(lengths), H, D, BF), cache, table, ints(lengths), window=window, sinks=sinks)
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("codes", [True, False])
def test_what_is_not_seen_has_no_effect(codes):
    """NaN in every place that is not seen, pages that are needed by nobody
    missing: between the first positions and the window, and behind the length."""
    H, Hk, D, page, lengths, window, sinks = 8, 2, 64, 16, [100, 200, 37], 20, 5
    need = [-(-n // page) for n in lengths]
    if codes:
        cache = narrow(sum(need), page, 1, Hk, D, seed=5)
    else:
        cache = [torch.randn(sum(need), page, Hk, D, generator=gen(i)).to(HF).cuda() for i in (1, 2)] + [None, None]
    table = tables(need, sum(need), wide=16)
    q = queries(3, H, D, HF)
    want = check_attention(q, cache, table, ints(lengths), window=window, sinks=sinks)
    for s, n in enumerate(lengths):
        for p in range(need[s] * page):
            if not (p < sinks or n - window <= p < n):
                at = int(table[s, p // page]), p % page
                for t in cache[:2]:
                    if codes:
                        t.view(torch.uint8)[at] = 0x7F
                    else:
                        t[at] = math.nan
                if codes:
                    cache[2][at], cache[3][at] = 255, 255
        for e in range(table.shape[1]):
            if not any(p < sinks or n - window <= p < n for p in range(e * page, (e + 1) * page)):
                table[s, e] = 10 ** 6
    got = fq.decode_attention(q, cache[0], cache[1], table, ints(lengths), window=window, sinks=sinks, k_scale=cache[2],
                              v_scale=cache[3])
    assert torch.equal(got, want)
    assert fq.fp4_status_sync() == fq.FP4_OK


def test_attention8_every_code_and_wide_scales():
    """Every code, and blocks whose scales differ by many binades: the weights
    times the values' scales, not the weights, decide what counts."""
    cache = cache8(20, 16, 4, 2, 64, seed=3, lo=100, hi=110)
    cache[2].copy_(torch.randint(112, 119, cache[2].shape, generator=gen(4)))
    cache[3].copy_(torch.randint(60, 170, cache[3].shape, generator=gen(5)))
    table = tables([8, 12], 20)
    check_attention(queries(2, 6, 64, BF) * 0.25, cache, table, ints([128, 190]))


def test_attention8_scales_of_dead_weight():
    """All weight on positions whose values' unit is 2^-100, the others' 2^20."""
    H, D, n = 2, 64, 64
    k, v, ks, vs = narrow(4, 16, 16, 1, D)
    table = ints([[0, 1, 2, 3]])
    q = queries(1, H, D, BF)
    vs[:] = 147
    vs[2] = 27
    ks[:] = 90   # scores of next to nothing ...
    k.view(torch.uint8)[2] = 0
    q[:, :, 0] = 64.0
    k.view(torch.uint8)[2, :, :, 0] = 0x78  # ... but for page 2: 256 * 64 / 8 / 2 = 1024
    ks[2] = 126
    k.view(torch.uint8)[[0, 1, 3], :, :, 0] = 0xF8
    ks[[0, 1, 3]] = 126  # and the others at -1024: weights of e^-2000
    check_attention(q, (k, v, ks, vs), table, ints([n]))


def test_attention8_query_magnitudes():
    """Queries of BF16's whole range, a head each; zeros; small beside large."""
    cache = narrow(8, 16, 16, 1, 64, seed=6)
    table = tables([8], 8)
    q = queries(1, 8, 64, BF)
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3] *= 2.0 ** -128
    q[0, 4, ::2] *= 2.0 ** -18
    q[0, 5] *= 300
    check_attention(q, cache, table, ints([120]))
    check_attention(q.clone() * 1e30, [cache[0], cache[1], cache[2] - 40, cache[3]], table, ints([50]), scale=1e-20)


@pytest.mark.parametrize("n", [40, 3000])
def test_attention8_nan_stays_where_it_is(n):
    page, need = 16, -(-n // 16)
    k, v, ks, vs = narrow(need + 1, page, 16, 2, 64, seed=7)
    table = tables([need, 1], need + 1)
    q = queries(2, 8, 64, BF)
    ln = ints([n, 16])
    clean = fq.decode_attention(q, k, v, table, ln, k_scale=ks, v_scale=vs)
    at = int(table[0, (n - 3) // page]), (n - 3) % page
    v.view(torch.uint8)[at[0], at[1], 1, 9] = 0xFF
    got = fq.decode_attention(q, k, v, table, ln, k_scale=ks, v_scale=vs)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 4:, 9] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])
    k.view(torch.uint8)[at[0], at[1], 0, 2] = 0x7F   # a key: the heads that see it
    q[1, 6, 3] = math.inf                            # a query: its head
    got = check_attention(q, (k, v, ks, vs), table, ln)
    bad[0, :4] = True
    bad[1, 6] = True
    assert torch.equal(torch.isnan(got), bad)


@pytest.mark.parametrize("H,Hk,D,page,block,lengths,window,sinks", [
    (32, 8, 128, 64, 64, [20011], 0, 0), (32, 8, 128, 16, 16, [3000, 7, 9001, 0, 4096], 0, 0),
    (16, 16, 64, 32, 8, [5000, 4999, 3, 2500], 1000, 4), (24, 1, 128, 24, 24, [12345, 333], 0, 0),
    (8, 1, 256, 16, 16, [6000], 2049, 100), (4, 2, 192, 128, 32, [9999, 100], 0, 0)])
def test_attention8_long(H, Hk, D, page, block, lengths, window, sinks):
    """Rows cut into many parts, and parts of many rows, joined."""
    need = [-(-n // page) for n in lengths]
    cache = narrow(sum(need), page, block, Hk, D, seed=8, hnd=len(lengths) == 1)
    table = tables(need, sum(need))
    check_attention(queries(len(lengths), H, D, BF), cache, table, ints(lengths), window=window, sinks=sinks)


def test_attention8_many_sequences():
    S = 700
    lengths = torch.randint(0, 40, (S,), generator=gen(9)).tolist()
    need = [-(-n // 16) for n in lengths]
    cache = narrow(sum(need), 16, 16, 1, 64, seed=9)
    check_attention(queries(S, 4, 64, HF), cache, tables(need, sum(need)), ints(lengths))


def test_attention8_strides_streams_and_outputs():
    """Queries of a fused projection, a given output, another stream."""
    lengths = [50, 700]
    need = [-(-n // 16) for n in lengths]
    cache = narrow(sum(need), 16, 16, 2, 64)
    table = tables(need, sum(need))
    fused = queries(2, 12, 64, BF)
    out = torch.full((2, 10, 64), 7.0, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check_attention(fused[:, 2:10], cache, table, ints(lengths), out=out[:, 1:9], stream=s)
    s.synchronize()
    assert (out[:, 0] == 7).all() and (out[:, 9] == 7).all()


def test_attention8_lengths_and_pages_outside():
    k, v, ks, vs = narrow(4, 16, 16, 1, 64)
    table = ints([[0, 1], [2, 99], [3, 0]])
    q = queries(3, 2, 64, BF)
    got = fq.decode_attention(q, k, v, table, ints([-5, 20, 100]), k_scale=ks, v_scale=vs)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert not got[0].any()
    ref = Cache8(k, v, ks, vs)
    want, wv, _, _ = attention(q[1:], ref.values("k"), ref.values("v"), table[1:], torch.tensor([16, 32]), 64 ** -0.5, 0, 0)
    close(got[1:], want, 2.0 ** -12 * wv + 2 * HALF_ULP[BF] * want.abs(), "cut")


# --------------------------------------------------------------------- plan

def state(seqs, wide, pages, seed=0):
    table = torch.full((seqs, wide), -1, dtype=I32, device="cuda")
    return dict(lengths=ints([0] * seqs), page_table=table, room=ints([0] * seqs), pool=fq.page_pool(pages))


def check_plan(st, ref, new, page, tokens):
    """One plan of the library and of the definition: maps, state, status."""
    got = fq.page_plan(ints(new), st["lengths"], st["page_table"], st["room"], st["pool"], page, tokens=tokens)
    want, refused = ref.plan(new, tokens)
    assert (fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG) == refused
    if tokens is None:
        assert got is None
    else:
        for name, a, b in zip(("seq", "pos", "slot", "offsets"), got, want):
            assert a.tolist() == b, name
    assert st["lengths"].tolist() == ref.lengths and st["room"].tolist() == ref.room
    assert st["page_table"].tolist() == ref.table
    pool = st["pool"].tolist()
    assert pool[0] == len(ref.free) and pool[1] == 0 and pool[2:2 + pool[0]] == ref.free
    return got


@pytest.mark.parametrize("seqs,wide,pages,page,most", [(1, 4, 4, 16, 40), (5, 9, 30, 8, 20), (64, 20, 700, 16, 90), (513, 3, 900, 7, 5),
                                                       (1500, 4, 4000, 64, 100), (3, 600, 1000, 1, 300)])
def test_plan_by_steps(seqs, wide, pages, page, most):
    """Random steps: admissions, single tokens, roll-backs, ends; now and then
    more than there are pages, places or rows in the batch."""
    st = state(seqs, wide, pages)
    ref = Pages(st["lengths"], st["page_table"], st["room"], st["pool"], page)
    g = gen(seqs)
    for step in range(12):
        kind = step % 4
        new = torch.randint(0, most + 1, (seqs,), generator=g)
        if kind == 1:
            new = torch.ones(seqs, dtype=torch.long)
        elif kind == 2:
            new = torch.randint(-5, 6, (seqs,), generator=g)
        elif kind == 3:
            new = torch.where(torch.rand(seqs, generator=g) < 0.5, torch.tensor(-2 ** 31), new // 4)
        new = new.tolist()
        total = sum(max(n, 0) for n in new)
        tokens = [None, total, total + 13, total * 3 // 4][(step + step // 4) % 4]
        check_plan(st, ref, new, page, tokens)


def test_plan_large_batch():
    """A batch over many CTAs: prompts of a quarter million tokens, then back."""
    seqs, page = 96, 16
    n = torch.randint(0, 5500, (seqs,), generator=gen(1)).tolist()
    pages = sum(-(-a // page) for a in n)
    st = state(seqs, 400, pages + 5)
    start = {k: v.clone() for k, v in st.items()}
    ref = Pages(st["lengths"], st["page_table"], st["room"], st["pool"], page)
    check_plan(st, ref, n, page, sum(n) + 9)
    check_plan(st, ref, [-a for a in n], page, None)
    assert all(torch.equal(st[k], start[k]) for k in st)


def test_plan_general_way_and_a_graph():
    """Another stream gives the same; a captured step replayed gives out pages
    as sequences grow into them."""
    page, seqs = 4, 3
    st = state(seqs, 8, 20)
    ref = Pages(st["lengths"], st["page_table"], st["room"], st["pool"], page)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fq.page_plan(ints([3, 0, 9]), st["lengths"], st["page_table"], st["room"], st["pool"], page, tokens=14, stream=s)
    s.synchronize()
    want, _ = ref.plan([3, 0, 9], 14)
    assert [t.tolist() for t in got] == list(want)
    new = ints([1, 2, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fq.page_plan(new, st["lengths"], st["page_table"], st["room"], st["pool"], page, tokens=4)
    for step in range(8):
        if step == 5:
            new.copy_(ints([-1, 0, 1]))
        graph.replay()
        want, _ = ref.plan(new.tolist(), 4)
        assert [t.tolist() for t in got] == list(want)
        assert st["page_table"].tolist() == ref.table and st["lengths"].tolist() == ref.lengths
    assert fq.fp4_status_sync() == fq.FP4_OK


# ----------------------------------------------------------------- together

@pytest.mark.parametrize("H,Hk,D,page,block,window,sinks", [(8, 2, 64, 16, 16, 0, 0), (12, 4, 128, 8, 4, 30, 3)])
def test_plan_append_attention_together(H, Hk, D, page, block, window, sinks):
    """Prompts admitted, then steps of one token in a graph, with a sequence
    that ends and another that takes its place: each step against the definition."""
    seqs, wide = 3, 12
    st = state(seqs, wide, 30)
    cache = [torch.zeros(30, page, Hk, D, device="cuda").to(E4M3) for _ in range(2)]
    cache += [torch.zeros(30, page // block, Hk, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v, ks, vs = cache
    ref = Cache8(*cache)
    rope = exact_rope(page * wide, D)
    names = ("lengths", "page_table", "room", "pool")

    def plan(new, tokens):
        return fq.page_plan(new, *(st[n] for n in names), page, tokens=tokens)

    p = plan(ints([20, 0, 33]), 60)
    x = few_bits((60, 2 * Hk, D), BF, 1)
    fq.kv_append(x[:, :Hk], x[:, Hk:], k, v, st["page_table"], p.pos, seq=p.seq, rope=rope, k_scale=ks, v_scale=vs)
    ref.append(x[:, :Hk], x[:, Hk:], st["page_table"], p.pos.cpu(), p.seq.cpu(), rope, False)
    check_cache(cache, ref, "prompts")
    flat = k.view(torch.uint8).view(-1, Hk, D)
    slot = p.slot[:53].long()
    assert torch.equal(flat[slot].view(E4M3).float().cpu().double(), ref.k.view(-1, Hk, D)[slot.cpu()])

    new, row = ints([1, 0, 1]), torch.empty(2, H + 2 * Hk, D, dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = plan(new, 2)
        q = fq.kv_append(row[:, H:H + Hk], row[:, H + Hk:], k, v, st["page_table"], p.pos, seq=p.seq, q=row[:, :H], rope=rope,
                         k_scale=ks, v_scale=vs)
        full = torch.zeros(seqs, H, D, dtype=BF, device="cuda").index_copy(0, p.seq.clamp(min=0).long(), q)
        out = fq.decode_attention(full, k, v, st["page_table"], st["lengths"], window=window, sinks=sinks, k_scale=ks, v_scale=vs)
    for step in range(7):
        if step == 4:  # sequence 0 ends, sequence 1 begins
            fq.page_plan(ints([-2 ** 31, 0, 0]), *(st[n] for n in names), page)
            new.copy_(ints([0, 1, 1]))
        row.copy_(few_bits(row.shape, BF, 10 + step, 2.0 ** (step - 3)))
        graph.replay()
        ref.append(row[:, H:H + Hk], row[:, H + Hk:], st["page_table"], p.pos.cpu(), p.seq.cpu(), rope, False)
        check_cache(cache, ref, f"step {step}")
        want, wv, _, mag, floor = attention(full, ref.values("k"), ref.values("v"), st["page_table"], st["lengths"].cpu(), D ** -0.5,
                                            window, sinks, ref.units("v"))
        d = ((D / 16 + 8) * 2.0 ** -23 * mag)[:, :, None]
        close(out, want, (4 * d + 2.0 ** -14 + 40 * 2.0 ** -23) * wv + 2 * HALF_ULP[BF] * want.abs() + 2 * TINY[BF] + 2.0 ** -32 * floor,
              f"step {step}")
    assert fq.fp4_status_sync() == fq.FP4_OK
