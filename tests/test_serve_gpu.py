"""The serving operators on the GPU against their 64-bit definitions.

Tolerances, derived from the arithmetic (u: half a unit in the last place of
the output type, binary32 sums throughout):
  product    (K/16 + 16) 2^-23 S + 2 u |y|, S = sum |w x|: one rounding (up to
             a whole unit, the tensor core truncates) per 16 products and per
             join -- the bound of the BF16 GEMM
  rotation   2^-22 (|a cos| + |b sin|) + 2 u |y|: three binary32 roundings
  attention  a score is off by d = (D/16 + 8) 2^-23 max sum |q k| scale, which
             changes a weight and the sum by the factor 1 +- d each; weights
             as two 16-bit parts 2^-15; the sum over L positions as for the
             product: (4 d + 2^-14 + (L/16 + 32) 2^-23) sum w |v| + 2 u |out|
"""
import math

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300 import serve
from gpu_util import need_gpu
from serve_ref import HALF_ULP, TINY, attention, matvec, rotate, scale_values, tile

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
UE, NV, MX, UE32, CTA = (fq.FP4_FMT_UE5M3_B16, fq.FP4_FMT_NVFP4_B16, fq.FP4_FMT_MXFP4_B32,
                         fq.FP4_FMT_UE5M3_B32, fq.FP4_FMT_NVFP4_CTA)
PLAIN, MMA = fq.FP4_SF_PLAIN, fq.FP4_SF_MMA


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
    err = (got - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                             f"{got[i]} for {want[i]}, tolerance {tol[i]}")


# ------------------------------------------------------------------ product

def weight(n, k, fmt, layout, remap=True, seed=0):
    """A weight quantised by the library, as a user has it."""
    w = (torch.randn(n, k, generator=gen(seed)) * 0.02).to(BF).cuda()
    p = fq.params(format=fmt, sf_layout=layout)
    a = fq.amax_stripes(w)[0] if fmt == CTA else fq.amax(w)[0]
    return fq.quantize(w, a, p, remap=remap)


def random_copy(n, k, fmt, layout, seed=0):
    """Random payload bytes and random scale codes over the format's range."""
    g = gen(seed)
    q = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    block = 32 if fmt in (MX, UE32) else 16
    cols = k // block
    if fmt == MX:
        sf = torch.randint(100, 141, (n, cols), generator=g, dtype=torch.int32)
    else:
        sf = torch.randint(0, (0xF8 if fmt in (UE, UE32) else 0x7F), (n, cols), generator=g,
                           dtype=torch.int32)
    sf = sf.to(torch.uint8)
    if layout == MMA and fmt == UE32:
        sf = sf.repeat_interleave(2, 1)
    sf = tile(sf) if layout == MMA else sf.contiguous().view(-1)
    return fq.Quantized(q.cuda(), sf.cuda(), torch.tensor([0.37], device="cuda"), None, fmt, layout)


def check_matvec(x, w, out_dtype, y=None):
    want, s = matvec(x, w)
    y = fq.matvec(x, w, out_dtype=out_dtype) if y is None else y
    assert y.dtype == out_dtype
    tol = (w.k / 16 + 16) * 2.0 ** -23 * s + 2 * HALF_ULP[out_dtype] * want.abs() + 2 * TINY[out_dtype]
    close(y, want, tol, f"N {w.rows} K {w.k} M {x.shape[0] if x.dim() == 2 else 1}")
    return y


@pytest.mark.parametrize("fmt,layout,remap", [(NV, PLAIN, True), (NV, MMA, True), (UE, PLAIN, True),
                                              (UE, MMA, True), (UE, MMA, False), (MX, PLAIN, True),
                                              (MX, MMA, True), (UE32, PLAIN, True),
                                              (UE32, MMA, True), (CTA, PLAIN, True), (CTA, MMA, True)])
@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (3, 300, 4096), (16, 129, 1088), (17, 128, 192),
                                   (40, 77, 320)])
def test_matvec_formats_and_layouts(fmt, layout, remap, m, n, k):
    w = weight(n, k, fmt, layout, remap)
    x = torch.randn(m, k, generator=gen(1)).to(BF).cuda()
    check_matvec(x, w, BF)
    check_matvec(x.to(HF), w, F32)
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("k", [16, 32, 48, 112, 128, 144, 496, 2064, 8208])
@pytest.mark.parametrize("m,n", [(1, 1), (2, 15), (7, 17), (8, 130), (9, 1001)])
def test_matvec_odd_sizes(m, n, k):
    w = random_copy(n, k, UE, PLAIN, seed=k + n)
    x = torch.randn(m, k, generator=gen(2)).cuda()
    check_matvec(x.to(HF), w, F32)
    check_matvec(x.to(BF), w, F32)


@pytest.mark.parametrize("fmt,layout", [(NV, PLAIN), (NV, MMA), (UE, PLAIN), (UE, MMA), (MX, PLAIN),
                                        (MX, MMA), (UE32, PLAIN), (UE32, MMA)])
def test_matvec_every_code(fmt, layout):
    """Random bytes: every payload byte, and scale codes over the whole range."""
    w = random_copy(640, 1024, fmt, layout, seed=3)
    x = torch.randn(5, 1024, generator=gen(4)).to(BF).cuda()
    check_matvec(x, w, F32)


@pytest.mark.parametrize("fmt,code", [(NV, 0x7F), (UE, 0xFF), (MX, 0xFE), (UE32, 0xFF)])
@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 17, 21, 30, 129])
@pytest.mark.parametrize("m", [2, 11])
def test_matvec_rows_that_begin_inside_words(fmt, code, blocks, m):
    """Plain scales of every pitch: each row has its own codes, and a row whose
    codes are NaN (MXFP4, which has none: 2^127) changes itself alone."""
    n, k = 75, blocks * (32 if fmt in (MX, UE32) else 16)
    w = random_copy(n, k, fmt, PLAIN, seed=blocks)
    x = torch.randn(m, k, generator=gen(36)).to(HF).cuda()
    y = check_matvec(x, w, F32)
    w.sf.view(n, blocks)[[0, 33, n - 1]] = code
    z = fq.matvec(x, w, out_dtype=F32)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[0, 33, n - 1]] = True
    assert (fmt == MX or torch.isnan(z[:, bad]).all()) and torch.equal(z[:, ~bad], y[:, ~bad])


def test_matvec_tall_and_long():
    """Over 65535 rows, and a row longer than any shared-memory tile."""
    w = random_copy(70001, 64, NV, PLAIN)
    x = torch.randn(2, 64, generator=gen(5)).to(BF).cuda()
    check_matvec(x, w, F32)
    w = random_copy(40, 65536 + 16, NV, PLAIN)
    x = torch.randn(16, 65536 + 16, generator=gen(6)).to(HF).cuda()
    check_matvec(x, w, F32)


def test_matvec_activation_magnitudes():
    """Outliers 2^12 above the rest, tokens of very different size, zeros,
    BF16's extremes, signed zeros and subnormals."""
    k = 1024
    w = random_copy(200, k, NV, PLAIN, seed=7)
    x = torch.randn(8, k, generator=gen(8))
    x[0, ::100] *= 4096
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 0
    x[4, :512] *= 1e-6
    x[5] = -0.0
    x[6] *= 1e-38
    check_matvec(x.to(BF).cuda(), w, F32)
    h = torch.randn(4, k, generator=gen(9))
    h[0] *= 6e-8
    h[1] *= 1000
    h[2, 5] = 65504
    check_matvec(h.to(HF).cuda(), w, F32)


def test_matvec_nonfinite_stays_in_its_token():
    w = random_copy(64, 256, NV, PLAIN, seed=10)
    x = torch.randn(4, 256, generator=gen(11)).to(BF)
    x[1, 17] = float("nan")
    x[2, 200] = float("inf")
    y = fq.matvec(x.cuda(), w, out_dtype=F32).cpu()
    want, _ = matvec(x, w)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    fine = torch.isfinite(want)
    assert torch.equal(y[~fine & ~torch.isnan(want)].double(), want[~fine & ~torch.isnan(want)])
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()


def test_matvec_strides_out_and_vector():
    n, k = 100, 256
    w = weight(n, k, NV, PLAIN)
    wide = torch.randn(6, 3 * k + 1, generator=gen(12)).to(BF).cuda()
    for start in (0, 8, 1):  # aligned and odd starts; the row pitch is odd
        check_matvec(wide[:, start:start + k], w, F32)
    x = wide[:, :k].contiguous()
    big = torch.full((6, n + 5), 7.0, device="cuda", dtype=BF)
    out = big[:, 2:2 + n]
    assert fq.matvec(x, w, out=out) is out
    check_matvec(x, w, BF, y=out)
    assert (big[:, :2] == 7).all() and (big[:, 2 + n:] == 7).all()  # nothing beside it is written
    y = fq.matvec(x[0], w)
    assert y.shape == (n,) and torch.equal(y, fq.matvec(x[:1], w)[0])
    flat = x[:1].expand(5, k)  # rows of stride 0 are refused by the library
    with pytest.raises(fq.FP4Error):
        fq.matvec(flat, w)


def test_matvec_empty():
    w = weight(64, 128, NV, PLAIN)
    assert fq.matvec(torch.empty(0, 128, dtype=BF, device="cuda"), w).shape == (0, 64)
    none = fq.Quantized(torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
                        torch.empty(0, dtype=torch.uint8, device="cuda"),
                        torch.ones(1, device="cuda"), None, NV, PLAIN)
    y = fq.matvec(torch.empty(3, 0, dtype=BF, device="cuda"), none)
    assert y.shape == (3, 5) and (y == 0).all()


def test_matvec_repeats_exactly_and_on_other_streams():
    w = weight(1000, 4096, UE, MMA)
    x = torch.randn(4, 4096, generator=gen(13)).to(BF).cuda()
    y = fq.matvec(x, w)
    assert all(torch.equal(y, fq.matvec(x, w)) for _ in range(5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = fq.matvec(x, w, stream=side)
    with torch.cuda.stream(side):
        z2 = fq.matvec(x, w)
    side.synchronize()
    assert torch.equal(y, z) and torch.equal(y, z2)


def test_matvec_serves_the_gemms_copy():
    """One tensor-core-layout copy gives the GEMM and the product the same
    weight: the product of the dequantised plain copy."""
    w_src = (torch.randn(256, 512, generator=gen(14)) * 0.02).to(BF).cuda()
    a = fq.amax(w_src)[0]
    m = fq.quantize(w_src, a, fq.params(format=UE, sf_layout=MMA))
    p = fq.quantize(w_src, a, fq.params(format=UE, sf_layout=PLAIN))
    x = torch.randn(3, 512, generator=gen(15)).to(BF).cuda()
    ym, yp = fq.matvec(x, m, out_dtype=F32), fq.matvec(x, p, out_dtype=F32)
    _, s = matvec(x, p)
    close(ym, yp.cpu().double(), 2 * (512 / 16 + 16) * 2.0 ** -23 * s, "layouts")
    assert torch.equal(p.q, m.q)


# ------------------------------------------------------------------- append

def cache(pages, page, heads, dim, dtype, order="nhd", fill=None, seed=0):
    shape = (pages, page, heads, dim) if order == "nhd" else (pages, heads, page, dim)
    made = []
    for i in range(2):
        t = torch.randn(shape, generator=gen(seed + i)).to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype)
        t = t.cuda()
        made.append(t.transpose(1, 2) if order == "hnd" else t)
    return made


def check_append(k, v, kp, vp, table, pos, seq, q, rope, interleaved, q_out=None):
    dtype, page = kp.dtype, kp.shape[1]
    want_k, want_v = kp.cpu().double().clone(), vp.cpu().double().clone()
    tol_k = torch.zeros_like(want_k)
    u = HALF_ULP[dtype]
    rk, mk = rotate(k, rope, pos, interleaved)
    ps, sq = pos.tolist(), (range(len(pos)) if seq is None else seq.tolist())
    for t, (p, s) in enumerate(zip(ps, sq)):
        if p < 0:
            continue
        at = (int(table[s, p // page]), p % page)
        want_k[at], want_v[at] = rk[t], v[t].cpu().double()
        tol_k[at] = 2.0 ** -22 * mk[t] + (2 * u * rk[t].abs() + 2 * TINY[dtype]) * (mk[t] > 0)
    rq, mq = rotate(q, rope, pos, interleaved) if q is not None else (None, None)
    got = fq.kv_append(k, v, kp, vp, table, pos, seq=seq, q=q, rope=rope, interleaved=interleaved,
                       q_out=q_out)
    close(kp, want_k, tol_k, "keys")
    assert torch.equal(vp.cpu().double(), want_v)
    if q is None:
        assert got is None
    else:
        skipped = (pos.cpu() < 0)[:, None, None]
        rq = torch.where(skipped, 0.0, rq)
        tol = 2.0 ** -22 * mq + (2 * u * rq.abs() + 2 * TINY[dtype]) * (mq > 0)
        close(got, rq, torch.where(skipped, 0.0, tol), "queries")
    return got


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("heads,hk,dim,rot,page,inter", [
    (8, 2, 128, 128, 16, False), (4, 4, 64, 32, 8, True), (6, 3, 80, 80, 24, False),
    (5, 1, 96, 48, 16, True), (2, 2, 256, 256, 64, False), (3, 3, 8, 0, 4, False),
    (4, 2, 40, 20, 7, False), (2, 1, 7, 6, 1, True), (8, 8, 128, 64, 32, False)])
def test_append_shapes(dtype, order, heads, hk, dim, rot, page, inter):
    T, S = 37, 5
    table = torch.randperm(S * 9, generator=gen(1)).view(S, 9)[:, :8].to(torch.int32).cuda()
    kp, vp = cache(S * 9, page, hk, dim, dtype, order)
    seq = torch.arange(T) % S
    pos = torch.arange(T) // S
    if 8 * page < 8:
        pos = pos % page
    pos[[3, 11]] = -1
    qkv = torch.randn(T, heads + 2 * hk, dim, generator=gen(2)).to(dtype).cuda()
    rope = fq.rope_table(16, rot) if rot else None
    check_append(qkv[:, heads:heads + hk], qkv[:, heads + hk:], kp, vp, table,
                 pos.to(torch.int32).cuda(), seq.to(torch.int32).cuda(), qkv[:, :heads], rope, inter)
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("dim,rot,inter,pad", [(80, 40, False, 0), (12, 8, False, 0), (20, 16, True, 0), (20, 0, False, 4),
                                               (64, 64, False, 4), (64, 32, True, 12), (252, 248, False, 0), (4, 0, False, 0)])
@pytest.mark.parametrize("T", [1, 50, 2500])
def test_append_pieces_of_eight_bytes(dim, rot, inter, pad, T):
    """Rows that are whole pieces of 4 elements but not of 8, by size or by
    stride."""
    heads, hk, page = 6, 2, 16
    pages = T // page + 2
    table = torch.randperm(pages, generator=gen(40))[None].to(torch.int32).cuda()
    kp, vp = (t[..., :dim] for t in cache(pages, page, hk, dim + pad, BF))
    qkv = torch.randn(T, heads + 2 * hk, dim + pad, generator=gen(41)).to(BF).cuda()[..., :dim]
    pos = torch.randperm(T, generator=gen(42)).to(torch.int32).cuda()
    check_append(qkv[:, heads:heads + hk], qkv[:, heads + hk:], kp, vp, table, pos,
                 torch.zeros(T, dtype=torch.int32).cuda(), qkv[:, :heads], fq.rope_table(T, rot) if rot else None, inter)
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("T", [1, 2, 200, 3001])
def test_append_token_counts_and_decode_form(T):
    page, hk, dim, heads = 16, 2, 128, 8
    table = torch.randperm(T * 2, generator=gen(3))[:T, None].to(torch.int32).cuda()
    kp, vp = cache(T * 2, page, hk, dim, BF)
    pos = torch.randint(0, page, (T,), generator=gen(4)).to(torch.int32).cuda()
    k, v, q = (torch.randn(T, h, dim, generator=gen(5 + h)).to(BF).cuda() for h in (hk, hk, heads))
    check_append(k, v, kp, vp, table, pos, None, q, fq.rope_table(page, dim), False)
    check_append(k, v, kp, vp, table, pos, None, None, fq.rope_table(page, dim), True)


def test_append_odd_strides_and_in_place_queries():
    """Pitches and starts that no 16-byte piece fits; q rotated in place."""
    T, hk, heads, dim, page = 9, 2, 4, 64, 8
    table = torch.arange(T)[:, None].to(torch.int32).cuda()
    raw = torch.randn(2, T * page * hk * (dim + 3) + 1, generator=gen(6)).to(HF).cuda()
    kp, vp = (r[1:].view(T, page, hk, dim + 3)[..., :dim] for r in raw)
    wide = torch.randn(T, heads + 2 * hk, dim + 1, generator=gen(7)).to(HF).cuda()[..., 1:]
    pos = torch.full((T,), 3, dtype=torch.int32).cuda()
    rope = fq.rope_table(4, dim)
    q = wide[:, :heads]
    before = q.clone()
    new = check_append(wide[:, heads:heads + hk], wide[:, heads + hk:], kp, vp, table, pos, None, q,
                       rope, False)
    assert torch.equal(q, before)
    same = fq.kv_append(wide[:, heads:heads + hk], wide[:, heads + hk:], kp, vp, table, pos, q=q,
                        rope=rope, q_out=q)
    assert same is q and torch.equal(q, new)


def test_append_reports_what_lies_outside():
    page, hk, dim = 4, 1, 64
    kp, vp = cache(3, page, hk, dim, BF)
    k = torch.randn(6, hk, dim, generator=gen(8)).to(BF).cuda()
    ik = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    table = torch.tensor([[0, 99], [1, -5]], dtype=torch.int32).cuda()
    rope = fq.rope_table(8, dim)
    before = kp.clone(), vp.clone()
    # page 99, page -5, position past the table, sequences 2 and -1, rotation past its table
    for pos, seq, rp in ((4, 0, rope), (5, 1, rope), (8, 0, rope), (0, 2, rope), (0, -1, rope),
                         (3, 0, rope[:3].contiguous())):
        q = fq.kv_append(k[:1], k[:1], kp, vp, table, ik(pos), seq=ik(seq), q=k[:1], rope=rp)
        assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
        assert (q == 0).all() and torch.equal(kp, before[0]) and torch.equal(vp, before[1])
    fq.kv_append(k[:1], k[:1], kp, vp, table, ik(3), seq=ik(0), rope=rope)
    assert fq.fp4_status_sync() == fq.FP4_OK and not torch.equal(kp, before[0])


# ---------------------------------------------------------------- attention

def pool(lengths, page, hk, dim, dtype, order="nhd", seed=0, poison=True):
    """A cache for these lengths, its pages in random order; places that no
    length reaches hold NaN, table entries that none reaches nonsense."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 2
    kp, vp = cache(total, page, hk, dim, dtype, order, seed=seed)
    order_ = torch.randperm(total, generator=gen(seed + 9))
    table = torch.full((len(lengths), max(need + [0]) + 1), 2 ** 30, dtype=torch.int32)
    used = torch.zeros(total, page, dtype=torch.bool)
    at = 0
    for s, n in enumerate(need):
        mine = order_[at:at + n]
        table[s, :n] = mine
        at += n
        for i, pg in enumerate(mine.tolist()):
            used[pg, :min(page, lengths[s] - i * page)] = True
    if poison:
        kp[~used.cuda()] = float("nan")
        vp[~used.cuda()] = float("nan")
    return kp, vp, table.cuda()


def check_attention(q, kp, vp, table, lengths, scale=None, window=0, out=None, what=""):
    D = q.shape[-1]
    sc = D ** -0.5 if scale is None else scale
    want, wv, lse_want, mag = attention(q, kp, vp, table, lengths, sc, window)
    got, lse = fq.decode_attention(q, kp, vp, table, lengths, scale=scale, window=window, out=out,
                                   return_lse=True)
    n = lengths.cpu().double()
    n = (n.clamp(max=window) if window else n)[:, None]
    d = (D / 16 + 8) * 2.0 ** -23 * mag
    sums = (n / 16 + 32) * 2.0 ** -23
    tol = (4 * d + 2.0 ** -14 + sums)[..., None] * wv + 2 * HALF_ULP[q.dtype] * want.abs() + 2 * TINY[q.dtype]
    close(got, want, tol, f"attention {what}")
    empty = lengths.cpu() == 0
    assert (got[empty.cuda()] == 0).all() and (lse[empty.cuda()] == -math.inf).all()
    ok = ~empty
    close(lse[ok.cuda()], lse_want[ok], (d + sums + 2.0 ** -20)[ok] + 2.0 ** -22 * lse_want[ok].abs(), "lse")
    return got


EDGES = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 129, 200, 0, 255, 257]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,hk,dim,page,order", [
    (8, 1, 128, 16, "nhd"), (4, 4, 64, 8, "hnd"), (10, 2, 80, 24, "nhd"), (12, 2, 96, 16, "hnd"),
    (16, 1, 256, 32, "nhd"), (6, 2, 192, 64, "nhd"), (20, 1, 64, 16, "nhd"), (3, 1, 8, 5, "nhd"),
    (2, 2, 40, 1, "hnd"), (32, 2, 128, 128, "hnd"), (7, 7, 104, 48, "nhd"), (33, 1, 128, 7, "nhd")])
def test_attention_shapes(dtype, heads, hk, dim, page, order):
    kp, vp, table = pool(EDGES, page, hk, dim, dtype, order)
    q = torch.randn(len(EDGES), heads, dim, generator=gen(1)).to(dtype).cuda()
    lengths = torch.tensor(EDGES, dtype=torch.int32).cuda()
    check_attention(q, kp, vp, table, lengths)
    for window in (1, 16, 50, 100000):
        check_attention(q, kp, vp, table, lengths, window=window, what=f"window {window}")
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("lengths", [[1], [300], [5000], [40001], [1] * 700, [0, 0, 0],
                                     [9000, 1, 0, 3, 4097], [64 * i for i in range(40)]])
@pytest.mark.parametrize("heads,hk,dim,dtype", [(8, 2, 128, BF), (4, 1, 64, HF), (2, 2, 256, BF)])
def test_attention_lengths(lengths, heads, hk, dim, dtype):
    kp, vp, table = pool(lengths, 16, hk, dim, dtype)
    q = torch.randn(len(lengths), heads, dim, generator=gen(2)).to(dtype).cuda()
    ln = torch.tensor(lengths, dtype=torch.int32).cuda()
    a = check_attention(q, kp, vp, table, ln)
    assert all(torch.equal(a, fq.decode_attention(q, kp, vp, table, ln)) for _ in range(3))


@pytest.mark.parametrize("seqs,heads,hk,dim,dtype", [(1, 4, 1, 128, BF), (3, 8, 2, 64, HF), (24, 8, 2, 128, HF),
                                                     (70, 6, 2, 80, BF), (5, 24, 2, 128, BF), (9, 4, 4, 256, HF),
                                                     (260, 4, 2, 64, BF)])
@pytest.mark.parametrize("longest", [20, 130, 300, 700, 1400, 2100])
@pytest.mark.parametrize("window", [0, 77])
def test_attention_rows_shared_out(seqs, heads, hk, dim, dtype, longest, window):
    """Rows taken by one CTA, by a cluster or by equal slices, as their number
    and the room of the table say; empty, short and full ones side by side."""
    if seqs * longest > 60000:
        longest = 60000 // seqs
    g = gen(37)
    lengths = [(0, 1, 17, longest, longest // 2)[i % 5] if i % 3 else int(torch.randint(0, longest + 1, (1,), generator=g))
               for i in range(seqs)]
    lengths[0] = longest
    kp, vp, table = pool(lengths, 16, hk, dim, dtype)
    q = torch.randn(seqs, heads, dim, generator=gen(38)).to(dtype).cuda()
    check_attention(q, kp, vp, table, torch.tensor(lengths, dtype=torch.int32).cuda(), window=window)
    assert fq.fp4_status_sync() == fq.FP4_OK


def test_attention_scores_of_all_sizes():
    """A late position that outweighs all others, scores of thousands, equal
    scores, a negative scale, and a row whose scores are all minus infinity."""
    L, hk, dim = 1000, 1, 128
    kp, vp, table = pool([L] * 5, 16, hk, dim, BF)
    q = torch.randn(5, 4, dim, generator=gen(3)).to(BF).cuda()
    kp[table[0, 990 // 16], 990 % 16, 0] = (q[0, 0] * 8)
    q[1] *= 64
    q[2] = 0
    ln = torch.full((5,), L, dtype=torch.int32).cuda()
    check_attention(q, kp, vp, table, ln)
    check_attention(q, kp, vp, table, ln, scale=-0.3)
    check_attention(q, kp, vp, table, ln, scale=0.0)
    pages = table[3, :L // 16 + 1].long()
    kp[pages] = 0
    kp[pages, :, 0, 0] = float("-inf")
    q[3] = 0
    q[3, :, 0] = 1
    got, lse = fq.decode_attention(q, kp, vp, table, ln, return_lse=True)
    assert torch.isnan(got[3]).all() and (lse[3] == -math.inf).all()  # as softmax defines it
    assert torch.isfinite(got[[0, 1, 2, 4]]).all()
    kp[pages[5], 3, 0, 0] = 0.0  # one finite score: it takes all the weight
    got = fq.decode_attention(q, kp, vp, table, ln)
    assert torch.equal(got[3], vp[pages[5], 3, 0].expand(4, dim))


def test_attention_values_not_finite_stay_in_their_row():
    kp, vp, table = pool([100, 100], 16, 2, 64, BF)
    q = torch.randn(2, 4, 64, generator=gen(4)).to(BF).cuda()
    vp[table[0, 0], 0, 1, 5] = float("inf")
    got = fq.decode_attention(q, kp, vp, table, torch.tensor([100, 100], dtype=torch.int32).cuda()).cpu()
    want = torch.zeros(2, 4, 64, dtype=torch.bool)
    want[0, 2:, 5] = True
    assert torch.equal(~torch.isfinite(got), want) and (got[0, 2:, 5] == float("inf")).all()


def test_attention_strides_and_out():
    kp, vp, table = pool([70, 33, 0], 16, 2, 64, HF)
    wide = torch.randn(3, 9, 3, 80, generator=gen(5)).to(HF).cuda()
    q = wide[:, 1:7, 1, 8:72]
    ln = torch.tensor([70, 33, 0], dtype=torch.int32).cuda()
    big = torch.full((3, 6, 67), 7.0, dtype=HF, device="cuda")
    got = check_attention(q, kp, vp, table, ln, out=big[..., 1:65])
    assert got.data_ptr() == big[..., 1:65].data_ptr()
    assert (big[..., 0] == 7).all() and (big[..., 65:] == 7).all()


def test_attention_offsets_past_32_bits():
    """Pages 2^29 elements apart: their offsets pass 2^31 elements and 2^32
    bytes, in keys and values and through the append."""
    page, hk, dim, apart = 16, 1, 64, 2 ** 29
    raw = torch.empty(5 * apart + page * hk * dim * 2, dtype=BF, device="cuda")
    kp = raw.as_strided((6, page, hk, dim), (apart, hk * dim, dim, 1))
    vp = raw.as_strided((6, page, hk, dim), (apart, hk * dim, dim, 1), page * hk * dim)
    table = torch.tensor([[5, 0, 4]], dtype=torch.int32).cuda()
    L = 40
    k, v = (torch.randn(L, hk, dim, generator=gen(i)).to(BF).cuda() for i in (6, 7))
    pos = torch.arange(L, dtype=torch.int32).cuda()
    fq.kv_append(k, v, kp, vp, table, pos, seq=torch.zeros(L, dtype=torch.int32).cuda())
    q = torch.randn(1, 4, dim, generator=gen(8)).to(BF).cuda()
    got = fq.decode_attention(q, kp, vp, table, torch.tensor([L], dtype=torch.int32).cuda())
    flat_k, flat_v = (torch.zeros(3, page, hk, dim, dtype=BF) for _ in range(2))
    flat_k.view(-1, hk, dim)[:L], flat_v.view(-1, hk, dim)[:L] = k.cpu(), v.cpu()
    want, wv, _, mag = attention(q, flat_k, flat_v, torch.tensor([[0, 1, 2]]), torch.tensor([L]), dim ** -0.5, 0)
    tol = (4 * (dim / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -14 + (L / 16 + 32) * 2.0 ** -23)[..., None] * wv
    close(got, want, tol + 2.0 ** -8 * want.abs(), "far pages")


def test_attention_reports_what_lies_outside():
    kp, vp, table = pool([40, 40], 16, 1, 64, BF)
    q = torch.randn(2, 2, 64, generator=gen(9)).to(BF).cuda()
    ln = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    fine = fq.decode_attention(q, kp, vp, table, ln(40, 40))
    assert fq.fp4_status_sync() == fq.FP4_OK
    got = fq.decode_attention(q, kp, vp, table, ln(40, -3))  # negative: read as 0
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert torch.equal(got[0], fine[0]) and (got[1] == 0).all()
    got = fq.decode_attention(q, kp, vp, table[:, :3], ln(40, 1000))  # cut to 48 places
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert torch.equal(got[0], fine[0])
    bad = table.clone()
    bad[1, 1] = -1  # passed over: the other positions stand
    got = fq.decode_attention(q, kp, vp, bad, ln(40, 40))
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert torch.equal(got[0], fine[0]) and torch.isfinite(got[1]).all()
    short = table.clone()
    short[1, 1] = table[1, 2]
    want, wv, _, mag = attention(q[1:], kp, vp, short[1:], ln(24), 0.125, 0)
    tol = (4 * 12 * 2.0 ** -23 * mag + 2.0 ** -14 + 34 * 2.0 ** -23)[..., None] * wv
    close(got[1:], want, tol + 2.0 ** -8 * want.abs(), "a page passed over")


def test_attention_parts_join_by_lse():
    """Attention over two halves of a context joined by their lse is the
    attention over the whole."""
    L, page, hk, dim = 96, 16, 2, 64
    kp, vp, table = pool([L], page, hk, dim, BF)
    q = torch.randn(1, 4, dim, generator=gen(10)).to(BF).cuda()
    ln = lambda n: torch.tensor([n], dtype=torch.int32).cuda()  # noqa: E731
    whole, z = fq.decode_attention(q, kp, vp, table, ln(L), return_lse=True)
    a, za = fq.decode_attention(q, kp, vp, table[:, :3], ln(48), return_lse=True)
    b, zb = fq.decode_attention(q, kp, vp, table[:, 3:], ln(48), return_lse=True)
    joined = a.double() * (za - z).double().exp()[..., None] + b.double() * (zb - z).double().exp()[..., None]
    # each part is rounded to BF16 (2^-9 of itself), and so is the whole
    tol = 2.0 ** -8 * (a.double().abs() + b.double().abs() + whole.double().abs()) + 2.0 ** -13
    close(joined, whole.double().cpu(), tol.cpu(), "joined")


def test_attention_on_another_stream():
    kp, vp, table = pool([3000, 50], 16, 2, 128, BF)
    q = torch.randn(2, 8, 128, generator=gen(11)).to(BF).cuda()
    ln = torch.tensor([3000, 50], dtype=torch.int32).cuda()
    a = fq.decode_attention(q, kp, vp, table, ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = [fq.decode_attention(q, kp, vp, table, ln, stream=side) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(a, x) for x in b)


def test_scale_tables_of_the_reference():
    """The 64-bit tables the tests lean on, against torch's own E4M3."""
    codes = torch.arange(0x7F, dtype=torch.uint8)
    assert torch.equal(scale_values("e4m3")[:0x7F], codes.view(torch.float8_e4m3fn).double())
    assert scale_values("ue5m3")[0xF7] == 61440 and scale_values("ue5m3")[1] == 2.0 ** -17


class General:
    """A binding that leaves every call to the general way."""
    matvec = append = attention = staticmethod(lambda *a: NotImplemented)


def both_ways(monkeypatch, call):
    """The call through the compiled binding, which has to take it, and the
    general way."""
    bind, taken = serve._bind(), []

    class Watched:
        def __getattr__(self, name):
            def go(*a):
                r = getattr(bind, name)(*a)
                taken.append(r is not NotImplemented)
                return r
            return go

    monkeypatch.setattr(serve, "_bind", Watched)
    a = call()
    assert taken == [True]
    monkeypatch.setattr(serve, "_bind", General)
    return a, call()


@pytest.mark.parametrize("fmt,layout,remap", [(NV, PLAIN, True), (UE, MMA, True), (UE, MMA, False),
                                              (MX, MMA, True), (UE32, MMA, True), (CTA, PLAIN, True)])
@pytest.mark.parametrize("m", [None, 0, 1, 5])
def test_binding_and_general_way_agree_on_matvec(monkeypatch, fmt, layout, remap, m):
    w = weight(300, 512, fmt, layout, remap)
    wide = torch.randn(m or 1, 600, generator=gen(30)).to(BF).cuda()[:m, 8:520]
    x = wide[0] if m is None else wide
    for dtype in (None, BF, HF, F32):
        a, b = both_ways(monkeypatch, lambda: fq.matvec(x, w, out_dtype=dtype))
        assert a.dtype == b.dtype and a.device == b.device and torch.equal(a, b)
        monkeypatch.undo()


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("own_seq,with_q,rot,inter", [(True, True, 64, True), (False, True, 32, False),
                                                      (True, False, 64, False), (False, False, 0, False)])
def test_binding_and_general_way_agree_on_append(monkeypatch, order, dtype, own_seq, with_q, rot, inter):
    T, page, hk, heads, dim = 6, 8, 2, 4, 64
    table = torch.randperm(T, generator=gen(31)).view(T, 1).to(torch.int32).cuda()
    kp, vp = cache(T, page, hk, dim, dtype, order, fill=0.0)
    qkv = torch.randn(T, heads + 2 * hk, dim, generator=gen(32)).to(dtype).cuda()
    pos = torch.randint(0, page, (T,), generator=gen(33)).to(torch.int32).cuda()
    seq = torch.randperm(T, generator=gen(34)).to(torch.int32).cuda() if own_seq else None
    rope = fq.rope_table(page, rot) if rot else None

    def call():
        kp.zero_()
        vp.zero_()
        q = fq.kv_append(qkv[:, heads:heads + hk], qkv[:, heads + hk:], kp, vp, table, pos, seq=seq,
                         q=qkv[:, :heads] if with_q else None, rope=rope, interleaved=inter)
        return q, kp.clone(), vp.clone()

    (qa, ka, va), (qb, kb, vb) = both_ways(monkeypatch, call)
    assert torch.equal(ka, kb) and torch.equal(va, vb) and ka.any() and va.any()
    assert (qa is None and qb is None) if not with_q else torch.equal(qa, qb)


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lengths", [[0, 1, 70], [3000], [700, 2, 0, 1500]])
@pytest.mark.parametrize("scale,window", [(None, 0), (0.25, 0), (1, 100)])
def test_binding_and_general_way_agree_on_attention(monkeypatch, order, dtype, lengths, scale, window):
    kp, vp, table = pool(lengths, 16, 2, 64, dtype, order)
    q = torch.randn(len(lengths), 3, 6, 64, generator=gen(35)).to(dtype).cuda()[:, 1]
    ln = torch.tensor(lengths, dtype=torch.int32).cuda()
    a, b = both_ways(monkeypatch, lambda: fq.decode_attention(q, kp, vp, table, ln, scale=scale, window=window))
    assert torch.equal(a, b)


def test_refusals_of_cuda_tensors():
    """What does not fit is named the same through either way in."""
    w = weight(64, 128, NV, PLAIN)
    x = torch.zeros(2, 128, dtype=BF, device="cuda")
    for bad, why in ((x.float(), "bfloat16"), (x[:, :64], "columns"), (x[None], r"\[K\]"),
                     (x.cpu(), "device"), (x.t().contiguous().t(), "contiguous")):
        with pytest.raises(ValueError, match=why):
            fq.matvec(bad, w)
    with pytest.raises(ValueError, match="out_dtype"):
        fq.matvec(x, w, out_dtype=torch.int32)
    short = fq.Quantized(w.q, w.sf[:-1], w.s_dec, None, w.format, w.sf_layout)
    with pytest.raises(ValueError, match="scales"):
        fq.matvec(x, short)
    kp, vp, table = pool([20, 5], 16, 2, 64, BF)
    k, q = (torch.zeros(2, h, 64, dtype=BF, device="cuda") for h in (2, 4))
    ln = torch.tensor([20, 5], dtype=torch.int32).cuda()
    for args, why in (((q[:, :3], kp, vp, table, ln), "multiple"), ((q[:1], kp, vp, table, ln), "q must be"),
                      ((q, kp, vp, table, ln.long()), "int32"), ((q, kp, vp.half(), table, ln), "bfloat16"),
                      ((q, kp, vp, table.cpu(), ln), "device"), ((q, kp, vp, table.long(), ln), "int32"),
                      ((q.half(), kp, vp, table, ln), "dtype")):
        with pytest.raises(ValueError, match=why):
            fq.decode_attention(*args)
    with pytest.raises(ValueError, match="window"):
        fq.decode_attention(q, kp, vp, table, ln, window=-1)
    for args, kw, why in (((k[:, :1], k, kp, vp, table, ln), {}, "k must be"),
                          ((k, k.half(), kp, vp, table, ln), {}, "dtype"),
                          ((k, k, kp, vp, table, ln[:1]), {}, "int32"),
                          ((k, k, kp, vp, table[:1], ln), {}, "sequences"),
                          ((k, k, kp, vp, table, ln), dict(q=q[:, :3]), "multiple"),
                          ((k, k, kp, vp, table, ln), dict(rope=torch.zeros(4, 64).cuda().half()), "float32")):
        with pytest.raises(ValueError, match=why):
            fq.kv_append(*args, **kw)
    assert fq.fp4_status_sync() == fq.FP4_OK
