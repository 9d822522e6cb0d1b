"""The serving operators on values and layouts at the edge of what they take:
values that are not finite beside finite ones, scale bytes outside a weight,
several conditions in one status word, slices of attention in a chain."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from serve_ref import HALF_ULP, TINY, attention, tile
from test_serve_gpu import BF, F32, HF, MMA, MX, NV, PLAIN, UE, UE32, cache, check_matvec, close, gen, pool, random_copy

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    need_gpu()
    for _ in range(2):
        fq.fp4_status_sync()
    yield


# ------------------------------------------------- values that are not finite

def check_partly_finite(q, kp, vp, table, lengths):
    """Elements whose 64-bit value is finite lie within the operator's usual
    tolerance; the others are the same infinity or NaN."""
    D = q.shape[-1]
    want, wv, _, mag = attention(q, kp, vp, table, lengths, D ** -0.5, 0)
    got = fq.decode_attention(q, kp, vp, table, lengths).cpu().double()
    fine = torch.isfinite(want)
    assert not fine.all() and fine.any()
    d = (D / 16 + 8) * 2.0 ** -23 * mag
    sums = (lengths.cpu().double()[:, None] / 16 + 32) * 2.0 ** -23
    tol = (4 * d + 2.0 ** -14 + sums)[..., None] * wv + 2 * HALF_ULP[q.dtype] * want.abs() + 2 * TINY[q.dtype]
    close(got[fine], want[fine], tol[fine], "finite elements")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    odd = torch.isinf(want)
    assert torch.equal(got[odd], want[odd])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,hk,dim,page", [(8, 2, 128, 16), (4, 4, 64, 16), (16, 1, 64, 8), (32, 2, 128, 16),
                                               (6, 2, 192, 16), (8, 1, 256, 24), (10, 2, 80, 16)])
@pytest.mark.parametrize("lengths", [[21], [100, 90], [1000, 3], [9000, 5000]])
def test_attention_values_not_finite_leave_the_others_their_accuracy(dtype, heads, hk, dim, page, lengths):
    kp, vp, table = pool(lengths, page, hk, dim, dtype)
    q = torch.randn(len(lengths), heads, dim, generator=gen(50)).to(dtype).cuda()
    at = lambda s, p: (int(table[s, p // page]), p % page)  # noqa: E731
    last = lengths[0] - 1
    vp[at(0, 3)][0, 5] = float("inf")
    vp[at(0, last)][0, dim - 1] = float("-inf")
    vp[at(0, 7)][hk - 1, 9] = float("nan")
    vp[at(0, 2)][0, 17], vp[at(0, last // 2)][0, 17] = float("inf"), float("-inf")
    check_partly_finite(q, kp, vp, table, torch.tensor(lengths, dtype=torch.int32).cuda())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_a_query_head_that_is_not_finite_is_alone(dtype):
    kp, vp, table = pool([60, 700], 16, 2, 128, dtype)
    q = torch.randn(2, 8, 128, generator=gen(51)).to(dtype).cuda()
    ln = torch.tensor([60, 700], dtype=torch.int32).cuda()
    q[1, 2, 77] = float("nan")
    check_partly_finite(q, kp, vp, table, ln)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("away", [10.0, 30.0, 60.0])
def test_attention_small_weight_of_an_infinite_value(dtype, away):
    """A weight of e^-away is no zero: its infinity is the result."""
    kp, vp, table = pool([50], 16, 1, 64, dtype)
    kp[table[0, :4].long()] = 0
    q = torch.zeros(1, 2, 64, dtype=dtype, device="cuda")
    q[..., 0] = 8
    kp[table[0, 1], 4, 0, 0] = -away  # score 8 x -away / 8
    vp[table[0, 1], 4, 0, 6] = float("-inf")
    check_partly_finite(q, kp, vp, table, torch.tensor([50], dtype=torch.int32).cuda())


# ------------------------------------------------ scale bytes outside a weight

@pytest.mark.parametrize("fmt", [NV, UE, MX, UE32])
@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 7, 18, 33, 65])
@pytest.mark.parametrize("m", [1, 11])
def test_matvec_padding_of_the_tiled_scales_has_no_effect(fmt, blocks, m):
    """The tiled layout's bytes past a row's end and past the last row may hold
    anything."""
    block = 32 if fmt in (MX, UE32) else 16
    n, k = 75, blocks * block
    w = random_copy(n, k, fmt, MMA, seed=blocks)
    x = torch.randn(m, k, generator=gen(52)).to(BF).cuda()
    y = fq.matvec(x, w, out_dtype=F32)
    cols = k // (16 if fmt == UE32 else block)
    view = w.sf.view(1, -(-cols // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)  # [tile row, word, line, tile column, byte]
    inside = torch.zeros(128, -(-cols // 4) * 4, dtype=torch.bool, device="cuda")
    inside[:n, :cols] = True
    inside = inside.view(1, 4, 32, -1, 4)
    for code in (0xFF, 0x7F, 0xFE, 0x80):
        view[~inside] = code
        assert torch.equal(fq.matvec(x, w, out_dtype=F32), y), code


@pytest.mark.parametrize("layout", [PLAIN, MMA])
@pytest.mark.parametrize("m", [1, 9])
def test_matvec_e8m0_codes_of_every_size(layout, m):
    """Rows whose codes span 30 binades each, from 2^-107 to 2^103."""
    n, k = 181, 1152
    w = random_copy(n, k, MX, PLAIN, seed=70)
    codes = 20 + torch.arange(n)[:, None] + torch.randint(0, 31, (n, k // 32), generator=gen(71))
    codes = codes.to(torch.uint8)
    sf = tile(codes) if layout == MMA else codes.contiguous().view(-1)
    w = fq.Quantized(w.q, sf.cuda(), w.s_dec, None, MX, layout)
    x = torch.randn(m, k, generator=gen(72)).cuda()
    check_matvec(x.to(BF), w, F32)
    check_matvec(x.to(HF), w, F32)


@pytest.mark.parametrize("layout", [PLAIN, MMA])
@pytest.mark.parametrize("m", [1, 5, 16])
@pytest.mark.parametrize("k", [96, 512, 1024])
def test_matvec_e8m0_nan_is_nan(layout, m, k):
    """E8M0 255 is NaN: the rows that hold one are NaN, no other changes."""
    n = 200
    w = random_copy(n, k, MX, layout, seed=k)
    x = torch.randn(m, k, generator=gen(53)).to(HF).cuda()
    y = fq.matvec(x, w, out_dtype=F32)
    cols, rows = k // 32, [0, 31, 77, n - 1]
    for i, r in enumerate(rows):
        c = (i * 5) % cols
        at = r * cols + c if layout == PLAIN else (r // 128 * -(-cols // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
        w.sf[at] = 255
    z = fq.matvec(x, w, out_dtype=F32)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[rows] = True
    assert torch.isnan(z[:, bad]).all() and torch.equal(z[:, ~bad], y[:, ~bad])


# ------------------------------------------------------------- the status word

def test_a_bad_index_is_not_lost_beside_another_condition():
    kp, vp = cache(2, 4, 1, 64, BF)
    k = torch.zeros(1, 1, 64, dtype=BF, device="cuda")
    ints = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731

    def bad_index():
        fq.kv_append(k, k, kp, vp, ints(9)[None], ints(0))

    bad_index()
    fq.amax(torch.full((16, 64), float("nan"), dtype=BF, device="cuda"))
    assert fq.fp4_status_sync() == fq.FP4_ERR_NONFINITE
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert fq.fp4_status_sync() == fq.FP4_OK
    bad_index()
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG and fq.fp4_status_sync() == fq.FP4_OK


# ----------------------------------------------------------- slices in a chain

@pytest.mark.parametrize("seqs,heads,hk,dim,longest", [(1, 8, 2, 128, 9000), (40, 8, 4, 64, 2500), (6, 16, 8, 128, 4000)])
def test_attention_by_slices_in_a_chain(seqs, heads, hk, dim, longest):
    """Steps of product, append, attention by slices (a second launch joins the
    rows, wide for few of them and narrow for many) and product, lengths
    changing in between, back to back and from a graph: the bits of the same
    steps with a wait after every call."""
    page, hidden, steps = 16, heads * dim, 5
    wide = -(-(longest + steps) // page)
    assert fq.fp4_decode_attention_workspace(seqs, wide * page, heads, hk, dim) > 0
    kp, vp = cache(seqs * wide, page, hk, dim, BF)
    table = torch.randperm(seqs * wide, generator=gen(60)).view(seqs, wide).to(torch.int32).cuda()
    start = torch.randint(1, longest, (seqs,), generator=gen(61), dtype=torch.int32)
    start[0] = longest
    start = start.cuda()
    w = [random_copy(n, k, NV, MMA, seed=n) for n, k in (((heads + 2 * hk) * dim, hidden), (hidden, hidden))]
    x0 = torch.randn(seqs, hidden, generator=gen(62)).to(BF).cuda()
    rope = fq.rope_table(longest + steps, dim)
    old, lengths = (kp.clone(), vp.clone()), start.clone()

    def reset():
        kp.copy_(old[0])
        vp.copy_(old[1])
        lengths.copy_(start)

    def run(wait):
        x, kept = x0, []
        for _ in range(steps):
            qkv = fq.matvec(x, w[0]).view(seqs, heads + 2 * hk, dim)
            wait()
            q, k, v = (qkv * qkv.abs().amax().reciprocal()).split([heads, hk, hk], 1)
            q = fq.kv_append(k, v, kp, vp, table, lengths, q=q, rope=rope)
            wait()
            lengths.add_(1)
            a = fq.decode_attention(q, kp, vp, table, lengths)
            wait()
            y = fq.matvec(a.view(seqs, -1), w[1])
            wait()
            x = y * y.abs().amax().reciprocal()
            kept += [q, a, y]
        return kept

    reset()
    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(t).all() for t in want)
    for _ in range(5):
        reset()
        got = run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        reset()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = run(lambda: None)
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fq.fp4_status_sync() == fq.FP4_OK
