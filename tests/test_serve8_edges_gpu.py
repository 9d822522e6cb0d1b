"""The operators around a cache in 8 bits where sizes, addresses and the order of
calls are at their ends."""
import math

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from serve8_ref import E4M3, Cache8, Pages
from test_serve8_gpu import (BF, HF, I32, cache8, check_attention, check_cache, check_plan, few_bits, gen, ints, narrow,
                             queries, state, tables)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    need_gpu()
    fq.fp4_status_sync()
    yield
    torch.cuda.synchronize()
    fq.fp4_status_sync()


@pytest.mark.parametrize("D", [32, 48, 112, 144, 160, 176, 208, 224, 240])
@pytest.mark.parametrize("page", [32, 20])
def test_every_head_size(D, page):
    """Heads that fill no piece of what a warp copies: append, read, attention."""
    need = [4, 9]
    k, v, ks, vs = cache8(13, page, page // 4, 3, D, seed=D)
    table = tables(need, 13)
    ref = Cache8(k, v, ks, vs)
    n = [3 * page + 5, 9 * page - 1]
    seq, pos = ints([0] * n[0] + [1] * n[1]), ints(list(range(n[0])) + list(range(n[1])))
    x = few_bits((sum(n), 6, D), HF, D)
    fq.kv_append(x[:, :3], x[:, 3:], k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
    ref.append(x[:, :3], x[:, 3:], table, pos.cpu(), seq.cpu(), None, False)
    check_cache((k, v, ks, vs), ref)
    at = table.cpu().long()[seq.cpu().long(), pos.cpu().long() // page]
    got = fq.kv_read(k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs, dtype=BF)
    for t, which in zip(got, "kv"):
        assert torch.equal(t.cpu().double(), ref.values(which)[at, pos.cpu().long() % page])
    check_attention(queries(2, 6, D, BF), (k, v, ks, vs), table, ints(n))
    check_attention(queries(2, 6, D, HF), (k, v, ks, vs), table, ints(n), window=40, sinks=19)


def test_a_block_as_long_as_a_long_page():
    k, v, ks, vs = cache8(3, 300, 300, 2, 64)
    table = tables([3], 3)
    ref = Cache8(k, v, ks, vs)
    done = 0
    for n in (290, 1, 305, 4):
        x = few_bits((n, 4, 64), BF, n, 2.0 ** (done / 100))
        seq, pos = ints([0] * n), ints(list(range(done, done + n)))
        fq.kv_append(x[:, :2], x[:, 2:], k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
        ref.append(x[:, :2], x[:, 2:], table, pos.cpu(), seq.cpu(), None, False)
        check_cache((k, v, ks, vs), ref, f"{n} more")
        done += n


def test_one_key_head_many_short_runs():
    """Groups of lanes with runs of their own, of different lengths, some with
    infinities, some that do not fit a group's rows."""
    g = gen(3)
    lens = torch.randint(1, 9, (400,), generator=g).tolist()
    start = torch.randint(0, 30, (400,), generator=g).tolist()
    k, v, ks, vs = cache8(1200, 16, 8, 1, 128)
    table = tables([3] * 400, 1200)
    ref = Cache8(k, v, ks, vs)
    seq = ints([s for s, n in enumerate(lens) for _ in range(n)])
    pos = ints([a + j for a, n in zip(start, lens) for j in range(n)])
    T = len(seq)
    x = few_bits((T, 2, 128), BF, 4)
    hit = torch.randint(0, T, (40,), generator=g)
    x[hit, hit % 2, hit % 128] = math.inf
    x[hit[:10], 0, 5] = math.nan
    fq.kv_append(x[:, :1], x[:, 1:], k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs)
    ref.append(x[:, :1], x[:, 1:], table, pos.cpu(), seq.cpu(), None, False)
    check_cache((k, v, ks, vs), ref)


def test_far_pages():
    """A cache of more than 2^31 elements: its last pages, and pages further
    apart than 32 bits."""
    page, H, D, P = 64, 8, 128, 33000
    big = [torch.empty(P, page, H, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.zeros(P, 4, H, dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = narrow(5, page, 16, H, D, seed=1)
    where = [P - 1, 0, P - 2, 17, P - 5]
    for i, at in enumerate(where):
        for t, f in zip(big + scales, small):
            t.view(torch.uint8)[at] = f.view(torch.uint8)[i]
    q, ln = queries(1, 32, D, BF), ints([300])
    near, far = ints([[0, 1, 2, 3, 4]]), ints([where])
    pos, seq = ints(list(range(300))), ints([0] * 300)
    x = torch.randn(20, 2 * H, D, generator=gen(2)).to(BF).cuda()

    def run(k, v, ks, vs, table):
        a = fq.decode_attention(q, k, v, table, ln, k_scale=ks, v_scale=vs)
        fq.kv_append(x[:, :H], x[:, H:], k, v, table, ints(list(range(295, 315))), seq=seq[:20], k_scale=ks, v_scale=vs)
        return (a, fq.decode_attention(q, k, v, table, ints([315]), window=100, sinks=3, k_scale=ks, v_scale=vs),
                *fq.kv_read(k, v, table, pos, seq=seq, k_scale=ks, v_scale=vs))

    copy = [t.clone() for t in small]
    want = run(*copy, near)
    assert all(torch.equal(a, b) for a, b in zip(run(*big, *scales, far), want))
    del big
    step = 2 ** 31 + 4096
    flat = torch.empty(2 * step + 2 ** 20 + page * H * D, dtype=torch.uint8, device="cuda")
    wide = [flat[o:].as_strided((3, page, H, D), (step, H * D, D, 1)) for o in (0, 2 ** 20)]
    for t, f in zip(wide, small):
        t.copy_(f.view(torch.uint8)[:3])
    copy = [t[:3].clone() for t in small]
    out = []
    for k, v in ((copy[0], copy[1]), (wide[0].view(E4M3), wide[1].view(E4M3))):
        out.append((fq.decode_attention(q, k, v, near[:, :3], ints([150]), k_scale=copy[2], v_scale=copy[3]),
                    *fq.kv_read(k, v, near[:, :3], pos[:180], seq=seq[:180], k_scale=copy[2], v_scale=copy[3])))
    assert all(torch.equal(a, b) for a, b in zip(out[1][1:], out[0][1:]))
    # (other sums of the same terms: a BF16 rounding apart, 2^-9 of each at most)
    assert (out[0][0].float() - out[1][0].float()).abs().max() <= 2.0 ** -8 * out[0][0].float().abs().max()


def test_nothing_to_do():
    k, v, ks, vs = cache8(2, 16, 16, 2, 64)
    table, none = ints([[0, 1]]), torch.zeros(0, dtype=I32, device="cuda")
    e = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    assert fq.kv_append(e, e, k, v, table, none, seq=none, k_scale=ks, v_scale=vs) is None
    got = fq.kv_read(k, v, table, none, seq=none, k_scale=ks, v_scale=vs)
    assert got[0].shape == (0, 2, 64)
    out = fq.decode_attention(torch.zeros(0, 4, 64, dtype=BF, device="cuda"), k, v, table[:0], none, k_scale=ks, v_scale=vs)
    assert out.shape == (0, 4, 64)
    p = fq.page_plan(none, none, table[:0], none, fq.page_pool(3), 16, tokens=5)
    assert p.seq.tolist() == [-1] * 5 and p.offsets.tolist() == [0]
    st = state(2, 0, 0)  # rows without pages, a pool without pages
    assert fq.page_plan(ints([0, 3]), st["lengths"], st["page_table"], st["room"], st["pool"], 16, tokens=0).offsets.tolist() == [0, 0, 3]
    assert st["lengths"].tolist() == [0, 0] and fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG


def test_plan_extremes():
    """Counts and lengths at the ends of 32 bits, a pool that is fuller than
    itself, pages that go back where others are given out in the same call."""
    st = state(4, 8, 12)
    ref = Pages(st["lengths"], st["page_table"], st["room"], st["pool"], 4)
    check_plan(st, ref, [9, 32, 0, 7], 4, 60)
    check_plan(st, ref, [2 ** 31 - 1, -2 ** 31, 1, 2 ** 31 - 1], 4, None)
    check_plan(st, ref, [-3, 30, 1, -2], 4, 31)
    check_plan(st, ref, [20, -9, 0, -5], 4, 25)
    check_plan(st, ref, [-2 ** 31] * 4, 4, 3)
    assert sorted(st["pool"].tolist()[2:]) == list(range(12))
    st["pool"][0] = 99  # more than there are: as many as there are
    fq.page_plan(ints([1, 0, 0, 0]), st["lengths"], st["page_table"], st["room"], st["pool"], 4)
    assert st["pool"][0] == 11 and fq.fp4_status_sync() == fq.FP4_OK


def test_two_graphs_replayed_in_turn():
    """Append and attention captured twice, for two caches, replayed in turn and
    among eager calls: each gives what eager calls give."""
    H, Hk, D, page = 16, 4, 128, 16
    x = [torch.randn(5, H + 2 * Hk, D, generator=gen(i)).to(BF).cuda() for i in range(2)]
    rope = fq.rope_table(4096, D)

    def make(i):
        c = narrow(5 * 160, page, 16, Hk, D, seed=i)
        return c, tables([160] * 5, 800, seed=i), ints([300 * i + 500, 2000, 17, 1000, 2500 - 900 * i])

    def step(c, table, ln, x):
        q = fq.kv_append(x[:, H:H + Hk], x[:, H + Hk:], c[0], c[1], table, ln, q=x[:, :H], rope=rope, k_scale=c[2], v_scale=c[3])
        ln += 1
        return fq.decode_attention(q, c[0], c[1], table, ln, k_scale=c[2], v_scale=c[3])

    a, b = [make(i) for i in range(2)], [make(i) for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        step(*make(i), x[i])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*a[i], x[i]))
        graphs.append(g)
    for n in range(6):
        for i in (0, 1) if n % 2 else (1, 0):
            graphs[i].replay()
            want = step(*b[i], x[i])
            assert torch.equal(outs[i], want), (n, i)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [step(*b[i], x[i]) for i in range(2)]
        s.synchronize()
    for i in range(2):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], got[i])
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("seqs,longest", [(1, 9000), (33, 700), (200, 90)])
def test_parts_repeat_exactly(codes, seqs, longest):
    """The same call gives the same bits, whatever ran before it."""
    page, Hk, D = 16, 4, 64
    lengths = torch.randint(0, longest + 1, (seqs,), generator=gen(seqs)).tolist()
    lengths[-1] = longest
    need = [-(-n // page) for n in lengths]
    if codes:
        c = narrow(sum(need), page, 16, Hk, D)
    else:
        c = [torch.randn(sum(need), page, Hk, D, generator=gen(i)).to(HF).cuda() for i in (1, 2)] + [None, None]
    table, q, ln = tables(need, sum(need)), queries(seqs, 8, D, HF), ints(lengths)
    call = lambda: fq.decode_attention(q, c[0], c[1], table, ln, window=400, sinks=7, k_scale=c[2], v_scale=c[3])  # noqa: E731
    first = call()
    for _ in range(20):
        assert torch.equal(call(), first)
