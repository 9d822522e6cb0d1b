"""page_plan up to a length that is not whole pages: all results are integers and
have to be equal."""
import ctypes

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300 import build as fbuild
from fp4_block_scaled_quantize_gb300 import serve
from fp4_block_scaled_quantize_gb300.decode import FP4DecodeAttention, PagedCache
from gpu_util import need_gpu
from serve8_ref import Pages

I32, A = torch.int32, 4096


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def test_refusals_before_any_launch():
    fbuild.build()
    p = fq.fp4_plan_params(new_tokens=A, lengths=A, room=A, table=A, table_stride=4, pool=A, pool_pages=8, tokens=-1, seqs=2,
                           seq_pages=4, page_size=16)
    assert serve._lib().fp4_page_plan_within(ctypes.byref(p), -1, None) == fq.FP4_ERR_INVALID_ARG
    assert serve._lib().fp4_page_plan_within(None, 5, None) == fq.FP4_ERR_INVALID_ARG
    i = torch.zeros(2, dtype=I32)
    for most, why in ((-1, "max_len"), (3, "CUDA")):
        with pytest.raises(ValueError, match=why):
            fq.page_plan(i, i, torch.zeros(2, 3, dtype=I32), i, torch.zeros(5, dtype=I32), 16, max_len=most)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,wide,page,most,few", [(5, 9, 8, 61, False), (300, 6, 16, 81, False), (300, 3, 4, 9, True),
                                                     (700, 5, 16, 9, True), (40, 400, 16, 6001, False), (3, 4, 8, 0, False),
                                                     (3, 4, 8, 10 ** 12, False), (64, 20, 7, 133, False)])
def test_sequences_up_to_a_length(seqs, wide, page, most, few):
    """Random steps: what would pass stays as it is and has places -1, as if it
    were not there for the rest."""
    need_gpu()
    fq.fp4_status_sync()
    lengths, room = ints([0] * seqs), ints([0] * seqs)
    table, pool = torch.full((seqs, wide), -1, dtype=I32, device="cuda"), fq.page_pool(seqs * wide)
    ref = Pages(lengths, table, room, pool, page)
    g = torch.Generator().manual_seed(seqs)
    top = min(most, wide * page)
    passed = 0
    for step in range(14):
        new = torch.randint(-4, 5, (seqs,), generator=g) if few else torch.randint(-top // 2 - 3, top + 9, (seqs,), generator=g)
        if step % 3 == 2:
            new = torch.ones(seqs, dtype=torch.long)
        new = new.tolist()
        over = [n > 0 and L + n > top for n, L in zip(new, ref.lengths)]
        passed += sum(over)
        total = sum(max(n, 0) for n in new)
        tokens = total + 5 if step % 2 else None
        got = fq.page_plan(ints(new), lengths, table, room, pool, page, tokens=tokens, max_len=most)
        want, refused = ref.plan([0 if o else n for n, o in zip(new, over)], tokens)
        assert not refused and (fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG) == any(over)
        assert lengths.tolist() == ref.lengths and room.tolist() == ref.room and table.tolist() == ref.table
        assert pool.tolist()[2:2 + len(ref.free)] == ref.free and pool[0] == len(ref.free)
        if tokens is None:
            continue
        seq, pos, slot, at = [], [], [], 0
        for s, (n, o) in enumerate(zip(new, over)):
            seq += [s] * n
            if o:
                pos += [-1] * n
                slot += [-1] * n
            elif n > 0:
                pos += want[1][at:at + n]
                slot += want[2][at:at + n]
                at += n
        pad = [-1] * (tokens - total)
        assert got.seq.tolist() == seq + pad and got.pos.tolist() == pos + pad and got.slot.tolist() == slot + pad
        assert got.offsets.tolist() == [sum(max(m, 0) for m in new[:s]) for s in range(seqs + 1)]
    assert passed or most > wide * page


@pytest.mark.gpu
def test_more_than_the_limit_already():
    """Lengths past the limit stay without new tokens, and may shrink."""
    need_gpu()
    fq.fp4_status_sync()
    st = ints([20, 20, 20]), torch.tensor([[0, 1, 2], [3, 4, 5], [6, 7, 8]], dtype=I32, device="cuda"), ints([24] * 3)
    pool = ints([0, 0] + [0] * 9)
    fq.page_plan(ints([0, -3, -10]), *st, pool, 8, max_len=12)
    assert fq.fp4_status_sync() == fq.FP4_OK
    assert st[0].tolist() == [20, 17, 10] and st[2].tolist() == [24, 24, 16] and pool[:3].tolist() == [1, 0, 8]
    fq.page_plan(ints([1, 0, 2]), *st, pool, 8, max_len=12)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG and st[0].tolist() == [20, 17, 12]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
def test_a_cache_keeps_its_max_len(dtype):
    """On the device as on the host: no position past max_len, in the middle of a
    page, is given, and none is counted that the layer's rotation does not reach."""
    need_gpu()
    fq.fp4_status_sync()
    g = torch.Generator().manual_seed(3)
    w = [(torch.randn(s, generator=g) * 0.06).to(torch.bfloat16).cuda() for s in ((256, 128), (128, 128))]
    layer = FP4DecodeAttention(*w, 2, 1, 64, 100)
    cache = PagedCache(2, 100, 1, 64, page_size=64, dtype=dtype, on_device=True)
    p = cache.plan(ints([101, 99]), tokens=200)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert cache.lengths.tolist() == [0, 99] and p.pos.tolist()[:101] == [-1] * 101
    x = torch.randn(200, 128, generator=g).to(torch.bfloat16).cuda()
    layer.prefill(x, cache, p.seq, p.pos)
    assert cache.step().tolist() == [0, 99] and cache.lengths.tolist() == [1, 100]
    assert fq.fp4_status_sync() == fq.FP4_OK
    pos = cache.step()
    y = layer(x[:2], cache, pos)
    assert pos.tolist() == [1, -1] and cache.lengths.tolist() == [2, 100] and not y[1].any()
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("most,given", [(10, [0, 9]), (2 ** 64 + 5, [12, 9])])
def test_the_general_way(most, given):
    """Another stream; a limit that no integer of the library holds is none."""
    need_gpu()
    fq.fp4_status_sync()
    st = ints([0, 0]), torch.full((2, 4), -1, dtype=I32, device="cuda"), ints([0, 0])
    pool, new = fq.page_pool(8), ints([12, 9])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, None):
        got = fq.page_plan(new, *st, pool, 4, tokens=21, max_len=most, stream=stream)
        torch.cuda.synchronize()
        assert st[0].tolist() == given and got.pos.tolist() == list(range(12)) * bool(given[0]) + [-1] * 12 * (not given[0]) + list(range(9))
        assert (fq.fp4_status_sync() == fq.FP4_OK) == (given[0] == 12)
        fq.page_plan(ints([-12, -9]), *st, pool, 4)
