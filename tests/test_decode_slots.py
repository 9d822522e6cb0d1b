"""The decoding layer's cache where not every slot takes part in a step: pages
given back, slots without pages, sequences past their pages, paused ones."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300.decode import FP4DecodeAttention, PagedCache
from gpu_util import need_gpu
from test_decode import reference

H, HK, D, HIDDEN, PAGE = 8, 2, 64, 256, 8


def named(cache):
    """The pages that each row of the table names."""
    return [[p for p in row if p >= 0] for row in cache.table.tolist()]


def test_no_two_rows_name_one_page():
    c = PagedCache(4, 40, 2, 8, pages=7, page_size=16, device="cpu")
    assert named(c) == [[], [], [], []]
    c.reserve([32, 0, 16, 0])
    c.release(0)
    assert named(c)[0] == [] and int(c.lengths[0]) == 0
    c.reserve([0, 40, 16, 40])
    assert named(c) == c._owned
    pages = sum(named(c), [])
    assert len(pages) == len(set(pages)) == 7
    c.release(1)
    c.reserve([1, 0, 33, 40])
    assert named(c) == c._owned and len(set(sum(named(c), []))) == 7


def layer_of(seed=5, max_len=64, **kw):
    g = torch.Generator().manual_seed(seed)
    w = [(torch.randn(s, generator=g) * 0.06).to(torch.bfloat16).cuda()
         for s in (((H + 2 * HK) * D, HIDDEN), (HIDDEN, H * D))]
    return FP4DecodeAttention(*w, H, HK, D, max_len, **kw), g


def filled(cache, g):
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
    return cache


@pytest.mark.gpu
def test_slots_without_a_page_touch_nobody_elses():
    """A step with an unreserved, a released and an outgrown slot: reported,
    nothing written for them, their lengths unchanged, the live sequences as
    in a step that leaves those slots out."""
    need_gpu()
    layer, g = layer_of()
    cache = filled(PagedCache(5, 64, HK, D, page_size=PAGE), g)
    cache.reserve([20, 0, 24, 0, 8])
    cache.release(2)
    cache.reserve([20, 0, 0, 40, 8])  # takes the pages of the released slot
    lengths = torch.tensor([5, 0, 0, 17, 8], dtype=torch.int32)  # the last one is full
    x = torch.randn(5, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    k0, v0 = cache.k.clone(), cache.v.clone()
    skip = torch.tensor([5, -1, -1, 17, -1], dtype=torch.int32).cuda()
    cache.lengths.copy_(lengths)
    want = layer(x, cache, skip)
    assert fq.fp4_status_sync() == fq.FP4_OK
    want_k, want_v = cache.k.clone(), cache.v.clone()
    cache.k.copy_(k0)
    cache.v.copy_(v0)
    cache.lengths.copy_(lengths)
    got = layer(x, cache)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)
    changed = (cache.k != k0).flatten(2).any(-1).nonzero().tolist()
    assert sorted(changed) == sorted([[cache._owned[0][0], 5], [cache._owned[3][2], 1]])
    assert torch.equal(got[[0, 3]], want[[0, 3]])
    assert cache.lengths.tolist() == [6, 0, 0, 18, 8]
    # the full one goes on once it has pages
    cache.reserve([20, 0, 0, 40, 9])
    layer(x, cache, torch.tensor([-1, -1, -1, -1, 8], dtype=torch.int32).cuda())
    assert fq.fp4_status_sync() == fq.FP4_OK and int(cache.lengths[4]) == 9


@pytest.mark.gpu
def test_positions_past_the_rotation_table_do_not_count():
    """A table of rotations shorter than the pages: a position past it is
    reported and the length stays."""
    need_gpu()
    layer, g = layer_of(max_len=10)
    cache = filled(PagedCache(2, 16, HK, D, page_size=PAGE), g)
    cache.reserve([16, 16])
    cache.lengths.copy_(torch.tensor([10, 3], dtype=torch.int32))
    x = torch.randn(2, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    k0 = cache.k.clone()
    layer(x, cache)
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
    assert cache.lengths.tolist() == [10, 4]
    assert (cache.k != k0).flatten(2).any(-1).sum() == 1


@pytest.mark.gpu
def test_a_paused_sequence_goes_on_where_it_was():
    """A sequence left out of some steps (position -1) keeps its length and
    its history: its outputs are the bits of the same tokens without a pause,
    and what the 64-bit definition gives (tolerance as for a conversation)."""
    need_gpu()
    layer, g = layer_of()
    steps, pause = 14, range(5, 9)
    xs = torch.randn(steps, 3, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    cache = PagedCache(3, 32, HK, D, page_size=PAGE)
    cache.reserve([32] * 3)
    kept = []
    for i in range(steps):
        if i in pause:
            pos = cache.lengths.clone()
            pos[1] = -1
            y = layer(xs[i], cache, pos)
            assert (y[1] == 0).all() and int(cache.lengths[1]) == pause[0]
        else:
            y = layer(xs[i], cache)
            kept.append(y[1])
    assert cache.lengths.tolist() == [steps, steps - len(pause), steps]
    assert fq.fp4_status_sync() == fq.FP4_OK
    mine = [i for i in range(steps) if i not in pause]
    other = PagedCache(3, 32, HK, D, page_size=PAGE)
    other.reserve([32] * 3)
    alone = [layer(xs[i], other)[1] for i in mine]
    assert all(torch.equal(a, b) for a, b in zip(kept, alone))
    want = reference(layer, xs[mine][:, 1:2], [0])
    rms = want.pow(2).mean().sqrt()
    assert ((torch.stack(kept).cpu().double() - want[:, 0]).abs() <= 2.0 ** -4 * rms).all()


@pytest.mark.gpu
def test_a_step_of_another_size_is_refused_and_changes_nothing():
    need_gpu()
    layer, g = layer_of()
    cache = filled(PagedCache(3, 32, HK, D, page_size=PAGE), g)
    cache.reserve([32] * 3)
    cache.lengths.fill_(4)
    k0 = cache.k.clone()
    x = torch.randn(4, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    ints = torch.full((4,), 4, dtype=torch.int32, device="cuda")
    for bad in ((x[:2], cache, ints[:2]), (x[:2], cache), (x, cache, ints), (x[:3], cache, ints[:2]),
                (x[:3], cache, ints[:3].long()), (x[:3], cache, ints[:3].cpu()), (x[0], cache)):
        with pytest.raises(ValueError):
            layer(*bad)
        assert cache.lengths.tolist() == [4] * 3 and torch.equal(cache.k, k0)


@pytest.mark.gpu
def test_no_rotation():
    """rot_dim 0 rotates nothing: the step of a table of ones and zeros."""
    need_gpu()
    ys = []
    for rot in (0, D):
        layer, g = layer_of(rot_dim=rot)
        if rot:
            layer.rope[:, :D // 2] = 1
            layer.rope[:, D // 2:] = 0
        cache = PagedCache(2, 32, HK, D, page_size=PAGE)
        cache.reserve([32] * 2)
        xs = torch.randn(6, 2, HIDDEN, generator=g).to(torch.bfloat16).cuda()
        ys.append([layer(x, cache) for x in xs])
        seq = torch.zeros(4, dtype=torch.int32, device="cuda")
        layer.prefill(xs[:2].reshape(4, -1), cache, seq, torch.arange(4, dtype=torch.int32).cuda())
        ys[-1].append(cache.k[cache._owned[0][0], :4].clone())
    assert fq.fp4_status_sync() == fq.FP4_OK
    assert all(torch.equal(a, b) for a, b in zip(*ys))
