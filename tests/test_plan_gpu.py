"""page_plan's two ways on the GPU against the definition on lists
(serve8_ref.py): few tokens a sequence, and pages that come and go in one call
of many CTAs.  All results are integers and have to be equal."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from serve8_ref import Pages

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    need_gpu()
    fq.fp4_status_sync()
    yield


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class State:
    def __init__(self, seqs, wide, pages, page):
        self.lengths, self.room = ints([0] * seqs), ints([0] * seqs)
        self.table = torch.full((seqs, wide), -1, dtype=torch.int32, device="cuda")
        self.pool, self.page = fq.page_pool(pages), page
        self.ref = Pages(self.lengths, self.table, self.room, self.pool, page)

    def step(self, new, tokens):
        got = fq.page_plan(ints(new), self.lengths, self.table, self.room, self.pool, self.page, tokens=tokens)
        want, refused = self.ref.plan(new, tokens)
        assert (fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG) == refused
        if tokens is None:
            assert got is None
        else:
            for name, a, b in zip(("seq", "pos", "slot", "offsets"), got, want):
                assert a.tolist() == b, name
        assert self.lengths.tolist() == self.ref.lengths and self.room.tolist() == self.ref.room
        assert self.table.tolist() == self.ref.table
        pool = self.pool.tolist()
        assert pool[0] == len(self.ref.free) and pool[1] == 0 and pool[2:2 + pool[0]] == self.ref.free
        return refused


@pytest.mark.parametrize("seqs,wide,pages,page", [(1, 3, 3, 2), (7, 4, 20, 1), (200, 6, 500, 3), (511, 2, 900, 4), (512, 5, 1200, 2),
                                                  (513, 5, 1200, 2)])
def test_few_tokens(seqs, wide, pages, page):
    """Up to four tokens more or fewer, five in some steps; batches that are too
    small, that fit, and that go on over several CTAs; full rows, an empty pool."""
    st = State(seqs, wide, pages, page)
    g = torch.Generator().manual_seed(seqs)
    refusals = 0
    for step in range(20):
        low = -4 if step % 5 == 4 else -1
        new = torch.randint(low, 6 if step % 7 == 6 else 5, (seqs,), generator=g)
        if step % 6 == 5:
            new = torch.ones(seqs, dtype=torch.long)
        new = new.tolist()
        total = sum(max(n, 0) for n in new)
        refusals += st.step(new, [None, total, total + 7001, total * 2 // 3][(step + step // 4) % 4])
    assert refusals  # of rows, pages or places, in some step


def test_few_tokens_where_rooms_are_larger():
    """Sequences whose pages hold far more than their tokens give the rest back
    with the first token that goes."""
    st = State(3, 50, 120, 2)
    st.step([80, 60, 7], 147)
    st.lengths.copy_(ints([5, 60, 0]))
    st.ref.lengths = [5, 60, 0]
    st.step([-1, 2, -4], 2)
    st.step([4, -3, 4], None)


@pytest.mark.parametrize("seqs,wide,pages,page", [(300, 40, 3000, 4), (512, 30, 2500, 16), (700, 20, 4000, 3)])
def test_pages_both_ways_over_many_ctas(seqs, wide, pages, page):
    """Prompts and ends in one call: what goes back lies on places of the stack
    that other CTAs read."""
    st = State(seqs, wide, pages, page)
    g = torch.Generator().manual_seed(pages)
    for step in range(12):
        new = torch.randint(0, wide * page, (seqs,), generator=g)
        ends = torch.rand(seqs, generator=g) < (0.0 if step == 0 else 0.6)
        new = torch.where(ends, torch.tensor(-2 ** 31), new // (1 + step % 3)).tolist()
        total = sum(max(n, 0) for n in new)
        st.step(new, [total, total + 9000, None][step % 3])


def test_captured_steps_repeat():
    """A captured decoding step that gives tokens out and takes them back leaves
    every word as it was, however often it is replayed."""
    st = State(256, 8, 1500, 4)
    st.step([13 + s % 9 for s in range(256)], None)
    start = [t.clone() for t in (st.lengths, st.room, st.table, st.pool)]
    more, less = ints([1 + s % 4 for s in range(256)]), ints([-1 - s % 4 for s in range(256)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        maps = fq.page_plan(more, st.lengths, st.table, st.room, st.pool, 4, tokens=5000)
        fq.page_plan(less, st.lengths, st.table, st.room, st.pool, 4)
    for _ in range(50):
        graph.replay()
    want, _ = st.ref.plan(more.tolist(), 5000)
    assert [t.tolist() for t in maps] == list(want)
    assert all(torch.equal(a, b) for a, b in zip((st.lengths, st.room, st.table, st.pool), start))
    assert fq.fp4_status_sync() == fq.FP4_OK
