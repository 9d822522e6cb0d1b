"""The order of a call's tokens in kv_append to a cache in 8 bits: those of one
block stand side by side, or the call is reported."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from serve8_ref import Cache8
from test_serve8_gpu import BF, cache8, check_cache, few_bits, gen, ints, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    need_gpu()
    fq.fp4_status_sync()
    yield
    torch.cuda.synchronize()
    fq.fp4_status_sync()


def append(c, table, seq, pos, x):
    fq.kv_append(x[:, :1], x[:, 1:], c[0], c[1], table, ints(pos), seq=ints(seq), k_scale=c[2], v_scale=c[3])
    return fq.fp4_status_sync()


def stand_apart(seq, pos, block):
    """By definition: a block whose tokens are not neighbours in ascending order."""
    groups = {}
    for t, (s, p) in enumerate(zip(seq, pos)):
        if p >= 0:
            groups.setdefault((s, p // block), []).append((t, p))
    return any(b[0] != a[0] + 1 or b[1] != a[1] + 1 for g in groups.values() for a, b in zip(g, g[1:]))


@pytest.mark.parametrize("seqs,steps", [(5, 3), (40, 2), (700, 4)])
@pytest.mark.parametrize("start", [0, 3])
def test_drafts_by_step_and_by_sequence(seqs, steps, start):
    """[step][sequence] is reported; [sequence][step] holds what it should."""
    c = cache8(seqs, 16, 16, 1, 32)
    table, ref = tables([1] * seqs, seqs), Cache8(*c)
    x = few_bits((seqs * steps, 2, 32), BF, 1)
    seq, pos = [s for s in range(seqs) for _ in range(steps)], [start + j for _ in range(seqs) for j in range(steps)]
    assert append(c, table, seq, pos, x) == fq.FP4_OK
    ref.append(x[:, :1], x[:, 1:], table, torch.tensor(pos), torch.tensor(seq), None, False)
    check_cache(c, ref)
    seq, pos = [s for _ in range(steps) for s in range(seqs)], [start + j for j in range(steps) for _ in range(seqs)]
    assert append(c, table, seq, pos, x) == fq.FP4_ERR_INVALID_ARG


@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (24, 8), (64, 64), (20, 4)])
@pytest.mark.parametrize("seqs,longest", [(1, 20), (4, 100), (60, 30), (300, 12), (3, 900)])
def test_layouts_at_random(page, block, seqs, longest):
    """Runs of all sequences, cut at random places or at blocks' ends and put in any
    order, with tokens that are left out between them: reported if and only if a
    block's tokens stand apart."""
    g = gen(seqs + page)
    need = -(-longest // page) + 1
    c = cache8(seqs * need, page, block, 1, 16)
    table = tables([need] * seqs, seqs * need)
    seen = set()
    for case in range(24):
        runs = []
        for s in range(seqs):
            n, at = int(torch.randint(0, longest + 1, (1,), generator=g)), int(torch.randint(0, page, (1,), generator=g))
            end = at + n
            while at < end:
                k = int(torch.randint(1, n + 1, (1,), generator=g)) if case % 3 else n
                k = min(k, end - at)
                if case % 3 == 1 and at + k < end:  # only at blocks' ends
                    k = min((at + k + block - 1) // block * block, end) - at
                runs.append([(s, at + j) for j in range(k)])
                at += k
        order = torch.randperm(len(runs), generator=g).tolist()
        tokens = []
        for i in order:
            tokens += runs[i] + ([(0, -1)] if case % 4 == 3 else [])
        if case == 23 and len(tokens) > 1:  # one of them at the other end
            tokens.append(tokens.pop(0))
        if not tokens:
            continue
        seq, pos = [s for s, _ in tokens], [p for _, p in tokens]
        apart = stand_apart(seq, pos, block)
        seen.add(apart)
        got = append(c, table, seq, pos, few_bits((len(seq), 2, 16), BF, case))
        assert (got == fq.FP4_ERR_INVALID_ARG) == apart, case
    assert False in seen and (True in seen or block == 1)


def test_the_same_place_twice_inside_a_block():
    c, x = cache8(3, 16, 16, 1, 16), few_bits((4, 2, 16), BF, 1)
    assert append(c, tables([1] * 3, 3), [0, 1, 0, 2], [5, 5, 5, 5], x) == fq.FP4_ERR_INVALID_ARG
    assert append(c, tables([1] * 3, 3), [0, 0, 1, 2], [5, 5, 5, 5], x) == fq.FP4_ERR_INVALID_ARG
    assert append(c, tables([1] * 3, 3), [0, 0, 1, 2], [5, 6, 5, 5], x) == fq.FP4_OK


@pytest.mark.parametrize("apart", [False, True])
def test_more_tokens_than_are_looked_at_together(apart):
    """Two tokens of one block, side by side or at the two ends of a large call of
    single tokens."""
    T = 100000
    c = cache8(T, 2, 2, 1, 16)
    table = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    seq, pos = list(range(T)), [1] * T
    pos[0] = 0
    if apart:
        seq[T - 1] = 0
    else:
        seq[1] = 0
    x = torch.randn(T, 2, 16, generator=gen(1)).to(BF).cuda()
    assert append(c, table, seq, pos, x) == (fq.FP4_ERR_INVALID_ARG if apart else fq.FP4_OK)


def test_other_calls_are_left_alone():
    """Whole prompts and single tokens, without seq, with blocks of one place."""
    c, x = cache8(64, 16, 1, 1, 16), few_bits((40, 2, 16), BF, 1)
    assert append(c, tables([4] * 10, 64), [i % 10 for i in range(40)], [i // 10 for i in range(40)], x) == fq.FP4_OK
    c = cache8(64, 16, 16, 1, 16)
    fq.kv_append(x[:, :1], x[:, 1:], c[0], c[1], tables([1] * 40, 64), ints([7] * 40), k_scale=c[2], v_scale=c[3])
    assert fq.fp4_status_sync() == fq.FP4_OK
    assert append(c, tables([4], 64), [0] * 40, list(range(3, 43)), x) == fq.FP4_OK
