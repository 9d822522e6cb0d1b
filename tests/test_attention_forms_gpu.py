"""The two forms of attention over a cache in 16 bits: with first positions that
stay visible, and without."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from test_serve8_gpu import BF, HF, check_attention, gen, ints, queries, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("H,Hk,D,page", [(32, 8, 128, 16), (16, 16, 64, 32), (40, 2, 64, 16), (32, 2, 128, 24), (4, 2, 192, 16), (8, 2, 256, 64)])
@pytest.mark.parametrize("lengths", [[300], [9001], [500] * 8, [0, 4000, 17, 2500, 1] * 3])
def test_first_positions_that_change_nothing(lengths, H, Hk, D, page, dtype):
    """A window over everything makes both forms see the same: the same bits; and
    each is what the definition says."""
    need_gpu()
    fq.fp4_status_sync()
    need = [-(-n // page) for n in lengths]
    g = gen(H)
    cache = [torch.randn(sum(need), page, Hk, D, generator=g).to(dtype).cuda() for _ in range(2)] + [None, None]
    table, q, ln = tables(need, sum(need)), queries(len(lengths), H, D, dtype), ints(lengths)
    plain = check_attention(q, cache, table, ln)
    assert torch.equal(check_attention(q, cache, table, ln, window=2 ** 31 - 1, sinks=3), plain)
    check_attention(q, cache, table, ln, window=150)
    check_attention(q, cache, table, ln, window=150, sinks=40)
    assert fq.fp4_status_sync() == fq.FP4_OK
