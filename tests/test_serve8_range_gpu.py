"""Attention over a cache in 8 bits where the values' scales lie at the ends of
E8M0, and so far apart that a result is made of weights that binary32 does not
hold, and where queries are infinite: tolerances are those of test_serve8_gpu.py."""
import math

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from gpu_util import need_gpu
from test_serve8_gpu import BF, HF, check_attention, gen, ints, narrow, queries, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    need_gpu()
    fq.fp4_status_sync()
    yield


# rows of one warp, of a CTA, of a cluster; equal slices, joined wide and narrow
ROWS = [([40], 16, 1), ([300], 32, 8), ([1, 17, 200, 3, 90] * 20, 8, 2), ([20011], 32, 8), ([3000, 7, 9001, 0, 4096], 32, 8),
        ([5000] * 12, 8, 2)]


def rows_of(lengths, H, Hk, D, seed):
    need = [-(-n // 16) for n in lengths]
    cache = narrow(sum(need), 16, 16, Hk, D, seed=seed)
    return cache, tables(need, sum(need), seed=seed), queries(len(lengths), H, D, BF, seed), ints(lengths)


def unit_codes(cache, lo, hi, seed):
    """The values' scale codes anew, from [lo, hi); values of at most one unit."""
    cache[3].copy_(torch.randint(lo, hi, cache[3].shape, generator=gen(seed)))
    v = cache[1].view(torch.uint8)
    v.copy_(torch.where(v & 127 > 0x38, v & 0x80 | 0x38, v))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,H,Hk", ROWS)
@pytest.mark.parametrize("lo,hi", [(0, 1), (0, 8), (5, 12), (247, 255), (254, 255), (0, 255)])
def test_scales_at_the_ends(lo, hi, lengths, H, Hk, D):
    """Units of 2^-127 (what blocks of the smallest values have) to 2^127: BF16
    holds what comes out of all of them."""
    cache, table, q, ln = rows_of(lengths, H, Hk, D, 11)
    unit_codes(cache, lo, hi, 12)
    out = check_attention(q, cache, table, ln)
    assert torch.isfinite(out).all() and out.any()
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [40, 300, 2000, 9000, 40000])
def test_large_units_behind_small_weights(n, dtype):
    """The first half of a row at scores 104 below the second's, weights of 2^-150,
    with units of 2^127 for 2^-20: both halves make the result, and they are parts of
    their own where the row is cut."""
    H, Hk, D, page = 4, 2, 64, 8
    need = -(-n // page)
    cache = narrow(need, page, 8, Hk, D, seed=n)
    table = ints([list(range(need))])
    q = queries(1, H, D, dtype, 5)
    q[:, :, 0] = 8.0
    k = cache[0].view(torch.uint8)
    k.zero_()
    half = need // 2
    k[:half, :, :, 0], k[half:, :, :, 0] = 0x80 | 0x4D, 0x4D  # -6.5 and 6.5
    cache[2].fill_(127)
    cache[3][:half], cache[3][half:] = 254, 107
    v = cache[1].view(torch.uint8)
    v.copy_(torch.where(v & 127 > 0x50, v & 0x80 | 0x50, v))
    check_attention(q, cache, table, ints([n]), scale=1.0)
    cache[3][half:] = 0  # the second half next to nothing: the first one's is the result
    check_attention(q, cache, table, ints([n]), scale=1.0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("lengths,H,Hk", [([1, 0, 5], 4, 2)] + ROWS)
def test_infinite_queries_over_keys_of_one_sign(lengths, H, Hk, sign, dtype):
    """Every score of the head is the same infinity: the head and its lse are NaN,
    whichever it is; the others keep their accuracy (not their bits: a head whose
    maximum moves takes the warp's others along, an exponential's rounding, which
    check_attention's tolerance counts)."""
    cache, table, q, ln = rows_of(lengths, H, Hk, 64, 13)
    q = q.to(dtype)
    cache[0].view(torch.uint8)[..., 3] = 0x38
    q[:, :, 3] = 0.0
    q[:, 1, 3] = sign * math.inf
    check_attention(q, cache, table, ln)
    got, got_lse = fq.decode_attention(q, cache[0], cache[1], table, ln, k_scale=cache[2], v_scale=cache[3], return_lse=True)
    there = ln > 0
    assert torch.isnan(got[there, 1]).all() and torch.isnan(got_lse[there, 1]).all()
    assert not got[~there].any() and (got_lse[~there] == -math.inf).all()
