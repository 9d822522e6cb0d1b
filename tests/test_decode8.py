"""The decoding layer over a cache in 8 bits, with first positions that stay
visible, and with pages handed out on the device."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300.decode import FP4DecodeAttention, PagedCache
from gpu_util import need_gpu
from serve8_ref import seen_positions
from serve_ref import rotate, weight_values

E4M3, I32 = torch.float8_e4m3fn, torch.int32
H, HK, D, HIDDEN = 8, 2, 64, 256


def make_layer(seed=3, max_len=64, **kw):
    g = torch.Generator().manual_seed(seed)
    w = [(torch.randn(s, generator=g) * s[1] ** -0.5).to(torch.bfloat16).cuda() for s in (((H + 2 * HK) * D, HIDDEN), (HIDDEN, H * D))]
    return FP4DecodeAttention(*w, H, HK, D, max_len, **kw), g


def test_caches_say_what_they_are():
    c = PagedCache(2, 40, 2, 16, page_size=32, dtype=E4M3, device="cpu")
    assert c.k.dtype == E4M3 and c.k_scale.shape == (4, 2, 2) and c.v_scale.dtype == torch.uint8
    assert PagedCache(2, 40, 2, 16, page_size=24, dtype=E4M3, device="cpu").k_scale.shape == (4, 1, 2)
    assert PagedCache(2, 40, 2, 16, page_size=24, block=6, dtype=E4M3, device="cpu").v_scale.shape == (4, 4, 2)
    assert PagedCache(2, 40, 2, 16, device="cpu").k_scale is None
    for kw in (dict(block=5, dtype=E4M3), dict(block=0, dtype=E4M3), dict(block=16)):
        with pytest.raises(ValueError, match="block"):
            PagedCache(2, 40, 2, 16, page_size=32, device="cpu", **kw)
    with pytest.raises(ValueError, match="host"):
        c.plan(torch.zeros(2, dtype=I32))
    c = PagedCache(2, 40, 2, 16, pages=3, device="cpu", on_device=True)
    assert c.pool.tolist() == [3, 0, 2, 1, 0]
    with pytest.raises(ValueError, match="device"):
        c.reserve([1, 1])
    with pytest.raises(ValueError, match="device"):
        c.release(0)


def expected(layer, cache, x, pos, window, sinks):
    """The layer's output for one token of each sequence over what the cache
    holds (read back), in 64 bits; rows at position -1 are zero."""
    wq, wo = weight_values(layer.w_qkv), weight_values(layer.w_o)
    qkv = (x.cpu().double() @ wq.t()).view(len(pos), H + 2 * HK, D)
    q, _ = rotate(qkv[:, :H], layer.rope, torch.tensor(pos).clamp(min=0), False)
    out = torch.zeros(len(pos), wo.shape[0], dtype=torch.float64)
    for s, p in enumerate(pos):
        if p < 0:
            continue
        at = seen_positions(p + 1, window, sinks)
        k, v = cache.read(torch.full((len(at),), s, dtype=I32, device="cuda"), torch.tensor(at, dtype=I32, device="cuda"))
        score = torch.einsum("kgd,nkd->kgn", q[s].view(HK, H // HK, D), k.cpu().double()) * D ** -0.5
        out[s] = torch.einsum("kgn,nkd->kgd", torch.softmax(score, -1), v.cpu().double()).reshape(-1) @ wo.t()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,page,block,window,sinks", [(E4M3, 16, 16, 0, 0), (E4M3, 12, 4, 9, 3), (torch.bfloat16, 16, None, 9, 3)])
def test_steps_over_what_the_cache_holds(dtype, page, block, window, sinks):
    """A prompt, then steps in which sequences come, go and wait.  Tolerance as
    for the 16-bit conversation: queries, attention and output are each rounded
    to BF16, per element under 2^-4 of the output's root mean square."""
    need_gpu()
    layer, g = make_layer(window=window, sinks=sinks)
    cache = PagedCache(3, 64, HK, D, pages=9, page_size=page, dtype=dtype, block=block, on_device=True)
    plan = cache.plan(torch.tensor([19, 0, 5], dtype=I32, device="cuda"), tokens=26)
    layer.prefill(torch.randn(26, HIDDEN, generator=g).to(torch.bfloat16).cuda(), cache, plan.seq, plan.pos)
    assert cache.lengths.tolist() == [19, 0, 5]
    for i in range(14):
        if i == 6:
            cache.plan(torch.tensor([-100, 0, 0], dtype=I32, device="cuda"))  # the first one ends
        new = torch.tensor([int(i < 6 or i > 9), int(i > 2), int(i % 3 > 0)], dtype=I32, device="cuda")
        x = torch.randn(3, HIDDEN, generator=g).to(torch.bfloat16).cuda()
        pos = cache.step(new)
        before = cache.lengths.tolist()
        y = layer(x, cache, pos)
        assert cache.lengths.tolist() == before
        want = expected(layer, cache, x, pos.tolist(), window, sinks)
        err = (y.cpu().double() - want).abs().max() / want.pow(2).mean().sqrt()
        assert err <= 2.0 ** -4, (i, float(err))
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.gpu
def test_a_graph_hands_out_its_own_pages():
    """Steps captured together with cache.step go on over page borders, and give
    the bits of eager steps over pages reserved on the host; where pages run
    out a sequence stays, and the step says so."""
    need_gpu()
    layer, g = make_layer()
    a = PagedCache(2, 64, HK, D, page_size=4, dtype=E4M3, block=4)
    b = PagedCache(2, 64, HK, D, pages=6, page_size=4, dtype=E4M3, block=4, on_device=True)
    xs = torch.randn(14, 2, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    a.reserve([64, 64])
    layer(xs[0], PagedCache(2, 8, HK, D, dtype=E4M3, on_device=True), torch.zeros(2, dtype=I32, device="cuda") - 1)  # warm up
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos = b.step()
        y = layer(x, b, pos)
    for i in range(12):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(y, layer(xs[i], a)), i
    assert fq.fp4_status_sync() == fq.FP4_OK
    x.copy_(xs[12])
    graph.replay()  # position 12: no page left
    assert pos.tolist() == [-1, -1] and b.lengths.tolist() == [12, 12] and not y.any()
    assert fq.fp4_status_sync() == fq.FP4_ERR_INVALID_ARG
