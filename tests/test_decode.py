"""The decoding layer: page accounting on the host, and on the GPU a
conversation stepped token by token against the whole computation in 64 bits
on the layer's own dequantised weights."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300.decode import FP4DecodeAttention, PagedCache
from fp4_block_scaled_quantize_gb300.linear import FP4Linear
from gpu_util import need_gpu
from serve_ref import rotate, weight_values


def test_pages_are_counted():
    c = PagedCache(3, 40, 2, 8, pages=5, page_size=16, device="cpu")
    c.reserve([17, 0, 16])
    owned = [list(o) for o in c._owned]
    assert [len(o) for o in owned] == [2, 0, 1] and len(set(sum(owned, []))) == 3
    assert c.table[0, :2].tolist() == owned[0]
    c.reserve([17, 20, 3])  # what a sequence has stays
    assert c._owned[0] == owned[0] and len(c._owned[1]) == 2 and not c._free
    with pytest.raises(RuntimeError):
        c.reserve([33, 20, 3])
    assert [len(o) for o in c._owned] == [2, 2, 1]
    c.release(1)
    c.reserve([33, 0, 0])
    assert len(c._owned[0]) == 3
    with pytest.raises(ValueError):
        c.reserve([41, 0, 0])
    with pytest.raises(ValueError):
        c.reserve([1, 1])
    with pytest.raises(ValueError):
        PagedCache(0, 4, 1, 8, device="cpu")


def reference(layer, xs, start, interleaved=False, window=0):
    """Outputs of every step for tokens xs [steps, seqs, hidden], sequence s
    beginning at position start[s], in 64 bits."""
    wq, wo = weight_values(layer.w_qkv), weight_values(layer.w_o)
    H, Hk, D = layer.heads, layer.kv_heads, layer.head_dim
    steps, seqs, _ = xs.shape
    qkv = (xs.cpu().double() @ wq.t()).view(steps, seqs, H + 2 * Hk, D)
    out = torch.zeros(steps, seqs, wo.shape[0], dtype=torch.float64)
    for s in range(seqs):
        pos = torch.arange(steps) + start[s]
        q, _ = rotate(qkv[:, s, :H], layer.rope, pos, interleaved)
        k, _ = rotate(qkv[:, s, H:H + Hk], layer.rope, pos, interleaved)
        v = qkv[:, s, H + Hk:]
        for i in range(steps):
            j = slice(max(0, i + 1 - window) if window else 0, i + 1)
            score = torch.einsum("kgd,nkd->kgn", q[i].view(Hk, H // Hk, D), k[j]) * D ** -0.5
            a = torch.einsum("kgn,nkd->kgd", torch.softmax(score, -1), v[j])
            out[i, s] = a.reshape(-1) @ wo.t()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,window,interleaved", [(fq.FP4_FMT_UE5M3_B16, 0, False),
                                                    (fq.FP4_FMT_NVFP4_B16, 7, True)])
def test_conversation_matches_the_whole_computation(fmt, window, interleaved):
    """Tolerance: q, k, v, the attention's and the layer's output are each
    rounded to BF16 (2^-9 of their size); a relative change of 2^-8 in q and k
    moves a score of size up to 4 by 2^-6, a weight by as much.  Summed over
    the output product that is well under 2^-5 of the output's root mean
    square, taken per element as 2^-4 of it."""
    need_gpu()
    g = torch.Generator().manual_seed(3)
    hidden, H, Hk, D, seqs, steps = 256, 8, 2, 64, 3, 21
    qkv = FP4Linear(hidden, (H + 2 * Hk) * D, format=fmt)
    o = FP4Linear(H * D, hidden, format=fmt)
    with torch.no_grad():
        qkv.weight.copy_(torch.randn(qkv.weight.shape, generator=g) * hidden ** -0.5)
        o.weight.copy_(torch.randn(o.weight.shape, generator=g) * (H * D) ** -0.5)
    layer = FP4DecodeAttention.from_linear(qkv, o, H, Hk, D, 64, window=window, interleaved=interleaved)
    cache = PagedCache(seqs, 64, Hk, D, page_size=8)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    xs = torch.randn(steps, seqs, hidden, generator=g).to(torch.bfloat16).cuda()
    want = reference(layer, xs, [0] * seqs, interleaved, window)
    for i in range(steps):
        cache.reserve([i + 1] * seqs)
        y = layer(xs[i], cache)
        assert cache.lengths.tolist() == [i + 1] * seqs
        err = (y.cpu().double() - want[i]).abs()
        rms = want[i].pow(2).mean().sqrt()
        assert (err <= 2.0 ** -4 * rms).all(), (i, float(err.max() / rms))
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.gpu
def test_prefill_then_steps_in_a_graph():
    """Prompts written in one call, then steps replayed from one CUDA graph:
    the same outputs as stepping through all tokens."""
    need_gpu()
    g = torch.Generator().manual_seed(4)
    hidden, H, Hk, D, seqs, prompt, steps = 128, 4, 4, 32, 2, 9, 5
    w = torch.randn((H + 2 * Hk) * D, hidden, generator=g).to(torch.bfloat16).cuda() * 0.1
    wo = torch.randn(hidden, H * D, generator=g).to(torch.bfloat16).cuda() * 0.1
    layer = FP4DecodeAttention(w, wo, H, Hk, D, 32)
    xs = torch.randn(prompt + steps, seqs, hidden, generator=g).to(torch.bfloat16).cuda()
    one = PagedCache(seqs, 32, Hk, D, page_size=16)
    one.reserve([32] * seqs)
    ys = [layer(x, one).clone() for x in xs][prompt:]

    two = PagedCache(seqs, 32, Hk, D, page_size=16)
    two.reserve([32] * seqs)
    seq = torch.arange(seqs).repeat(prompt).to(torch.int32).cuda()
    pos = torch.arange(prompt).repeat_interleave(seqs).to(torch.int32).cuda()
    layer.prefill(xs[:prompt].reshape(-1, hidden), two, seq, pos)
    x = torch.empty_like(xs[0])
    two.lengths.fill_(prompt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a first call outside the graph
        x.copy_(xs[prompt])
        layer(x, two)
    torch.cuda.current_stream().wait_stream(side)
    two.lengths.fill_(prompt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, two)
    two.lengths.fill_(prompt)
    for i in range(steps):
        x.copy_(xs[prompt + i])
        graph.replay()
        assert torch.equal(y, ys[i]), i
    assert two.lengths.tolist() == [prompt + steps] * seqs
    assert fq.fp4_status_sync() == fq.FP4_OK


@pytest.mark.gpu
def test_weights_that_do_not_fit_are_refused():
    need_gpu()
    w = torch.zeros(96, 64, dtype=torch.bfloat16, device="cuda") + 1
    with pytest.raises(ValueError):
        FP4DecodeAttention(w, w, 3, 2, 16, 8)
    with pytest.raises(ValueError):
        FP4DecodeAttention(w, w, 4, 2, 16, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,hidden,heads,hk,dim,start", [(1, 512, 8, 2, 64, 0), (7, 256, 4, 4, 64, 40),
                                                            (2, 1024, 8, 1, 128, 900)])
def test_calls_in_a_row_wait_for_each_other(seqs, hidden, heads, hk, dim, start):
    """Steps issued back to back, each call reading what the one before it
    wrote, give the bits of the same steps with a wait after every call; so do
    the same steps from a CUDA graph."""
    need_gpu()
    g = torch.Generator().manual_seed(seqs)
    w = [(torch.randn(s, generator=g) * 0.06).to(torch.bfloat16).cuda()
         for s in (((heads + 2 * hk) * dim, hidden), (hidden, heads * dim))]
    steps = 6
    layer = FP4DecodeAttention(*w, heads, hk, dim, start + steps)
    up = fq.quantize(w[1], fq.amax(w[1])[0], fq.params(format=fq.FP4_FMT_NVFP4_B16))
    x0 = torch.randn(seqs, hidden, generator=g).to(torch.bfloat16).cuda()
    cache = PagedCache(seqs, start + steps, hk, dim, page_size=16)
    cache.reserve([start + steps] * seqs)
    old = [torch.randn(cache.k.shape, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]

    def reset():
        cache.k.copy_(old[0])
        cache.v.copy_(old[1])
        cache.lengths.fill_(start)

    def run(wait):
        x, kept = x0, []
        for _ in range(steps):
            # the layer's calls, one by one: each depends on the one before
            pos = cache.lengths.clone()
            qkv = fq.matvec(x, layer.w_qkv).view(seqs, heads + 2 * hk, dim)
            wait()
            q, k, v = qkv.split([heads, hk, hk], 1)
            q = fq.kv_append(k, v, cache.k, cache.v, cache.table, pos, q=q, rope=layer.rope)
            wait()
            cache.lengths.add_(1)
            a = fq.decode_attention(q, cache.k, cache.v, cache.table, cache.lengths)
            wait()
            y = fq.matvec(a.view(seqs, -1), layer.w_o)
            wait()
            z = fq.matvec(a.view(seqs, -1), up, out=y)  # over what was just written
            wait()
            x = fq.matvec(z.view(seqs, -1)[:, :hidden], layer.w_qkv)[:, :hidden]
            wait()
            kept += [qkv, q, a, z, x]
        return kept

    reset()
    want = run(torch.cuda.synchronize)
    for _ in range(10):
        reset()
        got = run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        reset()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = run(lambda: None)
    for _ in range(5):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.isfinite(t).all() for t in want)
