"""The decoding layer as a module: its weights are its state."""
import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300.decode import FP4DecodeAttention
from gpu_util import need_gpu

H, HK, D, HIDDEN = 8, 2, 64, 256


def copy_of(rows, k, seed, fmt=fq.FP4_FMT_UE5M3_B16):
    g = torch.Generator().manual_seed(seed)
    p = lambda *s: torch.randint(0, 100, s, generator=g, dtype=torch.int32).to(torch.uint8)  # noqa: E731
    sf = p(fq.fp4_sf_bytes(fmt, rows, k, fq.FP4_SF_MMA))
    return fq.Quantized(p(rows, k // 2), sf, torch.rand(1, generator=g),
                        torch.zeros(rows, dtype=torch.int8), fmt, fq.FP4_SF_MMA)


def test_the_weights_are_the_modules_state():
    """A saved layer holds its weights; loading them, and moving the module,
    changes what it multiplies."""
    def make(seed):
        return FP4DecodeAttention(copy_of((H + 2 * HK) * D, HIDDEN, seed), copy_of(HIDDEN, H * D, seed + 1), H, HK, D, 8)

    a, b = make(1), make(2)
    state = a.state_dict()
    for name in ("w_qkv", "w_o"):
        w = getattr(a, name)
        for part in (w.q, w.sf, w.s_dec, w.row_shift):
            assert any(t.shape == part.shape and torch.equal(t, part) for t in state.values())
    assert not torch.equal(a.w_qkv.q, b.w_qkv.q)
    b.load_state_dict(state)
    for name in ("w_qkv", "w_o"):
        x, y = getattr(a, name), getattr(b, name)
        for part in ("q", "sf", "s_dec", "row_shift"):
            assert torch.equal(getattr(x, part), getattr(y, part))
        assert (x.format, x.sf_layout) == (y.format, y.sf_layout)
    c = make(3)
    c.load_state_dict({k: v.clone() for k, v in state.items()}, assign=True)
    assert torch.equal(c.w_o.q, a.w_o.q)
    moved = make(1).to("meta")
    assert moved.w_qkv.q.is_meta and moved.w_o.sf.is_meta and moved.w_o.row_shift.is_meta
    # the format travels with them
    d = FP4DecodeAttention(copy_of((H + 2 * HK) * D, HIDDEN, 5, fmt=fq.FP4_FMT_UE5M3_B32), copy_of(HIDDEN, H * D, 6),
                           H, HK, D, 8)
    d.load_state_dict(state)
    assert d.w_qkv.format == fq.FP4_FMT_UE5M3_B16


@pytest.mark.gpu
def test_a_loaded_layer_answers_as_the_saved_one():
    need_gpu()
    from fp4_block_scaled_quantize_gb300.decode import PagedCache
    g = torch.Generator().manual_seed(9)

    def make():
        w = [(torch.randn(s, generator=g) * 0.06).to(torch.bfloat16).cuda()
             for s in (((H + 2 * HK) * D, HIDDEN), (HIDDEN, H * D))]
        return FP4DecodeAttention(*w, H, HK, D, 16)

    def answer(layer):
        cache = PagedCache(2, 16, HK, D, page_size=8)
        cache.reserve([4, 4])
        return layer(x, cache)

    x = torch.randn(2, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    a, b = make(), make()
    want = answer(a)
    assert not torch.equal(want, answer(b))
    b.load_state_dict(a.state_dict())
    assert torch.equal(want, answer(b))
    assert torch.equal(want, answer(a.cpu().cuda()))
