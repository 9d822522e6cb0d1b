"""The serving operators without a GPU: struct layouts, argument checks (made
before any launch), the rotation table and the tests' own definitions."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300 import build as fbuild
from fp4_block_scaled_quantize_gb300 import serve
from serve_ref import rotate, scale_values, tile, untile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIGN, UNSUPPORTED, SHAPE = (fq.FP4_OK, fq.FP4_ERR_INVALID_ARG, fq.FP4_ERR_ALIGNMENT,
                                          fq.FP4_ERR_UNSUPPORTED, fq.FP4_ERR_SHAPE)


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return serve._lib()


def test_struct_layouts_match_the_header():
    structs = (serve.fp4_kv_cache, serve.fp4_append_params, serve.fp4_attention_params)
    lines = []
    for s in structs:
        lines.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({s.__name__}, {f[0]}));' for f in s._fields_]
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "fp4.h"\nint main(void){'
           + "\n".join(lines) + "return 0;}")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in structs:
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


@pytest.mark.parametrize("packed,cls", [(serve._APPEND, serve.fp4_append_params),
                                        (serve._ATTENTION, serve.fp4_attention_params)])
def test_packed_structs_fill_the_ctypes_layout(packed, cls):
    """A packed struct read back as the ctypes class has every value in its field."""
    names = [f[0] for f in serve.fp4_kv_cache._fields_] + [f[0] for f in cls._fields_[1:]]
    values = [float(i) if n == "scale" else i + 1 for i, n in enumerate(names)]
    got = cls.from_buffer_copy(packed.pack(*values))
    n = len(serve.fp4_kv_cache._fields_)
    read = [getattr(got.cache, k) for k in names[:n]] + [getattr(got, k) for k in names[n:]]
    assert read == values


A = 4096  # an aligned address that is never followed


def test_matvec_refusals_before_any_launch(L):
    def call(rows=64, k=128, fmt=1, q=A, sf=A, sd=A, shift=None, layout=0, x=A, xs=None, xt=0, M=2,
             y=A, ys=None, yt=0):
        op = fq.fp4_operand(q, sf, sd, shift, fmt, rows, k)
        return L.fp4_matvec(ctypes.byref(op), layout, x, k if xs is None else xs, xt, M, y,
                            rows if ys is None else ys, yt, None)

    assert call(M=0) == OK and call(rows=0) == OK
    assert L.fp4_matvec(None, 0, A, 128, 0, 1, A, 64, 0, None) == INVALID
    assert call(fmt=9) == INVALID and call(layout=2) == INVALID
    assert call(xt=3) == INVALID and call(yt=-1) == INVALID
    assert call(xt=fq.FP4_F32) == UNSUPPORTED
    assert call(M=-1) == INVALID and call(rows=-1) == INVALID and call(xs=-1) == INVALID
    assert call(k=24) == SHAPE and call(fmt=2, k=48) == SHAPE and call(k=2 ** 31) == SHAPE
    assert call(xs=64) == SHAPE and call(ys=63) == SHAPE
    assert call(shift=A) == UNSUPPORTED and call(shift=A, layout=1) == UNSUPPORTED
    assert call(shift=A, fmt=0, layout=0) == UNSUPPORTED
    for missing in ("q", "sf", "sd", "x", "y"):
        assert call(**{missing: None}) == INVALID, missing
    assert call(q=A + 8) == ALIGN and call(sf=A + 4) == ALIGN and call(x=A + 1) == ALIGN
    assert call(sd=A + 2) == ALIGN and call(y=A + 2, yt=2) == ALIGN and call(y=A + 1) == ALIGN


def kv(**kw):
    d = dict(k=A, v=A, k_page=2048, k_place=128, k_head=64, v_page=2048, v_place=128, v_head=64,
             table=A, table_stride=4, pages=8, seqs=2, seq_pages=4, page_size=16, kv_heads=2,
             head_dim=64, type=0)
    d.update(kw)
    return fq.fp4_kv_cache(*[d[f[0]] for f in fq.fp4_kv_cache._fields_])


BAD_CACHES = [(dict(type=2), INVALID), (dict(type=-1), INVALID), (dict(pages=-1), INVALID),
              (dict(seqs=-1), INVALID), (dict(page_size=0), INVALID), (dict(kv_heads=0), INVALID),
              (dict(head_dim=0), INVALID), (dict(head_dim=264), SHAPE), (dict(k_place=-1), INVALID),
              (dict(seq_pages=2 ** 30), SHAPE), (dict(k=None), INVALID), (dict(v=None), INVALID),
              (dict(table=None), INVALID), (dict(table=A + 2), ALIGN), (dict(v=A + 1), ALIGN)]


@pytest.mark.parametrize("cache,code", BAD_CACHES)
def test_caches_are_refused_before_any_launch(L, cache, code):
    p = fq.fp4_append_params(cache=kv(**cache), k=A, v=A, pos=A, tokens=1)
    assert L.fp4_kv_append(ctypes.byref(p), None) == code
    p = fq.fp4_attention_params(cache=kv(**cache), lengths=A, q=A, out=A, heads=2)
    assert L.fp4_decode_attention(ctypes.byref(p), None) == code


def test_append_refusals_before_any_launch(L):
    def call(cache=None, **kw):
        d = dict(k=A, v=A, q=A, q_out=A, pos=A, rope=A, rope_len=8, tokens=2, heads=4, rot_dim=64)
        d.update(kw)
        p = fq.fp4_append_params(cache=cache or kv(), **d)
        return L.fp4_kv_append(ctypes.byref(p), None)

    assert L.fp4_kv_append(None, None) == INVALID
    assert call(tokens=0) == OK
    assert call(tokens=-1) == INVALID and call(tokens=2 ** 31) == SHAPE
    assert call(rot_dim=3) == SHAPE and call(rot_dim=66) == SHAPE and call(rot_dim=-2) == INVALID
    assert call(heads=3) == SHAPE and call(heads=0) == INVALID and call(q_out=None) == INVALID
    assert call(k=None) == INVALID and call(v=None) == INVALID and call(pos=None) == INVALID
    assert call(rope=None) == INVALID and call(rope_len=-1) == INVALID
    assert call(k_token=-8) == INVALID and call(qo_head=-8) == INVALID
    assert call(k=A + 1) == ALIGN and call(q=A + 1) == ALIGN and call(seq=A + 2) == ALIGN
    assert call(rope=A + 2) == ALIGN


def test_attention_refusals_before_any_launch(L):
    def call(cache=None, **kw):
        d = dict(lengths=A, q=A, out=A, q_seq=256, q_head=64, out_seq=256, out_head=64, heads=4,
                 workspace=A, workspace_bytes=2 ** 40, scale=0.125)
        d.update(kw)
        p = fq.fp4_attention_params(cache=cache or kv(), **d)
        return L.fp4_decode_attention(ctypes.byref(p), None)

    assert L.fp4_decode_attention(None, None) == INVALID
    assert call(cache=kv(seqs=0)) == OK
    assert call(heads=3) == SHAPE and call(heads=0) == INVALID and call(window=-1) == INVALID
    assert call(cache=kv(head_dim=60)) == SHAPE
    assert call(lengths=None) == INVALID and call(q=None) == INVALID and call(out=None) == INVALID
    assert call(q=A + 8) == ALIGN and call(q_head=60) == ALIGN and call(cache=kv(k_place=100)) == ALIGN
    assert call(cache=kv(v_page=2044)) == ALIGN and call(cache=kv(k=A + 8)) == ALIGN
    assert call(lse=A + 2) == ALIGN and call(out=A + 1) == ALIGN
    assert call(q_seq=-8) == INVALID
    f = L.fp4_decode_attention_workspace
    assert f(0, 64, 4, 2, 64) == 0
    assert f(2, 64, 3, 2, 64) == -1 and f(2, 64, 4, 0, 64) == -1 and f(2, 64, 4, 2, 60) == -1
    assert f(-1, 64, 4, 2, 64) == -1 and f(2, -1, 4, 2, 64) == -1


def test_python_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    q = fq.Quantized(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(32, dtype=torch.uint8),
                     torch.ones(1), None, fq.FP4_FMT_NVFP4_B16, fq.FP4_SF_PLAIN)
    x = torch.zeros(2, 64, dtype=bf)
    for bad, why in ((x, "CUDA"), (x.float(), "bfloat16"), (x[:, :32], "columns"), (x[None], r"\[K\]"),
                     (torch.zeros(64, 2, dtype=bf).t(), "contiguous")):
        with pytest.raises(ValueError, match=why):
            fq.matvec(bad, q)
    small = fq.Quantized(q.q, q.sf[:31], q.s_dec, None, q.format, q.sf_layout)
    with pytest.raises(ValueError, match="scales"):
        fq.matvec(x, small)
    with pytest.raises(ValueError, match="shifts"):
        fq.matvec(x, fq.Quantized(q.q, q.sf, q.s_dec, torch.zeros(8, dtype=torch.int8), q.format, 0))

    kp, vp = torch.zeros(4, 16, 2, 64, dtype=bf), torch.zeros(4, 16, 2, 64, dtype=bf)
    table, pos = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    k, heads = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 4, 64, dtype=bf)
    for args, kw, why in (
            ((k, k, kp, vp, table, pos), {}, "CUDA"),
            ((k.half(), k, kp, vp, table, pos), {}, "dtype"),
            ((k[:, :1], k, kp, vp, table, pos), {}, "k must be"),
            ((k, k, kp, vp, table, pos.long()), {}, "int32"),
            ((k, k, kp, vp, table.long(), pos), {}, "int32"),
            ((k, k, kp, vp, table[:2], pos), {}, "sequences"),
            ((k, k, kp[0], vp, table, pos), {}, "k_pages"),
            ((k, k, kp, vp.half(), table, pos), {}, "bfloat16"),
            ((k, k, kp, vp, table, pos), dict(rope=torch.zeros(4, 64, dtype=torch.float64)), "float32"),
            ((k, k, kp, vp, table, pos), dict(q_out=heads), "CUDA|without q")):
        with pytest.raises(ValueError, match=why):
            fq.kv_append(*args, **kw)
    ln = pos
    for args, kw, why in (((heads, kp, vp, table, ln), {}, "CUDA"),
                          ((heads[:, :3], kp, vp, table, ln), {}, "multiple"),
                          ((heads[:2], kp, vp, table, ln), {}, "q must be"),
                          ((heads, kp, vp, table, ln[:2]), {}, "lengths"),
                          ((heads, kp, vp, table, ln), dict(window=-1), "window"),
                          ((heads.half(), kp, vp, table, ln), {}, "dtype")):
        with pytest.raises(ValueError, match=why):
            fq.decode_attention(*args, **kw)


def test_rope_table():
    t = fq.rope_table(50, 8, base=100.0, device="cpu")
    assert t.shape == (50, 8) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.tensor([1.0] * 4 + [0.0] * 4))
    assert abs(float(t[7, 1]) - torch.cos(torch.tensor(7 * 100 ** -0.25, dtype=torch.float64)).item()) < 1e-7
    with pytest.raises(ValueError):
        fq.rope_table(4, 3)


def test_reference_definitions():
    """The tests' own definitions: the tiled layout, and rotations keep length."""
    c = torch.randint(0, 256, (300, 9)).to(torch.uint8)
    t = tile(c)
    assert torch.equal(untile(t, 300, 9), c)
    r, col = 201, 6  # tile (1, 1), line 201 % 32, word (201 % 128) / 32, byte 6 % 4
    assert t[(1 * 3 + 1) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + col % 4] == c[r, col]
    assert scale_values("e8m0")[127] == 1 and scale_values("e4m3")[0x7E] == 448
    x = torch.randn(4, 2, 16, dtype=torch.float64)
    pos = torch.tensor([0, 1, 5, 9])
    for inter in (False, True):
        y, _ = rotate(x, fq.rope_table(10, 16, device="cpu"), pos, inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
        assert torch.equal(y[0], x[0])


def test_the_binding_leaves_what_is_not_ordinary():
    """The compiled binding takes CUDA tensors that fit each other; anything
    else it leaves to the general way, without an exception."""
    b = serve._bind()
    x, p = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    for args in ((), (x,) * 8, (x, x, x, x, None, 0, 0, None), (1, 2, 3, 4, 5, 6, 7, 8),
                 (x, x, x, x, None, "a", 0, None), (torch.nn.Parameter(x), x, x, x, None, 0, 0, None),
                 (x.to_sparse(), x, x, x, None, 0, 0, None)):
        assert b.matvec(*args) is NotImplemented
    for args in ((), (x, x, p, p, i[None], i, None, None, None, False), (None,) * 10):
        assert b.append(*args) is NotImplemented
    for args in ((), (x, p, p, i[None], i, None, 0), (None,) * 7, (x, p, p, i[None], i, "a", 2 ** 70)):
        assert b.attention(*args) is NotImplemented
