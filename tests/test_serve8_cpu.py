"""The operators around a cache in 8 bits without a GPU: struct layouts,
argument checks (made before any launch), and the tests' own definitions."""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

import fp4_block_scaled_quantize_gb300 as fq
from fp4_block_scaled_quantize_gb300 import build as fbuild
from fp4_block_scaled_quantize_gb300 import serve
from serve8_ref import E4M3, Cache8, Pages, nearest_e4m3, need_code, seen_positions

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIGN, SHAPE = fq.FP4_OK, fq.FP4_ERR_INVALID_ARG, fq.FP4_ERR_ALIGNMENT, fq.FP4_ERR_SHAPE
A = 4096  # an aligned address that is never followed


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return serve._lib()


STRUCTS = (serve.fp4_kv_scales, serve.fp4_append8_params, serve.fp4_attention8_params, serve.fp4_read_params,
           serve.fp4_plan_params)


def test_struct_layouts_match_the_header():
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({s.__name__}, {f[0]}));' for f in s._fields_]
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "fp4.h"\nint main(void){' + "\n".join(lines) + "return 0;}")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in STRUCTS:
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def leaves(obj, cls):
    """Values of a struct's fields in order, its parts' fields in their places."""
    out = []
    for name, kind in cls._fields_:
        v = getattr(obj, name)
        out += leaves(v, kind) if issubclass(kind, ctypes.Structure) else [v]
    return out


@pytest.mark.parametrize("packed,cls,n", [(lambda v: serve._APPEND.pack(*v[:37]) + serve._SCALES.pack(*v[37:]), serve.fp4_append8_params, 46),
                                          (lambda v: serve._READ.pack(*v), serve.fp4_read_params, 35),
                                          (lambda v: serve._PLAN.pack(*v), serve.fp4_plan_params, 15)])
def test_packed_structs_fill_the_ctypes_layout(packed, cls, n):
    values = list(range(1, n + 1))
    assert leaves(cls.from_buffer_copy(packed(values)), cls) == values


def cache(**kw):
    d = dict(k=A, v=A, k_page=2048, k_place=128, k_head=64, v_page=2048, v_place=128, v_head=64, table=A, table_stride=4,
             pages=8, seqs=2, seq_pages=4, page_size=16, kv_heads=2, head_dim=64, type=0)
    d.update(kw)
    return fq.fp4_kv_cache(*[d[f[0]] for f in fq.fp4_kv_cache._fields_])


def scales(**kw):
    d = dict(k_sf=A, v_sf=A, k_page=4, k_block=2, k_head=1, v_page=4, v_block=2, v_head=1, block=8)
    d.update(kw)
    return fq.fp4_kv_scales(*[d[f[0]] for f in fq.fp4_kv_scales._fields_])


BAD = [(dict(type=2), {}, INVALID), (dict(page_size=0), {}, INVALID), (dict(head_dim=264), {}, SHAPE),
       (dict(head_dim=72), {}, SHAPE), (dict(k=None), {}, INVALID), (dict(table=A + 2), {}, ALIGN),
       (dict(k=A + 8), {}, ALIGN), (dict(v_place=72), {}, ALIGN), ({}, dict(block=0), INVALID),
       ({}, dict(block=5), SHAPE), ({}, dict(block=32), SHAPE), ({}, dict(k_sf=None), INVALID),
       ({}, dict(v_sf=None), INVALID), ({}, dict(v_block=-1), INVALID), ({}, dict(k_page=-2), INVALID)]


@pytest.mark.parametrize("c,s,code", BAD)
def test_caches_are_refused_before_any_launch(L, c, s, code):
    p = fq.fp4_append8_params(fq.fp4_append_params(cache=cache(**c), k=A, v=A, pos=A, tokens=1), scales(**s))
    assert L.fp4_kv_append8(ctypes.byref(p), None) == code
    a = fq.fp4_attention_params(cache=cache(**c), lengths=A, q=A, out=A, heads=2, workspace=A, workspace_bytes=1 << 40)
    assert L.fp4_decode_attention8(ctypes.byref(fq.fp4_attention8_params(a, scales(**s))), None) == code
    r = fq.fp4_read_params(cache=cache(**c), scales=scales(**s), k_out=A, v_out=A, pos=A, tokens=1)
    if s.get("k_sf", A):  # (without: a cache in 16 bits, refused for its lone scales)
        assert L.fp4_kv_read(ctypes.byref(r), None) == code


def test_append_refusals_before_any_launch(L):
    def call(**kw):
        d = dict(k=A, v=A, q=A, q_out=A, pos=A, rope=A, rope_len=8, tokens=2, heads=4, rot_dim=64)
        d.update(kw)
        p = fq.fp4_append8_params(fq.fp4_append_params(cache=cache(), **d), scales())
        return L.fp4_kv_append8(ctypes.byref(p), None)

    assert L.fp4_kv_append8(None, None) == INVALID
    assert call(tokens=0) == OK
    assert call(tokens=-1) == INVALID and call(rot_dim=3) == SHAPE and call(rot_dim=66) == SHAPE
    assert call(heads=3) == SHAPE and call(q_out=None) == INVALID and call(k=None) == INVALID and call(pos=None) == INVALID
    assert call(rope=None) == INVALID and call(k_token=-8) == INVALID and call(k=A + 1) == ALIGN and call(seq=A + 2) == ALIGN


def test_attention_refusals_before_any_launch(L):
    def call(**kw):
        d = dict(lengths=A, q=A, out=A, q_seq=256, q_head=64, out_seq=256, out_head=64, heads=4, workspace=A,
                 workspace_bytes=2 ** 40, scale=0.125)
        d.update(kw)
        a = fq.fp4_attention_params(cache=cache(seqs=d.pop("seqs", 2), seq_pages=d.pop("seq_pages", 4)), **d)
        return L.fp4_decode_attention8(ctypes.byref(fq.fp4_attention8_params(a, scales())), None)

    assert L.fp4_decode_attention8(None, None) == INVALID
    assert call(seqs=0) == OK
    assert call(heads=3) == SHAPE and call(window=-1) == INVALID and call(sinks=-1) == INVALID
    assert call(lengths=None) == INVALID and call(q=A + 8) == ALIGN and call(q_head=60) == ALIGN and call(lse=A + 2) == ALIGN
    assert call(seq_pages=10 ** 6, workspace_bytes=16) == INVALID
    a = fq.fp4_attention_params(cache=cache(), lengths=A, q=A, out=A, q_seq=256, q_head=64, heads=4, sinks=-1)
    assert L.fp4_decode_attention(ctypes.byref(a), None) == INVALID
    f = L.fp4_decode_attention8_workspace
    assert f(0, 64, 4, 2, 64) == 0 and f(2, 64, 3, 2, 64) == -1 and f(2, 64, 4, 2, 72) == -1 and f(-1, 64, 4, 2, 64) == -1


def test_read_refusals_before_any_launch(L):
    def call(c=None, s=None, **kw):
        d = dict(k_out=A, v_out=A, k_token=128, k_out_head=64, v_token=128, v_out_head=64, pos=A, tokens=2)
        d.update(kw)
        return L.fp4_kv_read(ctypes.byref(fq.fp4_read_params(cache=c or cache(), scales=s or scales(), **d)), None)

    none = fq.fp4_kv_scales()
    assert L.fp4_kv_read(None, None) == INVALID
    assert call(tokens=0) == OK and call(s=none, tokens=0) == OK
    assert call(tokens=-1) == INVALID and call(k_token=-8) == INVALID and call(tokens=2 ** 31) == SHAPE
    assert call(k_out=None) == INVALID and call(v_out=None) == INVALID and call(pos=None) == INVALID
    assert call(k_out=A + 8) == ALIGN and call(v_token=124) == ALIGN and call(seq=A + 1) == ALIGN
    assert call(c=cache(head_dim=68), s=none) == SHAPE and call(c=cache(k_place=68), s=none) == ALIGN
    assert call(s=scales(k_sf=None)) == INVALID


def test_plan_refusals_before_any_launch(L):
    def call(**kw):
        d = dict(new_tokens=A, lengths=A, room=A, table=A, table_stride=4, pool=A, pool_pages=8, offsets=A, seq=A, pos=A, slot=A,
                 tokens=4, seqs=2, seq_pages=4, page_size=16)
        d.update(kw)
        return L.fp4_page_plan(ctypes.byref(fq.fp4_plan_params(**d)), None)

    assert L.fp4_page_plan(None, None) == INVALID
    for name in ("new_tokens", "lengths", "room", "table", "pool"):
        assert call(**{name: None}) == INVALID, name
    for name in ("seqs", "seq_pages", "pool_pages", "table_stride"):
        assert call(**{name: -1}) == INVALID, name
    assert call(page_size=0) == INVALID and call(seq_pages=2 ** 28) == SHAPE and call(tokens=2 ** 31) == SHAPE
    assert call(slot=A + 4) == ALIGN and call(pos=A + 2) == ALIGN and call(pool=A + 1) == ALIGN


def test_python_refusals():
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    kp = torch.zeros(4, 16, 2, 64, dtype=u8).view(E4M3)
    sc = torch.zeros(4, 2, 2, dtype=u8)
    table, pos = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    k, heads = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 4, 64, dtype=bf)
    both = dict(k_scale=sc, v_scale=sc)
    for args, kw, why in (
            ((k, k, kp, kp, table, pos), both, "CUDA"),
            ((k, k, kp, kp, table, pos), {}, "needs k_scale"),
            ((k, k, kp, kp, table, pos), dict(k_scale=sc), "needs k_scale"),
            ((k, k, kp.float().to(bf), kp.float().to(bf), table, pos), both, "belong"),
            ((k, k, kp, kp.float().to(bf), table, pos), both, "float8_e4m3fn"),
            ((k.float(), k.float(), kp, kp, table, pos), both, "rows must be"),
            ((k, k.half(), kp, kp, table, pos), both, "dtype"),
            ((k, k, kp, kp, table, pos), dict(k_scale=sc, v_scale=sc.int()), "v_scale"),
            ((k, k, kp, kp, table, pos), dict(k_scale=sc[:, :, :1], v_scale=sc), "k_scale"),
            ((k, k, kp, kp, table, pos), dict(k_scale=torch.zeros(4, 3, 2, dtype=u8), v_scale=sc), "k_scale"),
            ((k, k, kp, kp, table, pos), dict(k_scale=sc, v_scale=torch.zeros(4, 4, 2, dtype=u8)), "v_scale")):
        with pytest.raises(ValueError, match=why):
            fq.kv_append(*args, **kw)
    for args, kw, why in (((heads, kp, kp, table, pos), both, "CUDA"),
                          ((heads, kp, kp, table, pos), {}, "needs k_scale"),
                          ((heads.float(), kp, kp, table, pos), both, "rows must be"),
                          ((heads, kp, kp, table, pos), dict(both, sinks=-1), "sinks"),
                          ((heads, kp, kp, table, pos), dict(both, sinks=2 ** 31), "sinks"),
                          ((heads[:, :3], kp, kp, table, pos), both, "multiple")):
        with pytest.raises(ValueError, match=why):
            fq.decode_attention(*args, **kw)
    for args, kw, why in (((kp, kp, table, pos), both, "CUDA"),
                          ((kp, kp, table, pos), {}, "needs k_scale"),
                          ((kp, kp, table, pos), dict(both, dtype=torch.float32), "rows must be"),
                          ((k[None], k[None], table, pos), dict(dtype=torch.float16), "own dtype"),
                          ((kp, kp, table, pos.long()), both, "int32"),
                          ((kp, kp, table[:2], pos), both, "sequences"),
                          ((kp, kp, table, pos), dict(both, seq=pos[:2]), "seq")):
        with pytest.raises(ValueError, match=why):
            fq.kv_read(*args, **kw)
    pool = fq.page_pool(5, device="cpu")
    assert pool.tolist() == [5, 0, 4, 3, 2, 1, 0] and pool.dtype == i32
    good = dict(new=pos, lengths=pos, page_table=table, room=pos, pool=pool, page_size=16)
    for kw, why in ((dict(), "CUDA"), (dict(new=pos.long()), "new"), (dict(lengths=pos[:2]), "lengths"),
                    (dict(room=pos[:, None]), "room"), (dict(page_table=table.long()), "page_table"), (dict(pool=pool[:1]), "pool"),
                    (dict(pool=pool.long()), "pool"), (dict(page_size=0), "page_size"), (dict(tokens=-1), "tokens"),
                    (dict(page_table=torch.zeros(2, 3, dtype=i32).t()), "contiguous")):
        with pytest.raises(ValueError, match=why):
            fq.page_plan(**dict(good, **kw))


def test_the_binding_leaves_what_is_not_ordinary():
    b = serve._bind()
    x = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).view(E4M3)
    i = torch.zeros(3, dtype=torch.int32)
    for args in ((), (x, x, i[None], i, None, None, None, None), (None,) * 8):
        assert b.read(*args) is NotImplemented
    for args in ((), (i, i, i[None], i, i, 16, None), (None,) * 7):
        assert b.plan(*args) is NotImplemented
    for args in ((None,) * 12, (i, x, x, i[None], i, None, 0, 0, None, None)):
        assert (b.append if len(args) == 12 else b.attention)(*args) is NotImplemented


# ------------------------------------------------------- their own definitions

def test_definition_of_codes():
    """The rounding agrees with torch's conversion; every code is a fixed point;
    the unit is the smallest that fits."""
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3).float().double()
    finite = codes[torch.isfinite(codes)]
    assert torch.equal(nearest_e4m3(finite), finite) and finite.abs().max() == 448
    x = torch.randn(100000, dtype=torch.float64, generator=torch.Generator().manual_seed(0))
    x = (x * torch.exp2(torch.randint(-12, 6, x.shape, generator=torch.Generator().manual_seed(1)))).clamp(-448, 448).float()
    assert torch.equal(nearest_e4m3(x.double()), x.to(E4M3).float().double())
    for top in (448.0, 448.001, 447.9, 1.0, 0.0, 1e-45, 3.4e38, 2.0 ** -130, 7.0, 3.5, 3.5000002):
        c = need_code(top)
        assert 0 <= c <= 254 and math.ldexp(448.0, c - 127) >= top
        assert c == 0 or math.ldexp(448.0, c - 128) < top


def test_definition_of_an_append():
    """A block's scale rises with a larger token and takes the others along; a
    call that writes the first place begins the block."""
    zero = torch.zeros(1, 4, 1, 16)
    c = Cache8(zero, zero, torch.full((1, 1, 1), 200, dtype=torch.uint8), torch.zeros(1, 1, 1, dtype=torch.uint8))
    table, seq = torch.tensor([[0]]), torch.tensor([0])
    one = torch.ones(1, 1, 16)
    c.append(one, one, table, torch.tensor([0]), seq, None, False)
    assert c.ks.item() == 127 - 8 and c.k[0, 0, 0, 0] == 256  # 1 = 256 * 2^-8
    c.append(one * 448, one, table, torch.tensor([1]), seq, None, False)
    assert c.ks.item() == 127 and torch.equal(c.values("k")[0, :2, 0, 0], torch.tensor([1.0, 448.0], dtype=torch.float64))
    c.append(one, one, table, torch.tensor([2]), seq, None, False)
    assert c.ks.item() == 127
    c.append(one * 2, one, table, torch.tensor([0]), seq, None, False)
    assert c.ks.item() == 128 - 8


def test_definition_of_a_plan():
    none = torch.zeros(2, dtype=torch.int32)
    p = Pages(none, torch.full((2, 3), -1), none, fq.page_pool(3, device="cpu"), 4)
    maps, refused = p.plan([5, 2], 8)
    assert not refused and maps == ([0] * 5 + [1] * 2 + [-1], [0, 1, 2, 3, 4, 0, 1, -1], [0, 1, 2, 3, 4, 8, 9, -1], [0, 5, 7])
    assert p.lengths == [5, 2] and p.room == [8, 4] and p.table == [[0, 1, -1], [2, -1, -1]] and p.free == []
    assert p.plan([0, 3], 3)[1] and p.lengths == [5, 2]
    p.plan([-1, -9])
    assert p.table == [[0, -1, -1], [-1, -1, -1]] and p.free == [2, 1] and p.room == [4, 0]
    assert seen_positions(6, 2, 3) == [0, 1, 2, 4, 5] and seen_positions(3, 0, 1) == [0, 1, 2]
