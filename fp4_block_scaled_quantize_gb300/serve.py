"""Serving operators: products of 4-bit weights with a few tokens, a paged
cache of keys and values, and attention of one new token per sequence over it.

``fp4_*`` functions keep the C names and return a status code; ``matvec``,
``kv_append`` and ``decode_attention`` check their tensors, allocate outputs
and raise.  All of them only marshal arguments: the work is done by the
library's CUDA kernels.  An output or workspace that a function allocates for
a given ``stream`` belongs to that stream.

Host time counts here (a call's kernels run for a few microseconds).  The
ordinary call -- plain tensors that fit each other, the current stream, a new
output -- goes through the compiled ``_lib/_bind.so``, which reads the tensors
and fills the parameter struct; every other goes through this module, which
packs the same structs by ``struct`` in the layout of the ctypes classes.
"""
import ctypes
import importlib.machinery
import importlib.util
import os
import struct
from functools import lru_cache

import torch

from . import (FP4_FMT_NVFP4_CTA, FP4_FMT_UE5M3_B16, FP4_FMT_UE5M3_B32, FP4_SF_MMA, LIB_PATH,
               FP4Error, _stream, fp4_sf_bytes, lib, n_stripes)

FP4_BF16, FP4_F16, FP4_F32 = 0, 1, 2
_TYPES = {torch.bfloat16: FP4_BF16, torch.float16: FP4_F16, torch.float32: FP4_F32}
_HALVES = (torch.bfloat16, torch.float16)
_INT, _FLOAT = torch.int32, torch.float32


class fp4_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page", ctypes.c_int64),
                ("k_place", ctypes.c_int64), ("k_head", ctypes.c_int64), ("v_page", ctypes.c_int64),
                ("v_place", ctypes.c_int64), ("v_head", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("seqs", ctypes.c_int32), ("seq_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32)]


class fp4_append_params(ctypes.Structure):
    _fields_ = [("cache", fp4_kv_cache), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("qo_token", ctypes.c_int64), ("qo_head", ctypes.c_int64), ("pos", ctypes.c_void_p),
                ("seq", ctypes.c_void_p), ("rope", ctypes.c_void_p), ("rope_len", ctypes.c_int64),
                ("tokens", ctypes.c_int64), ("heads", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class fp4_attention_params(ctypes.Structure):
    _fields_ = [("cache", fp4_kv_cache), ("lengths", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("q_seq", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("out_seq", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


_CACHE = "PPqqqqqqPqqiiiiii"
_OPERAND = struct.Struct("@PPPPi4xqq")
_APPEND = struct.Struct("@" + _CACHE + "PPPPqqqqqqqqPPPqqiii4x")
_ATTENTION = struct.Struct("@" + _CACHE + "PPPPqqqqPqiif4x")

_entry = None


def _lib():
    """The library with the argument types of this module's entry points."""
    global _entry
    if _entry is None:
        L = lib()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.fp4_matvec.argtypes = [vp, i32, vp, i64, i32, i64, vp, i64, i32, vp]
        L.fp4_kv_append.argtypes = [vp, vp]
        L.fp4_decode_attention.argtypes = [vp, vp]
        L.fp4_decode_attention_workspace.argtypes = [i32, i64, i32, i32, i32]
        for f in ("fp4_matvec", "fp4_kv_append", "fp4_decode_attention"):
            getattr(L, f).restype = i32
        L.fp4_decode_attention_workspace.restype = i64
        _entry = L
    return _entry


@lru_cache(maxsize=1)
def _bind():
    """The compiled binding (raises OSError if it has not been built)."""
    path = os.path.join(os.path.dirname(LIB_PATH), "_bind.so")
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with "
                      "`python -c 'import __graft_entry__ as g; g.build()'`")
    spec = importlib.util.spec_from_file_location(
        "_bind", path, loader=importlib.machinery.ExtensionFileLoader("_bind", path))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.setup(FP4Error)
    return m


# ------------------------------------------------------------- raw entry points

def fp4_matvec(W, sf_layout, x, x_stride, x_type, M, y, y_stride, y_type, stream=None):
    return _lib().fp4_matvec(ctypes.byref(W), sf_layout, x.data_ptr(), x_stride, x_type, M,
                             y.data_ptr(), y_stride, y_type, _stream(stream))


def fp4_kv_append(p, stream=None):
    """p: an fp4_append_params, or the same bytes packed."""
    return _lib().fp4_kv_append(p if isinstance(p, bytes) else ctypes.byref(p), _stream(stream))


def fp4_decode_attention(p, stream=None):
    """p: an fp4_attention_params, or the same bytes packed."""
    return _lib().fp4_decode_attention(p if isinstance(p, bytes) else ctypes.byref(p),
                                       _stream(stream))


def fp4_decode_attention_workspace(seqs, room, heads, kv_heads, head_dim):
    return _lib().fp4_decode_attention_workspace(seqs, room, heads, kv_heads, head_dim)


# ------------------------------------------------------ allocating conveniences

def _new(sizes, dtype, device, stream):
    """A tensor for work on `stream`, which its memory then belongs to."""
    if stream is None:
        return torch.empty(sizes, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(sizes, dtype=dtype, device=device)


def _device(where, first, *rest):
    """Index of the one CUDA device of the tensors; it has to be the current
    one, because that is where kernels are launched."""
    dev = first.get_device()
    for t in rest:
        if t.get_device() != dev:
            raise ValueError(f"{where}: tensors must share one device")
    if dev < 0:
        raise ValueError(f"{where}: tensors must be on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{where}: the tensors' device is not the current one")
    return dev


def _handle(stream, dev):
    """The stream's handle (of the device's current stream by default; asked
    for directly, as a Stream object takes longer than the launch)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


@lru_cache(maxsize=1024)
def _room(format, rows, cols, layout):
    """(bytes of the scales, decode scales) of a copy of these sizes."""
    return (fp4_sf_bytes(format, rows, cols, layout),
            n_stripes(rows) if format == FP4_FMT_NVFP4_CTA else 1)


def matvec(x, w, out_dtype=None, out=None, stream=None):
    """y = x W^T for a few tokens: x [M, K] or [K] in bfloat16 or float16
    (rows may be strided), w a Quantized copy [N, K] in either scale layout.
    y is [M, N] (or [N]) in out_dtype -- x's dtype by default, or bfloat16,
    float16 or float32 -- or written to `out` (rows may be strided).  The
    activations are not quantised; see fp4_matvec in include/fp4.h."""
    if out is None and stream is None:
        y = _bind().matvec(x, w.q, w.sf, w.s_dec, w.row_shift, w.format, w.sf_layout, out_dtype)
        if y is not NotImplemented:
            return y
    q, sf, s_dec, shift, format, layout = w.q, w.sf, w.s_dec, w.row_shift, w.format, w.sf_layout
    dtype, sizes = x.dtype, x.shape
    if dtype not in _HALVES:
        raise ValueError("matvec: x must be bfloat16 or float16")
    if len(sizes) == 2:
        M = sizes[0]
    elif len(sizes) == 1:
        M = 1
    else:
        raise ValueError("matvec: x must be [K] or [M, K]")
    N, K = q.shape
    K *= 2
    if sizes[-1] != K:
        raise ValueError(f"matvec: x has {sizes[-1]} columns, the weight {K}")
    steps = x.stride()
    if K > 1 and steps[-1] != 1:
        raise ValueError("matvec: the last dimension of x must be contiguous")
    if not (q.is_contiguous() and sf.is_contiguous() and s_dec.is_contiguous()):
        raise ValueError("matvec: the weight copy is not contiguous")
    codes, scales = _room(format, N, K, layout)
    if sf.numel() < codes or s_dec.numel() < scales or s_dec.dtype != torch.float32 or \
            q.dtype != torch.uint8 or sf.dtype != torch.uint8:
        raise ValueError("matvec: the weight copy's scales do not fit its format and layout")
    if shift is not None and (format not in (FP4_FMT_UE5M3_B16, FP4_FMT_UE5M3_B32)
                              or layout != FP4_SF_MMA or shift.numel() < N
                              or shift.dtype != torch.int8 or not shift.is_contiguous()):
        raise ValueError("matvec: row shifts belong to UE5M3 copies in the tensor-core layout")
    dev = _device("matvec", x, q, sf, s_dec)
    if shift is not None:
        _device("matvec", x, shift)
    shape = (M, N) if len(sizes) == 2 else (N,)
    if out is None:
        if out_dtype is None:
            out_dtype = dtype
        elif out_dtype not in _TYPES:
            raise ValueError("matvec: out_dtype must be bfloat16, float16 or float32")
        out = _new(shape, out_dtype, x.device, stream)
        y_step = N
    else:
        if out.dtype not in _TYPES or out.shape != shape or (N > 1 and out.stride(-1) != 1) or \
                (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"matvec: out must be a {list(shape)} tensor with contiguous rows, in "
                             "bfloat16, float16 or float32")
        _device("matvec", x, out)
        out_dtype = out.dtype
        y_step = out.stride(0) if M > 1 else N
    op = _OPERAND.pack(q.data_ptr(), sf.data_ptr(), s_dec.data_ptr(),
                       0 if shift is None else shift.data_ptr(), format, N, K)
    code = _lib().fp4_matvec(op, layout, x.data_ptr(), steps[0] if M > 1 else K, _TYPES[dtype], M,
                             out.data_ptr(), y_step, _TYPES[out_dtype], _handle(stream, dev))
    if code:
        raise FP4Error(code, "fp4_matvec")
    return out


def _steps(where, name, t, sizes):
    """Strides of a tensor of these sizes whose last dimension is contiguous
    (0 along a dimension of one: it is never stepped along)."""
    if t.shape != sizes:
        raise ValueError(f"{where}: {name} must be {list(sizes)}, not {list(t.shape)}")
    steps = t.stride()
    if steps[-1] != 1 and sizes[-1] > 1:
        raise ValueError(f"{where}: the last dimension of {name} must be contiguous")
    return [0 if n == 1 else s for n, s in zip(sizes, steps)]


def _rows(where, name, t, sizes):
    """(token, head) strides of a [tokens, heads, head_dim] tensor."""
    if t.shape == sizes:
        a, b, c = t.stride()
        if c == 1 and not (a | b) & 7:
            return a, b
    return _steps(where, name, t, sizes)[:2]


def _cache_fields(where, k_pages, v_pages, page_table):
    """The fields of fp4_kv_cache, in order."""
    dtype, sizes, table = k_pages.dtype, k_pages.shape, page_table.shape
    if dtype not in _HALVES or v_pages.dtype is not dtype:
        raise ValueError(f"{where}: keys and values must both be bfloat16 or both float16")
    if len(sizes) != 4 or len(table) != 2:
        raise ValueError(f"{where}: k_pages must be [pages, page_size, kv_heads, head_dim], "
                         "page_table [seqs, pages of a sequence]")
    if page_table.dtype is not _INT:
        raise ValueError(f"{where}: page_table must be int32")
    pages, page, heads, dim = sizes
    if not (page and heads and dim):
        raise ValueError(f"{where}: pages without places, heads or elements")
    seqs, wide = table
    step, one = page_table.stride()
    if one != 1 and wide > 1:
        raise ValueError(f"{where}: the rows of page_table must be contiguous")
    ka, kb, kc, kd = k_pages.stride()
    va, vb, vc, vd = v_pages.stride()
    if kd != 1 or vd != 1 or v_pages.shape != sizes or (ka | kb | kc | va | vb | vc) & 7:
        ka, kb, kc, kd = _steps(where, "k_pages", k_pages, sizes)
        va, vb, vc, vd = _steps(where, "v_pages", v_pages, sizes)
    return (k_pages.data_ptr(), v_pages.data_ptr(), ka, kb, kc, va, vb, vc, page_table.data_ptr(),
            step if seqs > 1 else 0, pages, seqs, wide, page, heads, dim, _TYPES[dtype])


def _need_ints(where, name, t, n):
    if t.dtype is not _INT or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous int32 tensor of {n}")


def kv_append(k, v, k_pages, v_pages, page_table, pos, seq=None, q=None, rope=None,
              interleaved=False, q_out=None, stream=None):
    """Writes the keys k and values v [tokens, kv_heads, head_dim] of new
    tokens into a paged cache (k_pages, v_pages [pages, page_size, kv_heads,
    head_dim], any strides; page_table [seqs, pages of a sequence] int32) at
    positions pos [tokens] int32 of sequences seq [tokens] int32 (default:
    token t is the new token of sequence t).  With rope [positions, rot_dim]
    float32 (rope_table) keys and queries q [tokens, heads, head_dim] are
    rotated on the way.  Returns the rotated queries (q_out, new by default),
    or None without q.  Tokens at negative positions are skipped; no two tokens
    of a call may have the same place (it would hold parts of both)."""
    if stream is None and q_out is None:
        r = _bind().append(k, v, k_pages, v_pages, page_table, pos, seq, q, rope, interleaved)
        if r is not NotImplemented:
            return r
    where = "kv_append"
    cache = _cache_fields(where, k_pages, v_pages, page_table)
    dtype, Hk, D = k_pages.dtype, cache[14], cache[15]
    if k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError(f"{where}: q, k, v and the cache must share one dtype")
    T = k.shape[0]
    sizes = (T, Hk, D)
    ks, kh = _rows(where, "k", k, sizes)
    vs, vh = _rows(where, "v", v, sizes)
    _need_ints(where, "pos", pos, T)
    extra = []
    seq_at = rope_at = q_at = out_at = rot_dim = rope_len = heads = qs = qh = os_ = oh = 0
    if seq is not None:
        _need_ints(where, "seq", seq, T)
        extra.append(seq)
        seq_at = seq.data_ptr()
    elif T > cache[11]:
        raise ValueError(f"{where}: more tokens than sequences; give seq")
    if rope is not None:
        if rope.dtype is not _FLOAT or rope.dim() != 2 or not rope.is_contiguous():
            raise ValueError(f"{where}: rope must be a contiguous [positions, rot_dim] float32 tensor")
        extra.append(rope)
        rope_len, rot_dim = rope.shape
        rope_at = rope.data_ptr()
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else 0
        if q.dtype is not dtype:
            raise ValueError(f"{where}: q, k, v and the cache must share one dtype")
        if heads < 1 or heads % Hk:
            raise ValueError(f"{where}: q must be [tokens, heads, head_dim], heads a multiple of {Hk}")
        sizes = (T, heads, D)
        qs, qh = _rows(where, "q", q, sizes)
        if q_out is None:
            q_out = _new(sizes, dtype, q.device, stream)
            os_, oh = heads * D, D
        else:
            if q_out.dtype is not dtype:
                raise ValueError(f"{where}: q_out must have q's dtype")
            os_, oh = _rows(where, "q_out", q_out, sizes)
        extra += q, q_out
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError(f"{where}: q_out without q")
    dev = _device(where, k, v, k_pages, v_pages, page_table, pos, *extra)
    code = _lib().fp4_kv_append(
        _APPEND.pack(*cache, k.data_ptr(), v.data_ptr(), q_at, out_at, ks, kh, vs, vh, qs, qh, os_,
                     oh, pos.data_ptr(), seq_at, rope_at, rope_len, T, heads, rot_dim,
                     1 if interleaved else 0), _handle(stream, dev))
    if code:
        raise FP4Error(code, "fp4_kv_append")
    return q_out


def decode_attention(q, k_pages, v_pages, page_table, lengths, scale=None, window=0, out=None,
                     return_lse=False, stream=None):
    """Attention of one new token per sequence, q [seqs, heads, head_dim],
    over a paged cache (as in kv_append) that holds lengths [seqs] int32
    positions of each sequence, the new one among them.  scale defaults to
    head_dim ** -0.5; window > 0 sees the newest `window` positions only.
    Returns [seqs, heads, head_dim] in q's dtype (or `out`), and with
    return_lse also the logarithm of each row's sum of exponentials, float32
    [seqs, heads].  A sequence of length 0 gives zeros (and -inf)."""
    if out is None and stream is None and not return_lse:
        r = _bind().attention(q, k_pages, v_pages, page_table, lengths, scale, window)
        if r is not NotImplemented:
            return r
    where = "decode_attention"
    cache = _cache_fields(where, k_pages, v_pages, page_table)
    dtype, seqs, Hk, D = k_pages.dtype, cache[11], cache[14], cache[15]
    heads = q.shape[1] if q.dim() == 3 else 0
    if q.dtype is not dtype or heads < 1 or heads % Hk:
        raise ValueError(f"{where}: q must be [seqs, heads, head_dim] in the cache's dtype, heads a "
                         f"multiple of {Hk}")
    sizes = (seqs, heads, D)
    qs, qh = _rows(where, "q", q, sizes)
    _need_ints(where, "lengths", lengths, seqs)
    if window < 0 or window > 0x7FFFFFFF:
        raise ValueError(f"{where}: window must be >= 0")
    dev = _device(where, q, k_pages, v_pages, page_table, lengths)
    device = q.device
    if out is None:
        out = _new(sizes, dtype, device, stream)
        os_, oh = heads * D, D
    else:
        if out.dtype is not dtype:
            raise ValueError(f"{where}: out must have q's dtype")
        os_, oh = _rows(where, "out", out, sizes)
        _device(where, q, out)
    lse = _new((seqs, heads), _FLOAT, device, stream) if return_lse else None
    need = _workspace(seqs, cache[12] * cache[13], heads, Hk, D, dev)
    work = _new(need, torch.uint8, device, stream) if need > 0 else None
    code = _lib().fp4_decode_attention(
        _ATTENTION.pack(*cache, lengths.data_ptr(), q.data_ptr(), out.data_ptr(),
                        lse.data_ptr() if return_lse else 0, qs, qh, os_, oh,
                        work.data_ptr() if need > 0 else 0, need if need > 0 else 0, heads, window,
                        D ** -0.5 if scale is None else scale), _handle(stream, dev))
    if code:
        raise FP4Error(code, "fp4_decode_attention")
    return (out, lse) if return_lse else out


@lru_cache(maxsize=1024)
def _workspace(seqs, room, heads, kv_heads, head_dim, dev):
    """fp4_decode_attention_workspace for these sizes on device `dev` (the
    current one)."""
    return fp4_decode_attention_workspace(seqs, room, heads, kv_heads, head_dim)


def rope_table(positions, rot_dim, base=10000.0, device="cuda"):
    """cos and sin of the rotation of each position, float32 [positions,
    rot_dim]: cos(p base^(-2 i / rot_dim)) in column i, the sine rot_dim / 2
    columns on (angles and functions in 64 bits, rounded once)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rope_table: rot_dim must be even")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2.0 * i / rot_dim)
    return torch.cat([torch.cos(angle), torch.sin(angle)], -1).float().to(device)


__all__ = ["FP4_BF16", "FP4_F16", "FP4_F32", "fp4_append_params", "fp4_attention_params",
           "fp4_decode_attention", "fp4_decode_attention_workspace", "fp4_kv_append",
           "fp4_kv_cache", "fp4_matvec", "decode_attention", "kv_append", "matvec", "rope_table"]
