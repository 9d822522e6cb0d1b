// bind.cpp -- the serving calls' short way from Python into the library.
//
// A decoding step makes a handful of calls whose kernels run for a few
// microseconds; reading some forty tensor attributes and filling a parameter
// struct in Python takes longer than that.  Each function here does it for
// the ordinary call -- plain CUDA tensors of one device that fit each other,
// the current stream, a new output -- and returns NotImplemented for any
// other, or where anything looks wrong: serve.py then goes its general way,
// which handles strides, streams and outputs and names what it refuses.  A
// status the library returns is raised as FP4Error.
//
// A call issued back to back on a GB300's own CPU, the tensors read and the
// output made in Python / through Python's C interface / here (us): product
// 13.3 / 9.8 / 4.8, append of one token 14.6 / 10.2 / 4.2, attention
// of one short sequence 12.1 / 8.1 / 4.0.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "fp4.h"

namespace {

PyObject *error;  // FP4Error

// What the calls look at of a tensor.  Strides along dimensions of one are 0:
// they are never stepped along.
struct Tensor {
  const at::Tensor *t = nullptr;
  void *ptr;
  int dims;
  c10::ScalarType type;
  c10::DeviceIndex device;
  int64_t size[4], step[4];

  bool read(PyObject *o) {
    if (!THPVariable_CheckExact(o)) return false;
    t = &THPVariable_Unpack(o);
    if (!t->is_cuda() || t->layout() != c10::kStrided || t->dim() > 4) return false;
    dims = static_cast<int>(t->dim());
    type = t->scalar_type();
    device = t->get_device();
    ptr = t->data_ptr();
    const auto sizes = t->sizes(), steps = t->strides();
    for (int i = 0; i < dims; ++i) {
      size[i] = sizes[i];
      step[i] = size[i] == 1 ? 0 : steps[i];
    }
    return true;
  }
  template <class E>
  E *at() const { return static_cast<E *>(ptr); }
  // the last dimension can be read as consecutive elements
  bool rows_whole() const { return size[dims - 1] == 1 || step[dims - 1] == 1; }
  bool whole(c10::ScalarType of) const { return type == of && t->is_contiguous(); }
  int64_t elements() const { return t->numel(); }
  bool ints(int64_t n) const { return whole(c10::kInt) && dims == 1 && size[0] == n; }
};

// The library's code of a type, or -1.
int code_of(c10::ScalarType type) {
  return type == c10::kBFloat16 ? FP4_BF16 : type == c10::kHalf ? FP4_F16 : type == c10::kFloat ? FP4_F32 : -1;
}

bool is_half(c10::ScalarType type) { return type == c10::kBFloat16 || type == c10::kHalf; }

// A new tensor of these sizes beside `like`.
at::Tensor make(const Tensor &like, c10::ScalarType type, at::IntArrayRef sizes) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.t->device()));
}

// The current stream of the tensors' device, if that is the current one.
bool stream_of(c10::DeviceIndex device, void **stream) {
  if (c10::cuda::current_device() != device) return false;
  *stream = c10::cuda::getCurrentCUDAStream(device).stream();
  return true;
}

PyObject *general() {
  PyErr_Clear();
  Py_RETURN_NOTIMPLEMENTED;
}

// None or the tensor made, if the library took the call.
PyObject *finish(fp4_status code, const char *where, const at::Tensor &made) {
  if (code == FP4_OK) {
    if (!made.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(made);
  }
  PyObject *e = PyObject_CallFunction(error, "is", static_cast<int>(code), where);
  if (e) PyErr_SetObject(error, e);
  Py_XDECREF(e);
  return nullptr;
}

// matvec(x, q, sf, s_dec, row_shift or None, format, sf_layout, out_dtype or None)
PyObject *bind_matvec(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Tensor x, q, sf, sd, shift;
  if (n != 8 || !x.read(a[0]) || !q.read(a[1]) || !sf.read(a[2]) || !sd.read(a[3])) return general();
  const bool shifted = a[4] != Py_None;
  if (shifted && !shift.read(a[4])) return general();
  const long format = PyLong_AsLong(a[5]), layout = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return general();
  if (a[7] != Py_None && !THPDtype_Check(a[7])) return general();
  const c10::ScalarType type = a[7] == Py_None ? x.type : reinterpret_cast<THPDtype *>(a[7])->scalar_type;
  if (!is_half(x.type) || code_of(type) < 0 || (x.dims != 1 && x.dims != 2) || q.dims != 2) return general();
  const int64_t M = x.dims == 2 ? x.size[0] : 1, N = q.size[0], K = 2 * q.size[1];
  const int64_t scales = format == FP4_FMT_NVFP4_CTA ? (N + 127) / 128 : 1;
  const int64_t codes = fp4_sf_bytes(static_cast<int32_t>(format), N, K, static_cast<int32_t>(layout));
  if (x.size[x.dims - 1] != K || K == 0 || !x.rows_whole() || !q.whole(c10::kByte) || !sf.whole(c10::kByte) ||
      !sd.whole(c10::kFloat) || codes < 0 || sf.elements() < codes || sd.elements() < scales)
    return general();
  if (shifted && ((format != FP4_FMT_UE5M3_B16 && format != FP4_FMT_UE5M3_B32) || layout != FP4_SF_MMA ||
                  !shift.whole(c10::kChar) || shift.elements() < N || shift.device != x.device))
    return general();
  if (q.device != x.device || sf.device != x.device || sd.device != x.device) return general();
  void *stream;
  if (!stream_of(x.device, &stream)) return general();
  const int64_t sizes[2] = {M, N};
  const at::Tensor y = make(x, type, {sizes + 2 - x.dims, static_cast<size_t>(x.dims)});
  const fp4_operand w = {q.at<uint8_t>(), sf.at<uint8_t>(), sd.at<float>(), shifted ? shift.at<int8_t>() : nullptr,
                         static_cast<int32_t>(format), N, K};
  return finish(fp4_matvec(&w, static_cast<int32_t>(layout), x.ptr, M > 1 ? x.step[0] : K, code_of(x.type), M,
                           y.data_ptr(), N, code_of(type), stream),
                "fp4_matvec", y);
  END_HANDLE_TH_ERRORS
}

// The cache's fields from keys, values and the page table, if they fit.
bool read_cache(PyObject *const *a, fp4_kv_cache *c, Tensor *k) {
  Tensor v, table;
  if (!k->read(a[0]) || !v.read(a[1]) || !table.read(a[2])) return false;
  if (!is_half(k->type) || v.type != k->type || k->dims != 4 || v.dims != 4 ||
      std::memcmp(v.size, k->size, sizeof v.size) != 0 || table.type != c10::kInt || table.dims != 2 ||
      !k->rows_whole() || !v.rows_whole() || !table.rows_whole() || v.device != k->device || table.device != k->device)
    return false;
  for (int i = 1; i < 4; ++i)
    if (k->size[i] < 1 || k->size[i] > INT32_MAX) return false;
  if (table.size[0] > INT32_MAX || table.size[1] > INT32_MAX) return false;
  c->k = k->ptr;
  c->v = v.ptr;
  c->k_page = k->step[0], c->k_place = k->step[1], c->k_head = k->step[2];
  c->v_page = v.step[0], c->v_place = v.step[1], c->v_head = v.step[2];
  c->table = table.at<int32_t>();
  c->table_stride = table.step[0];
  c->pages = k->size[0];
  c->seqs = static_cast<int32_t>(table.size[0]);
  c->seq_pages = static_cast<int32_t>(table.size[1]);
  c->page_size = static_cast<int32_t>(k->size[1]);
  c->kv_heads = static_cast<int32_t>(k->size[2]);
  c->head_dim = static_cast<int32_t>(k->size[3]);
  c->type = code_of(k->type);
  return true;
}

// [tokens, heads, head_dim] of the cache's type and device.
bool rows_fit(const Tensor &t, const Tensor &cache, int64_t tokens, int64_t heads) {
  return t.type == cache.type && t.device == cache.device && t.dims == 3 && t.size[0] == tokens &&
         t.size[1] == heads && t.size[2] == cache.size[3] && t.rows_whole();
}

// Queries of that form whose heads share the cache's.
bool queries_fit(const Tensor &q, const Tensor &cache, int64_t tokens) {
  return q.dims == 3 && q.size[1] >= 1 && q.size[1] <= INT32_MAX && q.size[1] % cache.size[2] == 0 &&
         rows_fit(q, cache, tokens, q.size[1]);
}

// append(k, v, k_pages, v_pages, page_table, pos, seq, q, rope (each or None), interleaved)
PyObject *bind_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  fp4_append_params p{};
  Tensor cache, k, v, pos, seq, q, rope;
  if (n != 10 || !read_cache(a + 2, &p.cache, &cache) || !k.read(a[0]) || k.dims != 3 || !v.read(a[1]) ||
      !pos.read(a[5]))
    return general();
  const int64_t T = k.size[0];
  if (!rows_fit(k, cache, T, cache.size[2]) || !rows_fit(v, cache, T, cache.size[2]) || !pos.ints(T) ||
      pos.device != cache.device)
    return general();
  p.k = k.ptr, p.k_token = k.step[0], p.k_head = k.step[1];
  p.v = v.ptr, p.v_token = v.step[0], p.v_head = v.step[1];
  p.pos = pos.at<int32_t>();
  p.tokens = T;
  if (a[6] != Py_None) {
    if (!seq.read(a[6]) || !seq.ints(T) || seq.device != cache.device) return general();
    p.seq = seq.at<int32_t>();
  } else if (T > p.cache.seqs) {
    return general();
  }
  if (a[8] != Py_None) {
    if (!rope.read(a[8]) || !rope.whole(c10::kFloat) || rope.dims != 2 || rope.device != cache.device ||
        rope.size[1] > INT32_MAX)
      return general();
    p.rope = rope.at<float>();
    p.rope_len = rope.size[0];
    p.rot_dim = static_cast<int32_t>(rope.size[1]);
  }
  p.interleaved = PyObject_IsTrue(a[9]);
  if (p.interleaved < 0) return general();
  if (a[7] != Py_None && (!q.read(a[7]) || !queries_fit(q, cache, T))) return general();
  void *stream;
  if (!stream_of(cache.device, &stream)) return general();
  at::Tensor out;
  if (q.t) {
    out = make(q, q.type, {T, q.size[1], q.size[2]});
    p.q = q.ptr, p.q_token = q.step[0], p.q_head = q.step[1];
    p.q_out = out.data_ptr(), p.qo_token = q.size[1] * q.size[2], p.qo_head = q.size[2];
    p.heads = static_cast<int32_t>(q.size[1]);
  }
  return finish(fp4_kv_append(&p, stream), "fp4_kv_append", out);
  END_HANDLE_TH_ERRORS
}

// attention(q, k_pages, v_pages, page_table, lengths, scale or None, window)
PyObject *bind_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  fp4_attention_params p{};
  Tensor cache, q, lengths;
  if (n != 7 || !read_cache(a + 1, &p.cache, &cache) || !q.read(a[0]) || !queries_fit(q, cache, p.cache.seqs) ||
      !lengths.read(a[4]) || !lengths.ints(p.cache.seqs) || lengths.device != cache.device)
    return general();
  const long window = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return general();
  p.scale = static_cast<float>(a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(p.cache.head_dim))
                                               : PyFloat_AsDouble(a[5]));
  if (PyErr_Occurred() || !std::isfinite(p.scale) || window < 0 || window > INT32_MAX) return general();
  void *stream;
  if (!stream_of(cache.device, &stream)) return general();
  p.heads = static_cast<int32_t>(q.size[1]);
  p.window = static_cast<int32_t>(window);
  p.lengths = lengths.at<int32_t>();
  p.q = q.ptr, p.q_seq = q.step[0], p.q_head = q.step[1];
  const int64_t need = fp4_decode_attention_workspace(
      p.cache.seqs, static_cast<int64_t>(p.cache.seq_pages) * p.cache.page_size, p.heads, p.cache.kv_heads,
      p.cache.head_dim);
  const at::Tensor out = make(q, q.type, {q.size[0], q.size[1], q.size[2]});
  p.out = out.data_ptr(), p.out_seq = q.size[1] * q.size[2], p.out_head = q.size[2];
  at::Tensor work;  // freed in stream order: what runs on this stream has it until then
  if (need > 0) {
    work = make(q, c10::kByte, {need});
    p.workspace = work.data_ptr();
    p.workspace_bytes = need;
  }
  return finish(fp4_decode_attention(&p, stream), "fp4_decode_attention", out);
  END_HANDLE_TH_ERRORS
}

// setup(FP4Error)
PyObject *bind_setup(PyObject *, PyObject *type) {
  Py_INCREF(error = type);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction method(F *f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"setup", bind_setup, METH_O, "the exception that the calls raise"},
    {"matvec", method(bind_matvec), METH_FASTCALL, "ordinary matvec, or NotImplemented"},
    {"append", method(bind_append), METH_FASTCALL, "ordinary kv_append, or NotImplemented"},
    {"attention", method(bind_attention), METH_FASTCALL, "ordinary decode_attention, or NotImplemented"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
