/* bind.c -- the serving calls' short way from Python into the library.
 *
 * A decoding step makes a handful of calls whose kernels run for a few
 * microseconds; reading some forty tensor attributes and filling a parameter
 * struct in Python takes longer than that.  Each function here does it for
 * the ordinary call -- plain CUDA tensors of one device that fit each other,
 * the current stream, a new output -- and returns NotImplemented for any
 * other, or where anything looks wrong: serve.py then goes its general way,
 * which handles strides, streams and outputs and names what it refuses.  A
 * status the library returns is raised as FP4Error. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <string.h>

#include "fp4.h"

enum { kBf16 = FP4_BF16, kF16 = FP4_F16, kF32 = FP4_F32, kI32, kU8, kI8, kTypes };

static PyObject *tensor_type, *dtypes[kTypes], *empty, *raw_stream, *current_device, *error;
static PyObject *s_shape, *s_stride, *s_dtype, *s_data_ptr, *s_get_device, *s_device, *empty_names;

/* What the calls look at of a tensor.  Strides along dimensions of one are 0:
 * they are never stepped along. */
typedef struct {
  void *ptr;
  int dims, type;
  long device;
  int64_t size[4], step[4];
} Tensor;

static int read_tuple(PyObject *t, int64_t *to, int *n) {
  if (!t || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return 0;
  *n = (int)PyTuple_GET_SIZE(t);
  for (int i = 0; i < *n; ++i) {
    to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (to[i] == -1 && PyErr_Occurred()) return 0;
  }
  return 1;
}

static int read_tensor(PyObject *o, Tensor *t) {
  if ((PyObject *)Py_TYPE(o) != tensor_type) return 0;
  int ok = 0, steps = 0;
  PyObject *shape = PyObject_GetAttr(o, s_shape), *stride = PyObject_CallMethodNoArgs(o, s_stride);
  PyObject *dtype = PyObject_GetAttr(o, s_dtype), *ptr = PyObject_CallMethodNoArgs(o, s_data_ptr);
  PyObject *device = PyObject_CallMethodNoArgs(o, s_get_device);
  if (dtype && ptr && device && read_tuple(shape, t->size, &t->dims) && read_tuple(stride, t->step, &steps) &&
      steps == t->dims) {
    t->type = -1;
    for (int i = 0; i < kTypes; ++i)
      if (dtype == dtypes[i]) t->type = i;
    t->ptr = PyLong_AsVoidPtr(ptr);
    t->device = PyLong_AsLong(device);
    ok = t->type >= 0 && t->device >= 0 && !PyErr_Occurred();
    for (int i = 0; i < t->dims; ++i)
      if (t->size[i] == 1) t->step[i] = 0;
  }
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  Py_XDECREF(dtype);
  Py_XDECREF(ptr);
  Py_XDECREF(device);
  return ok;
}

static int contiguous(const Tensor *t) {
  int64_t n = 1;
  for (int i = t->dims - 1; i >= 0; --i) {
    if (t->size[i] != 1 && t->step[i] != n) return 0;
    n *= t->size[i];
  }
  return 1;
}

/* The last dimension can be read as consecutive elements. */
static int rows_whole(const Tensor *t) {
  return t->size[t->dims - 1] == 1 || t->step[t->dims - 1] == 1;
}

static int64_t elements(const Tensor *t) {
  int64_t n = 1;
  for (int i = 0; i < t->dims; ++i) n *= t->size[i];
  return n;
}

static int ints(const Tensor *t, int64_t n) {
  return t->type == kI32 && t->dims == 1 && t->size[0] == n && contiguous(t);
}

/* A new tensor of these sizes beside `like`. */
static PyObject *new_tensor(PyObject *like, int type, int dims, const int64_t *sizes) {
  PyObject *shape = PyTuple_New(dims), *device = PyObject_GetAttr(like, s_device), *made = NULL;
  if (shape && device) {
    int ok = 1;
    for (int i = 0; i < dims; ++i) {
      PyObject *n = PyLong_FromLongLong(sizes[i]);
      ok = ok && n;
      PyTuple_SET_ITEM(shape, i, n);
    }
    PyObject *args[3] = {shape, dtypes[type], device};
    if (ok) made = PyObject_Vectorcall(empty, args, 1, empty_names);
  }
  Py_XDECREF(shape);
  Py_XDECREF(device);
  return made;
}

/* The current stream of the tensors' device, if that is the current one. */
static int stream_of(long device, void **stream) {
  PyObject *now = PyObject_CallNoArgs(current_device);
  const long d = now ? PyLong_AsLong(now) : -1;
  PyObject *handle = NULL;
  if (now && d == device) handle = PyObject_CallOneArg(raw_stream, now);
  Py_XDECREF(now);
  if (!handle) return 0;
  *stream = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  return !PyErr_Occurred();
}

static PyObject *general(void) {
  PyErr_Clear();
  Py_RETURN_NOTIMPLEMENTED;
}

/* `made` (a reference that is passed on) if the library took the call. */
static PyObject *finish(fp4_status code, const char *where, PyObject *made) {
  if (code == FP4_OK) return made;
  Py_DECREF(made);
  PyObject *e = PyObject_CallFunction(error, "is", (int)code, where);
  if (e) PyErr_SetObject(error, e);
  Py_XDECREF(e);
  return NULL;
}

static void *address(PyObject *o) {
  PyObject *p = PyObject_CallMethodNoArgs(o, s_data_ptr);
  void *a = p ? PyLong_AsVoidPtr(p) : NULL;
  Py_XDECREF(p);
  return a;
}

/* matvec(x, q, sf, s_dec, row_shift or None, format, sf_layout, out_dtype or None) */
static PyObject *bind_matvec(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Tensor x, q, sf, sd, shift;
  if (n != 8 || !read_tensor(a[0], &x) || !read_tensor(a[1], &q) || !read_tensor(a[2], &sf) ||
      !read_tensor(a[3], &sd))
    return general();
  const int shifted = a[4] != Py_None;
  if (shifted && !read_tensor(a[4], &shift)) return general();
  const long format = PyLong_AsLong(a[5]), layout = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return general();
  int type = x.type;
  if (a[7] != Py_None)
    for (type = kBf16; type <= kF32 && a[7] != dtypes[type];) ++type;
  if ((x.type != kBf16 && x.type != kF16) || type > kF32 || (x.dims != 1 && x.dims != 2) || q.dims != 2)
    return general();
  const int64_t M = x.dims == 2 ? x.size[0] : 1, N = q.size[0], K = 2 * q.size[1];
  const int64_t scales = format == FP4_FMT_NVFP4_CTA ? (N + 127) / 128 : 1;
  if (x.size[x.dims - 1] != K || K == 0 || !rows_whole(&x) || !contiguous(&q) || !contiguous(&sf) ||
      !contiguous(&sd) || q.type != kU8 || sf.type != kU8 || sd.type != kF32 ||
      elements(&sf) < fp4_sf_bytes((int32_t)format, N, K, (int32_t)layout) || elements(&sd) < scales ||
      fp4_sf_bytes((int32_t)format, N, K, (int32_t)layout) < 0)
    return general();
  if (shifted && ((format != FP4_FMT_UE5M3_B16 && format != FP4_FMT_UE5M3_B32) || layout != FP4_SF_MMA ||
                  shift.type != kI8 || elements(&shift) < N || !contiguous(&shift) || shift.device != x.device))
    return general();
  if (q.device != x.device || sf.device != x.device || sd.device != x.device) return general();
  void *stream;
  if (!stream_of(x.device, &stream)) return general();
  const int64_t sizes[2] = {M, N};
  PyObject *y = new_tensor(a[0], type, x.dims, x.dims == 2 ? sizes : sizes + 1);
  if (!y) return NULL;
  const fp4_operand w = {q.ptr, sf.ptr, sd.ptr, shifted ? shift.ptr : NULL, (int32_t)format, N, K};
  return finish(fp4_matvec(&w, (int32_t)layout, x.ptr, M > 1 ? x.step[0] : K, x.type, M, address(y), N, type, stream),
                "fp4_matvec", y);
}

/* The cache's fields from keys, values and the page table; 0 if they do not fit. */
static int read_cache(PyObject *const *a, fp4_kv_cache *c, Tensor *k, long *device) {
  Tensor v, table;
  if (!read_tensor(a[0], k) || !read_tensor(a[1], &v) || !read_tensor(a[2], &table)) return 0;
  if ((k->type != kBf16 && k->type != kF16) || v.type != k->type || k->dims != 4 || v.dims != 4 ||
      memcmp(v.size, k->size, sizeof v.size) || table.type != kI32 || table.dims != 2 || !rows_whole(k) ||
      !rows_whole(&v) || !rows_whole(&table) || v.device != k->device || table.device != k->device)
    return 0;
  for (int i = 1; i < 4; ++i)
    if (k->size[i] < 1 || k->size[i] > INT32_MAX) return 0;
  if (table.size[0] > INT32_MAX || table.size[1] > INT32_MAX) return 0;
  const fp4_kv_cache made = {k->ptr, v.ptr, k->step[0], k->step[1], k->step[2], v.step[0], v.step[1], v.step[2],
                             table.ptr, table.step[0], k->size[0], (int32_t)table.size[0], (int32_t)table.size[1],
                             (int32_t)k->size[1], (int32_t)k->size[2], (int32_t)k->size[3], k->type};
  *c = made;
  *device = k->device;
  return 1;
}

/* [tokens, heads, head_dim] tensor of the cache's type and device (any heads if < 0). */
static int rows_fit(const Tensor *t, const Tensor *cache, int64_t tokens, int64_t heads) {
  return t->type == cache->type && t->device == cache->device && t->dims == 3 && t->size[0] == tokens &&
         (heads < 0 || t->size[1] == heads) && t->size[2] == cache->size[3] && rows_whole(t);
}

/* append(k, v, k_pages, v_pages, page_table, pos, seq, q, rope (each or None), interleaved) */
static PyObject *bind_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  fp4_append_params p;
  memset(&p, 0, sizeof p);
  Tensor cache, k, v, pos, seq, q, rope;
  long device;
  if (n != 10 || !read_cache(a + 2, &p.cache, &cache, &device) || !read_tensor(a[0], &k) || k.dims != 3 ||
      !read_tensor(a[1], &v))
    return general();
  const int64_t T = k.size[0];
  if (!rows_fit(&k, &cache, T, p.cache.kv_heads) || !rows_fit(&v, &cache, T, p.cache.kv_heads) ||
      !read_tensor(a[5], &pos) || !ints(&pos, T) || pos.device != device)
    return general();
  p.k = k.ptr, p.k_token = k.step[0], p.k_head = k.step[1];
  p.v = v.ptr, p.v_token = v.step[0], p.v_head = v.step[1];
  p.pos = pos.ptr;
  p.tokens = T;
  if (a[6] != Py_None) {
    if (!read_tensor(a[6], &seq) || !ints(&seq, T) || seq.device != device) return general();
    p.seq = seq.ptr;
  } else if (T > p.cache.seqs) {
    return general();
  }
  if (a[8] != Py_None) {
    if (!read_tensor(a[8], &rope) || rope.type != kF32 || rope.dims != 2 || !contiguous(&rope) ||
        rope.device != device || rope.size[1] > INT32_MAX)
      return general();
    p.rope = rope.ptr, p.rope_len = rope.size[0], p.rot_dim = (int32_t)rope.size[1];
  }
  p.interleaved = PyObject_IsTrue(a[9]);
  if (p.interleaved < 0) return general();
  void *stream;
  PyObject *out = NULL;
  if (a[7] == Py_None) {
    if (!stream_of(device, &stream)) return general();
    Py_INCREF(Py_None);
    out = Py_None;
  } else {
    if (!read_tensor(a[7], &q) || !rows_fit(&q, &cache, T, -1) || q.size[1] < 1 || q.size[1] > INT32_MAX ||
        q.size[1] % p.cache.kv_heads || !stream_of(device, &stream))
      return general();
    if (!(out = new_tensor(a[7], q.type, 3, q.size))) return NULL;
    p.q = q.ptr, p.q_token = q.step[0], p.q_head = q.step[1];
    p.q_out = address(out), p.qo_token = q.size[1] * q.size[2], p.qo_head = q.size[2];
    p.heads = (int32_t)q.size[1];
  }
  return finish(fp4_kv_append(&p, stream), "fp4_kv_append", out);
}

/* attention(q, k_pages, v_pages, page_table, lengths, scale or None, window) */
static PyObject *bind_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  fp4_attention_params p;
  memset(&p, 0, sizeof p);
  Tensor cache, q, lengths;
  long device;
  if (n != 7 || !read_cache(a + 1, &p.cache, &cache, &device) || !read_tensor(a[0], &q) ||
      !rows_fit(&q, &cache, p.cache.seqs, -1) || q.size[1] < 1 || q.size[1] > INT32_MAX || q.size[1] % p.cache.kv_heads || !read_tensor(a[4], &lengths) ||
      !ints(&lengths, p.cache.seqs) || lengths.device != device)
    return general();
  const long window = PyLong_AsLong(a[6]);
  p.scale = a[5] == Py_None ? (float)(1.0 / sqrt((double)p.cache.head_dim)) : (float)PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred() || !isfinite(p.scale) || window < 0 || window > INT32_MAX) return general();
  void *stream;
  if (!stream_of(device, &stream)) return general();
  p.heads = (int32_t)q.size[1];
  p.window = (int32_t)window;
  p.lengths = lengths.ptr;
  p.q = q.ptr, p.q_seq = q.step[0], p.q_head = q.step[1];
  const int64_t need = fp4_decode_attention_workspace(p.cache.seqs, (int64_t)p.cache.seq_pages * p.cache.page_size,
                                                      p.heads, p.cache.kv_heads, p.cache.head_dim);
  PyObject *out = new_tensor(a[0], q.type, 3, q.size), *work = NULL;
  if (!out) return NULL;
  p.out = address(out), p.out_seq = q.size[1] * q.size[2], p.out_head = q.size[2];
  if (need > 0) {
    if (!(work = new_tensor(a[0], kU8, 1, &need))) {
      Py_DECREF(out);
      return NULL;
    }
    p.workspace = address(work);
    p.workspace_bytes = need;
  }
  const fp4_status code = fp4_decode_attention(&p, stream);
  Py_XDECREF(work); /* freed in stream order: what runs on this stream has it until then */
  return finish(code, "fp4_decode_attention", out);
}

/* setup(torch.Tensor, (the dtypes in the order of the enum), torch.empty,
 * current raw stream of a device, current device, FP4Error) */
static PyObject *bind_setup(PyObject *self, PyObject *args) {
  (void)self;
  PyObject *types;
  if (!PyArg_ParseTuple(args, "OO!OOOO", &tensor_type, &PyTuple_Type, &types, &empty, &raw_stream, &current_device,
                        &error))
    return NULL;
  if (PyTuple_GET_SIZE(types) != kTypes) {
    PyErr_SetString(PyExc_ValueError, "setup: the dtypes");
    return NULL;
  }
  for (int i = 0; i < kTypes; ++i) Py_INCREF(dtypes[i] = PyTuple_GET_ITEM(types, i));
  Py_INCREF(tensor_type);
  Py_INCREF(empty);
  Py_INCREF(raw_stream);
  Py_INCREF(current_device);
  Py_INCREF(error);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", bind_setup, METH_VARARGS, "the objects of torch that the calls use"},
    {"matvec", (PyCFunction)(void (*)(void))bind_matvec, METH_FASTCALL, "ordinary matvec, or NotImplemented"},
    {"append", (PyCFunction)(void (*)(void))bind_append, METH_FASTCALL, "ordinary kv_append, or NotImplemented"},
    {"attention", (PyCFunction)(void (*)(void))bind_attention, METH_FASTCALL,
     "ordinary decode_attention, or NotImplemented"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__bind(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_device = PyUnicode_InternFromString("device");
  empty_names = Py_BuildValue("(OO)", s_dtype, s_device);
  if (!s_shape || !s_stride || !s_dtype || !s_data_ptr || !s_get_device || !s_device || !empty_names) return NULL;
  return PyModule_Create(&module);
}
