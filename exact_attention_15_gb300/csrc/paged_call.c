/*
 * The paged cache's torch calls from C: a decoding step's kernels take less time
 * than the interpreter needs for checking their arguments, so the common calls are
 * checked and made here, through the tensors' own Python attributes (no torch
 * header, nothing that depends on its version). Every function returns
 * NotImplemented for what it does not take at once (given outputs, another current
 * device, anything wrong); paged.py then goes through its own checks, which say
 * what is wrong. A non-zero status of the C ABI comes back as an int.
 *
 * What a call costs the host, from Python and from here, on three Grace hosts (they
 * differ): append 11.9 to 16.7 and 8.1 to 10.9 us, one-token attention of a short
 * context 13.9 to 18.5 and 8.5 to 12.3, a chunk call of one token 20 and 12.5.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>

#include "../../include/attn.h"

typedef int (*append_fn)(const attn_paged_cache*, const void*, const void*, const void*, void*, long long,
                         long long, long long, long long, int, int, int, const int*, const int*, const int*,
                         int, long long, const double*, int, int, attn_stream_t);
typedef int (*decode_fn)(const attn_paged_cache*, const void*, void*, float*, int, int, const int*,
                         const int*, int, long long, float, void*, size_t, attn_stream_t);
typedef int (*fwd_fn)(const attn_paged_cache*, const void*, void*, float*, int, int, int, const int*,
                      const int*, const int*, int, long long, int, float, void*, size_t, attn_stream_t);
typedef size_t (*bytes_fn)(const attn_paged_cache*, int, int, int, int, int);

static append_fn c_append;
static decode_fn c_decode;
static fwd_fn c_fwd;
static bytes_fn c_bytes;
/* from torch */
static PyObject *t_bf16, *t_f32, *t_f64, *t_i32, *t_u8, *f_empty, *f_empty_like, *f_device, *f_stream, *o_contiguous;
/* names */
static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_stride, *n_data_ptr;
static PyObject *kw_dtype_device, *kw_memory_format;

/* What a call knows of a tensor. */
typedef struct {
  long long size[3], stride[3];
  int dims, contiguous;
  void* ptr;
} view;

static int integers(PyObject* tuple, long long* out, int most) {
  if (!tuple || !PyTuple_Check(tuple)) return -1;
  const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
  if (n > most) return -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

/* 1 when t is a tensor of that dtype on device `index` with at most 3 dimensions. */
static int look(PyObject* t, PyObject* dtype, long index, view* v) {
  PyObject* x = PyObject_GetAttr(t, n_dtype);
  if (!x) return 0;
  Py_DECREF(x); /* dtypes are singletons that live on */
  if (x != dtype) return 0;
  x = PyObject_CallMethodNoArgs(t, n_get_device);
  if (!x) return 0;
  const long dev = PyLong_AsLong(x);
  Py_DECREF(x);
  if (dev != index) return 0;
  x = PyObject_GetAttr(t, n_shape);
  v->dims = integers(x, v->size, 3);
  Py_XDECREF(x);
  if (v->dims < 0) return 0;
  x = PyObject_CallMethodNoArgs(t, n_is_contiguous);
  if (!x) return 0;
  v->contiguous = x == Py_True;
  Py_DECREF(x);
  if (!v->contiguous) {
    x = PyObject_CallMethodNoArgs(t, n_stride);
    const int n = integers(x, v->stride, 3);
    Py_XDECREF(x);
    if (n != v->dims) return 0;
  }
  x = PyObject_CallMethodNoArgs(t, n_data_ptr);
  if (!x) return 0;
  v->ptr = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return !PyErr_Occurred();
}

/* [tokens, heads, d] whose tokens are contiguous but may lie apart. */
static int tokens_of(PyObject* t, long index, long long d, view* v, long long* apart) {
  if (!look(t, t_bf16, index, v) || v->dims != 3 || v->size[2] != d || v->size[0] > INT_MAX || v->size[1] > INT_MAX)
    return 0;
  if (v->contiguous) {
    *apart = v->size[1] * d;
    return 1;
  }
  if (v->stride[2] != 1 || (v->size[1] > 1 && v->stride[1] != d)) return 0;
  *apart = v->size[0] > 1 ? v->stride[0] : v->size[1] * d;
  return 1;
}

typedef struct {
  const int *lens, *table, *cu;
  int B, cols;
  long long stride;
} seqs;

static int seqs_of(PyObject* table, PyObject* lens, PyObject* cu, long index, long long tokens, seqs* s) {
  view v;
  if (!look(lens, t_i32, index, &v) || v.dims != 1 || !v.contiguous || v.size[0] >= INT_MAX) return 0;
  s->B = (int)v.size[0];
  s->lens = (const int*)v.ptr;
  if (!look(table, t_i32, index, &v) || v.dims != 2 || v.size[0] != s->B || v.size[1] > INT_MAX) return 0;
  s->cols = (int)v.size[1];
  s->stride = v.size[1];
  if (!v.contiguous) {
    if (s->cols > 1 && v.stride[1] != 1) return 0;
    if (s->B > 1) s->stride = v.stride[0];
  }
  s->table = (const int*)v.ptr;
  s->cu = NULL;
  if (cu == Py_None) return tokens == s->B;
  if (!look(cu, t_i32, index, &v) || v.dims != 1 || !v.contiguous || v.size[0] != (long long)s->B + 1) return 0;
  s->cu = (const int*)v.ptr;
  return 1;
}

/* The current stream when `index` is torch's current device. */
static int stream_of(PyObject* index_obj, long index, attn_stream_t* stream) {
  PyObject* x = PyObject_CallNoArgs(f_device);
  if (!x) return 0;
  const long now = PyLong_AsLong(x);
  Py_DECREF(x);
  if (now != index) return 0;
  x = PyObject_CallOneArg(f_stream, index_obj);
  if (!x) return 0;
  *stream = (attn_stream_t)PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return !PyErr_Occurred();
}

static PyObject* not_taken(void) {
  PyErr_Clear();
  Py_RETURN_NOTIMPLEMENTED;
}

static PyObject* new_tensor(PyObject* shape, PyObject* dtype, PyObject* device) {
  PyObject* a[3] = {shape, dtype, device};
  return shape ? PyObject_Vectorcall(f_empty, a, 1, kw_dtype_device) : NULL;
}

static int scale_of(PyObject* x, long long d, float* scale) {
  if (x == Py_None) {
    *scale = (float)(1.0 / sqrt((double)d));
    return 1;
  }
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) return 0;
  *scale = (float)v;
  return 1;
}

/* append(cache struct, index, q, k, v, page_table, kv_lens, cu_seqlens, inv_freq,
 *        interleaved, q_out) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) return not_taken();
  const attn_paged_cache* c = (const attn_paged_cache*)PyLong_AsVoidPtr(a[0]);
  const long index = PyLong_AsLong(a[1]);
  if (!c || PyErr_Occurred()) return not_taken();
  PyObject *q = a[2], *q_out = a[10];
  view k, v, x, y, f;
  long long ks, vs, qs = 0, os = 0;
  seqs s;
  if (!tokens_of(a[3], index, c->d, &k, &ks) || k.size[1] != c->H_kv || !tokens_of(a[4], index, c->d, &v, &vs) ||
      v.size[1] != c->H_kv || v.size[0] != k.size[0] || !seqs_of(a[5], a[6], a[7], index, k.size[0], &s))
    return not_taken();
  const double* freq = NULL;
  int rotary = 0, H_q = 0;
  if (a[8] != Py_None) {
    if (!look(a[8], t_f64, index, &f) || f.dims != 1 || !f.contiguous || f.size[0] > 4096) return not_taken();
    freq = (const double*)f.ptr;
    rotary = 2 * (int)f.size[0];
  }
  const int inter = PyObject_IsTrue(a[9]);
  attn_stream_t stream;
  if (inter < 0 || !stream_of(a[1], index, &stream)) return not_taken();
  PyObject* result = NULL;
  x.ptr = y.ptr = NULL;
  if (q == Py_None) {
    if (q_out != Py_None) return not_taken();
    result = Py_NewRef(Py_None);
  } else {
    if (!tokens_of(q, index, c->d, &x, &qs) || x.size[0] != k.size[0]) return not_taken();
    H_q = (int)x.size[1];
    if (q_out != Py_None) {
      if (!tokens_of(q_out, index, c->d, &y, &os) || y.size[0] != x.size[0] || y.size[1] != x.size[1])
        return not_taken();
      result = Py_NewRef(q_out);
    } else if (!rotary) {
      result = Py_NewRef(q);
    } else {
      PyObject* args[2] = {q, o_contiguous};
      result = PyObject_Vectorcall(f_empty_like, args, 1, kw_memory_format);
      if (!result || !tokens_of(result, index, c->d, &y, &os)) {
        Py_XDECREF(result);
        return not_taken();
      }
    }
    if (result == q && !rotary) { /* nothing to write */
      H_q = 0;
      x.ptr = y.ptr = NULL;
      qs = os = 0;
    }
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = c_append(c, x.ptr, k.ptr, v.ptr, y.ptr, qs, ks, vs, os, (int)k.size[0], s.B, H_q, s.cu, s.lens, s.table,
                    s.cols, s.stride, freq, rotary, inter, stream);
  Py_END_ALLOW_THREADS
  if (status) {
    Py_DECREF(result);
    return PyLong_FromLong(status);
  }
  return result;
}

/* The outputs and the workspace (None where there is none to have) of an attention call; 0
 * and nothing held on failure. */
static int outputs(PyObject* q, long long rows, long long cols, size_t bytes, PyObject* device, PyObject** o,
                   PyObject** lse, PyObject** ws, void** ptr) {
  PyObject* shape = Py_BuildValue("(LL)", rows, cols);
  PyObject* size = bytes ? PyLong_FromSize_t(bytes) : NULL;
  *o = PyObject_CallOneArg(f_empty_like, q);
  *lse = new_tensor(shape, t_f32, device);
  *ws = bytes ? new_tensor(size, t_u8, device) : Py_NewRef(Py_None);
  Py_XDECREF(shape);
  Py_XDECREF(size);
  PyObject* all[3] = {*o, *lse, *ws};
  int ok = 1;
  ptr[2] = NULL;
  for (int i = 0; ok && i < (bytes ? 3 : 2); ++i) {
    PyObject* x = all[i] ? PyObject_CallMethodNoArgs(all[i], n_data_ptr) : NULL;
    ptr[i] = x ? PyLong_AsVoidPtr(x) : NULL;
    ok = x != NULL;
    Py_XDECREF(x);
  }
  if (ok && !PyErr_Occurred()) return 1;
  for (int i = 0; i < 3; ++i) Py_XDECREF(all[i]);
  return 0;
}

static PyObject* answer(int status, PyObject* o, PyObject* lse, PyObject* ws) {
  Py_DECREF(ws);
  PyObject* r = status ? PyLong_FromLong(status) : PyTuple_Pack(2, o, lse);
  Py_DECREF(o);
  Py_DECREF(lse);
  return r;
}

/* decode(cache struct, index, device, q, page_table, kv_lens, scale) */
static PyObject* decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) return not_taken();
  const attn_paged_cache* c = (const attn_paged_cache*)PyLong_AsVoidPtr(a[0]);
  const long index = PyLong_AsLong(a[1]);
  if (!c || PyErr_Occurred()) return not_taken();
  view q;
  long long apart;
  seqs s;
  float scale;
  attn_stream_t stream;
  if (!tokens_of(a[3], index, c->d, &q, &apart) || !q.contiguous || q.size[1] < 1 || q.size[1] % c->H_kv ||
      !seqs_of(a[4], a[5], Py_None, index, q.size[0], &s) || !scale_of(a[6], c->d, &scale) ||
      !stream_of(a[1], index, &stream))
    return not_taken();
  const size_t bytes = c_bytes(c, s.B, s.B, (int)q.size[1], 0, s.cols);
  PyObject *o, *lse, *ws;
  void* ptr[3];
  if (!outputs(a[3], s.B, q.size[1], bytes, a[2], &o, &lse, &ws, ptr)) return not_taken();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = c_decode(c, q.ptr, ptr[0], (float*)ptr[1], s.B, (int)q.size[1], s.lens, s.table, s.cols, s.stride, scale,
                    ptr[2], bytes, stream);
  Py_END_ALLOW_THREADS
  return answer(status, o, lse, ws);
}

/* forward(cache struct, index, device, q, page_table, kv_lens, cu_seqlens, scale, causal) */
static PyObject* forward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 9 || a[6] == Py_None) return not_taken();
  const attn_paged_cache* c = (const attn_paged_cache*)PyLong_AsVoidPtr(a[0]);
  const long index = PyLong_AsLong(a[1]);
  if (!c || PyErr_Occurred()) return not_taken();
  view q;
  long long apart;
  seqs s;
  float scale;
  attn_stream_t stream;
  if (!tokens_of(a[3], index, c->d, &q, &apart) || !q.contiguous || q.size[1] < 1 || q.size[1] % c->H_kv ||
      !seqs_of(a[4], a[5], a[6], index, q.size[0], &s) || !scale_of(a[7], c->d, &scale) ||
      !stream_of(a[1], index, &stream))
    return not_taken();
  const int causal = PyObject_IsTrue(a[8]), T = (int)q.size[0], H_q = (int)q.size[1];
  if (causal < 0) return not_taken();
  const size_t bytes = c_bytes(c, T, s.B, H_q, 1, s.cols);
  PyObject *o, *lse, *ws;
  void* ptr[3];
  if (!outputs(a[3], H_q, T, bytes, a[2], &o, &lse, &ws, ptr)) return not_taken();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = c_fwd(c, q.ptr, ptr[0], (float*)ptr[1], T, s.B, H_q, s.cu, s.lens, s.table, s.cols, s.stride, causal, scale,
                 ptr[2], bytes, stream);
  Py_END_ALLOW_THREADS
  return answer(status, o, lse, ws);
}

/* setup(addresses of the four C functions, torch module) */
static PyObject* setup(PyObject* self, PyObject* args) {
  unsigned long long f[4];
  PyObject* torch;
  if (!PyArg_ParseTuple(args, "KKKKO", &f[0], &f[1], &f[2], &f[3], &torch)) return NULL;
  c_append = (append_fn)(size_t)f[0];
  c_decode = (decode_fn)(size_t)f[1];
  c_fwd = (fwd_fn)(size_t)f[2];
  c_bytes = (bytes_fn)(size_t)f[3];
  PyObject* low = PyObject_GetAttrString(torch, "_C");
  PyObject* cuda = PyObject_GetAttrString(torch, "cuda");
  if (!low || !cuda) return NULL;
  if (!(t_bf16 = PyObject_GetAttrString(torch, "bfloat16")) || !(t_f32 = PyObject_GetAttrString(torch, "float32")) ||
      !(t_f64 = PyObject_GetAttrString(torch, "float64")) || !(t_i32 = PyObject_GetAttrString(torch, "int32")) ||
      !(t_u8 = PyObject_GetAttrString(torch, "uint8")) || !(f_empty = PyObject_GetAttrString(torch, "empty")) ||
      !(f_empty_like = PyObject_GetAttrString(torch, "empty_like")) ||
      !(o_contiguous = PyObject_GetAttrString(torch, "contiguous_format")) ||
      !(f_device = PyObject_GetAttrString(cuda, "current_device")) ||
      !(f_stream = PyObject_GetAttrString(low, "_cuda_getCurrentRawStream")))
    return NULL;
  Py_DECREF(low);
  Py_DECREF(cuda);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, NULL},
    {"forward", (PyCFunction)(void (*)(void))forward, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__paged_call(void) {
  n_dtype = PyUnicode_InternFromString("dtype");
  n_shape = PyUnicode_InternFromString("shape");
  n_get_device = PyUnicode_InternFromString("get_device");
  n_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  n_stride = PyUnicode_InternFromString("stride");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  kw_dtype_device = Py_BuildValue("(ss)", "dtype", "device");
  kw_memory_format = Py_BuildValue("(s)", "memory_format");
  if (!n_dtype || !n_shape || !n_get_device || !n_is_contiguous || !n_stride || !n_data_ptr || !kw_dtype_device ||
      !kw_memory_format)
    return NULL;
  return PyModule_Create(&module);
}
