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
typedef int (*lists_fn)(const attn_paged_cache*, const void*, void*, float*, int, int, const int*, const int*, int,
                        long long, long long, float, void*, size_t, attn_stream_t);
typedef int (*bounds_fn)(const attn_paged_cache*, void*, int, int, const int*, const int*, const int*, int, long long,
                         attn_stream_t);
typedef int (*select_fn)(const attn_paged_cache*, const void*, const void*, int*, int*, int, int, int, const int*,
                         const int*, const int*, int, long long, int, int, int, attn_stream_t);
typedef size_t (*bytes_fn)(const attn_paged_cache*, int, int, int, int, int);

static append_fn c_append;
static decode_fn c_decode;
static fwd_fn c_fwd;
static bytes_fn c_bytes;
static lists_fn c_lists;
static bounds_fn c_bounds;
static select_fn c_select;
/* from torch */
static PyObject *t_bf16, *t_f32, *t_f64, *t_i32, *t_u8, *f_empty, *f_zeros, *f_empty_like, *f_device, *f_stream, *o_contiguous;
/* names */
static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_stride, *n_data_ptr;
static PyObject *kw_dtype_device, *kw_memory_format;

/* What a call knows of a tensor. */
enum { kDims = 4 };
typedef struct {
  long long size[kDims], stride[kDims];
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

/* 1 when t is a tensor of that dtype on device `index` with at most kDims dimensions. */
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
  v->dims = integers(x, v->size, kDims);
  Py_XDECREF(x);
  if (v->dims < 0) return 0;
  x = PyObject_CallMethodNoArgs(t, n_is_contiguous);
  if (!x) return 0;
  v->contiguous = x == Py_True;
  Py_DECREF(x);
  if (!v->contiguous) {
    x = PyObject_CallMethodNoArgs(t, n_stride);
    const int n = integers(x, v->stride, kDims);
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
  long long stride, head; /* head: entries between the lists of KV heads, 0 where they share a row */
} seqs;

/* lists: the page table may have a row for each of that many KV heads (0: it may not). */
static int seqs_of(PyObject* table, PyObject* lens, PyObject* cu, long index, long long tokens, int lists, seqs* s) {
  view v;
  if (!look(lens, t_i32, index, &v) || v.dims != 1 || !v.contiguous || v.size[0] >= INT_MAX) return 0;
  s->B = (int)v.size[0];
  s->lens = (const int*)v.ptr;
  if (!look(table, t_i32, index, &v) || (v.dims != 2 && (v.dims != 3 || !lists)) || v.size[0] != s->B) return 0;
  const int last = v.dims - 1;
  if (v.size[last] > INT_MAX || (last == 2 && v.size[1] != lists)) return 0;
  s->cols = (int)v.size[last];
  s->stride = last == 2 ? lists * v.size[2] : v.size[1];
  s->head = last == 2 ? v.size[2] : 0;
  if (!v.contiguous) {
    if (s->cols > 1 && v.stride[last] != 1) return 0;
    if (s->B > 1) s->stride = v.stride[0];
    if (last == 2 && lists > 1) s->head = v.stride[1];
  }
  if (last == 2 && s->head < 1) return 0; /* (paged.py says what is wrong) */
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

static PyObject* made(PyObject* by, PyObject* shape, PyObject* dtype, PyObject* device) {
  PyObject* a[3] = {shape, dtype, device};
  return shape ? PyObject_Vectorcall(by, a, 1, kw_dtype_device) : NULL;
}
static PyObject* new_tensor(PyObject* shape, PyObject* dtype, PyObject* device) {
  return made(f_empty, shape, dtype, device);
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
      v.size[1] != c->H_kv || v.size[0] != k.size[0] || !seqs_of(a[5], a[6], a[7], index, k.size[0], 0, &s))
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
      !seqs_of(a[4], a[5], Py_None, index, q.size[0], c->H_kv, &s) || !scale_of(a[6], c->d, &scale) ||
      !stream_of(a[1], index, &stream))
    return not_taken();
  const size_t bytes = c_bytes(c, s.B, s.B, (int)q.size[1], 0, s.cols);
  PyObject *o, *lse, *ws;
  void* ptr[3];
  if (!outputs(a[3], s.B, q.size[1], bytes, a[2], &o, &lse, &ws, ptr)) return not_taken();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = s.head ? c_lists(c, q.ptr, ptr[0], (float*)ptr[1], s.B, (int)q.size[1], s.lens, s.table, s.cols, s.stride,
                            s.head, scale, ptr[2], bytes, stream)
                  : c_decode(c, q.ptr, ptr[0], (float*)ptr[1], s.B, (int)q.size[1], s.lens, s.table, s.cols, s.stride,
                             scale, ptr[2], bytes, stream);
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
      !seqs_of(a[4], a[5], a[6], index, q.size[0], 0, &s) || !scale_of(a[7], c->d, &scale) ||
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

/* A contiguous tensor of bounds for that cache. */
static int bounds_of(PyObject* t, const attn_paged_cache* c, long index, view* v) {
  return look(t, t_bf16, index, v) && v->dims == 4 && v->contiguous && v->size[0] == c->num_pages &&
         v->size[1] == c->H_kv && v->size[2] == 2 && v->size[3] == c->d;
}

/* bounds(cache struct, index, bounds, page_table, kv_lens, cu_seqlens, tokens) */
static PyObject* bounds(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) return not_taken();
  const attn_paged_cache* c = (const attn_paged_cache*)PyLong_AsVoidPtr(a[0]);
  const long index = PyLong_AsLong(a[1]);
  if (!c || PyErr_Occurred()) return not_taken();
  view v, lens;
  seqs s;
  attn_stream_t stream;
  if (!look(a[4], t_i32, index, &lens) || lens.dims != 1) return not_taken();
  long long T = lens.size[0];
  if (a[6] != Py_None) {
    T = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred() || T < 0 || T > INT_MAX) return not_taken();
  } else if (a[5] != Py_None) {
    return not_taken();
  }
  if (!bounds_of(a[2], c, index, &v) || !seqs_of(a[3], a[4], a[5], index, T, 0, &s) || !stream_of(a[1], index, &stream))
    return not_taken();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = c_bounds(c, v.ptr, (int)T, s.B, s.cu, s.lens, s.table, s.cols, s.stride, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : Py_NewRef(a[2]);
}

/* select(cache struct, index, device, q, bounds, page_table, kv_lens, count, cu_seqlens, keep_first, keep_last) */
static PyObject* select_pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) return not_taken();
  const attn_paged_cache* c = (const attn_paged_cache*)PyLong_AsVoidPtr(a[0]);
  const long index = PyLong_AsLong(a[1]);
  if (!c || PyErr_Occurred()) return not_taken();
  view q, v;
  long long apart;
  seqs s;
  attn_stream_t stream;
  const long long count = PyLong_AsLongLong(a[7]), first = PyLong_AsLongLong(a[9]), last = PyLong_AsLongLong(a[10]);
  if (PyErr_Occurred() || count < 1 || count > INT_MAX || first < 0 || last < 1 || first > count || last > count - first)
    return not_taken();
  if (!tokens_of(a[3], index, c->d, &q, &apart) || !q.contiguous || q.size[1] < 1 || q.size[1] % c->H_kv ||
      !bounds_of(a[4], c, index, &v) || !seqs_of(a[5], a[6], a[8], index, q.size[0], 0, &s) ||
      !stream_of(a[1], index, &stream))
    return not_taken();
  PyObject* shape = Py_BuildValue("(LiL)", q.size[0], c->H_kv, count);
  PyObject* rows = Py_BuildValue("(L)", q.size[0]);
  PyObject* pages = new_tensor(shape, t_i32, a[2]);
  /* (rows behind the last sequence are not written: no keys for the attention that takes them) */
  PyObject* lens = made(s.cu ? f_zeros : f_empty, rows, t_i32, a[2]);
  Py_XDECREF(shape);
  Py_XDECREF(rows);
  PyObject* both[2] = {pages, lens};
  void* ptr[2] = {NULL, NULL};
  int ok = pages && lens;
  for (int i = 0; ok && i < 2; ++i) {
    PyObject* x = PyObject_CallMethodNoArgs(both[i], n_data_ptr);
    ptr[i] = x ? PyLong_AsVoidPtr(x) : NULL;
    ok = x != NULL;
    Py_XDECREF(x);
  }
  if (!ok || PyErr_Occurred()) {
    Py_XDECREF(pages);
    Py_XDECREF(lens);
    return not_taken();
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = c_select(c, q.ptr, v.ptr, (int*)ptr[0], (int*)ptr[1], (int)q.size[0], s.B, (int)q.size[1], s.cu, s.lens, s.table,
                    s.cols, s.stride, (int)count, (int)first, (int)last, stream);
  Py_END_ALLOW_THREADS
  PyObject* r = status ? PyLong_FromLong(status) : PyTuple_Pack(2, pages, lens);
  Py_DECREF(pages);
  Py_DECREF(lens);
  return r;
}

/* setup(addresses of the seven C functions, torch module) */
static PyObject* setup(PyObject* self, PyObject* args) {
  unsigned long long f[7];
  PyObject* torch;
  if (!PyArg_ParseTuple(args, "KKKKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &torch)) return NULL;
  c_append = (append_fn)(size_t)f[0];
  c_decode = (decode_fn)(size_t)f[1];
  c_fwd = (fwd_fn)(size_t)f[2];
  c_bytes = (bytes_fn)(size_t)f[3];
  c_lists = (lists_fn)(size_t)f[4];
  c_bounds = (bounds_fn)(size_t)f[5];
  c_select = (select_fn)(size_t)f[6];
  PyObject* low = PyObject_GetAttrString(torch, "_C");
  PyObject* cuda = PyObject_GetAttrString(torch, "cuda");
  if (!low || !cuda) return NULL;
  if (!(t_bf16 = PyObject_GetAttrString(torch, "bfloat16")) || !(t_f32 = PyObject_GetAttrString(torch, "float32")) ||
      !(t_f64 = PyObject_GetAttrString(torch, "float64")) || !(t_i32 = PyObject_GetAttrString(torch, "int32")) ||
      !(t_u8 = PyObject_GetAttrString(torch, "uint8")) || !(f_empty = PyObject_GetAttrString(torch, "empty")) ||
      !(f_zeros = PyObject_GetAttrString(torch, "zeros")) || !(f_empty_like = PyObject_GetAttrString(torch, "empty_like")) ||
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
    {"bounds", (PyCFunction)(void (*)(void))bounds, METH_FASTCALL, NULL},
    {"select", (PyCFunction)(void (*)(void))select_pages, METH_FASTCALL, NULL},
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
