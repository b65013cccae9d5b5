/* mk_bind.c -- the checks and the marshalling of the rotary, cache and paged attention calls, for
 * Python.  The calls of a decode step take the GPU a few microseconds, less than ctypes and
 * attribute look-ups in Python take the host (rope: 16 us of Python against 4 us in the library),
 * so their arguments are read here.  The functions take the entry point's address from the ctypes
 * library, so that whatever build of it is in use is the one that is called.
 * CPython C API only: tensors are read through their Python methods.  The interpreter's lock is given up for the
 * library's call, which waits where the GPU's queue is full: the arguments, and with them the memory that the call
 * reads, stay referenced by the caller. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "mk.h"

typedef struct {
  void *ptr;
  int dtype;               /* mk_dtype, or one of the below */
  int device, dims;
  long long shape[4], stride[4];
} tensor;
enum { T_I32 = 16, T_I64 = 17, T_F64 = 18, T_OTHER = 19 };

static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_get_device, *s_device, *s_kw;
static PyObject *dtypes[7];        /* bf16, f32, f16, e4m3, i32, i64, f64 */
static const int dtype_codes[7] = {MK_BF16, MK_F32, MK_F16, MK_E4M3, T_I32, T_I64, T_F64};
static PyObject *raw_stream;       /* torch._C._cuda_getCurrentRawStream */
static PyObject *empty;            /* torch.empty: 1.6 us; the method new_empty takes 5 */
static PyObject *current_device;   /* torch._C._cuda_getDevice */

static int refuse(const char *what) {
  PyErr_SetString(PyExc_ValueError, what);
  return -1;
}
#define NEED(cond, what) \
  do { if (!(cond)) { refuse(what); return NULL; } } while (0)

static int read_tensor(PyObject *t, tensor *o, const char *name) {
  PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!p) {
    PyErr_Format(PyExc_ValueError, "%s is not a tensor", name);
    return -1;
  }
  o->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  p = PyObject_GetAttr(t, s_dtype);
  if (!p) return -1;
  o->dtype = T_OTHER;
  for (int i = 0; i < 7; ++i)
    if (p == dtypes[i]) o->dtype = dtype_codes[i];
  Py_DECREF(p);
  p = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!p) return -1;
  o->device = (int)PyLong_AsLong(p);
  Py_DECREF(p);
  PyObject *shape = PyObject_GetAttr(t, s_shape), *stride = shape ? PyObject_CallMethodNoArgs(t, s_stride) : NULL;
  if (!stride || !PyTuple_Check(shape) || !PyTuple_Check(stride)) {
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    if (!PyErr_Occurred()) refuse("a tensor has no shape or stride");
    return -1;
  }
  o->dims = (int)PyTuple_GET_SIZE(shape);
  for (int i = 0; i < 4 && i < o->dims; ++i) {
    o->shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    o->stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, i));
  }
  Py_DECREF(shape);
  Py_DECREF(stride);
  return PyErr_Occurred() ? -1 : 0;
}

/* A [tokens x heads x d] tensor; the stride of a dimension of one (or no) element says nothing and becomes 0. */
static int read_rows(PyObject *t, tensor *o, const char *name, const tensor *like, int same_heads) {
  if (read_tensor(t, o, name)) return -1;
  if (o->dims != 3 || o->device < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be a [tokens x heads x d] CUDA tensor", name);
    return -1;
  }
  if (o->stride[2] != 1 && o->shape[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", name);
    return -1;
  }
  if (like && (o->dtype != like->dtype || o->device != like->device)) {
    PyErr_Format(PyExc_ValueError, "%s's type or device is not that of the others", name);
    return -1;
  }
  if (like && (o->shape[0] != like->shape[0] || o->shape[2] != like->shape[2] ||
               (same_heads && o->shape[1] != like->shape[1]))) {
    PyErr_Format(PyExc_ValueError, "%s's shape does not fit", name);
    return -1;
  }
  if (o->shape[0] <= 1) o->stride[0] = 0;
  if (o->shape[1] <= 1) o->stride[1] = 0;
  return 0;
}

static int read_rotation(PyObject *freqs, PyObject *positions, PyObject *start, PyObject *interleaved,
                         PyObject *inverse, PyObject *magnitude, long long tokens, int device, mk_rotation *r) {
  tensor t;
  if (read_tensor(freqs, &t, "freqs")) return -1;
  if (t.dtype != T_F64 || t.dims != 1 || (t.stride[0] != 1 && t.shape[0] > 1) || t.device != device)
    return refuse("freqs must be a contiguous float64 vector on the tensors' device");
  r->freqs = (const double *)t.ptr;
  r->rot = (int)(2 * (t.shape[0] < (1 << 20) ? t.shape[0] : (1 << 20)));
  r->positions = NULL;
  r->positions_64 = 0;
  if (positions != Py_None) {
    if (read_tensor(positions, &t, "positions")) return -1;
    long long n = 1;
    int plain = t.dims <= 4;
    for (int i = t.dims - 1; i >= 0 && plain; --i) {
      if (t.shape[i] > 1 && t.stride[i] != n) plain = 0;
      n *= t.shape[i];
    }
    if ((t.dtype != T_I32 && t.dtype != T_I64) || !plain || n != tokens || t.device != device)
      return refuse("positions must be int32 or int64, contiguous, one for each token, on the tensors' device");
    r->positions = t.ptr;
    r->positions_64 = t.dtype == T_I64;
  }
  r->start = PyLong_AsLongLong(start);
  r->interleaved = PyObject_IsTrue(interleaved);
  r->inverse = PyObject_IsTrue(inverse);
  r->magnitude = (float)PyFloat_AsDouble(magnitude);
  return PyErr_Occurred() ? -1 : 0;
}

static int read_seqs(PyObject *cu_q, PyObject *kv_len, PyObject *pages, int device, mk_seq_batch *s) {
  tensor c, l, p;
  if (read_tensor(cu_q, &c, "cu_q") || read_tensor(kv_len, &l, "kv_len") || read_tensor(pages, &p, "pages")) return -1;
  if (c.dtype != T_I32 || l.dtype != T_I32 || p.dtype != T_I32 || c.device != device || l.device != device ||
      p.device != device)
    return refuse("cu_q, kv_len and pages must be int32 on the tensors' device");
  if (c.dims != 1 || l.dims != 1 || (c.stride[0] != 1 && c.shape[0] > 1) || (l.stride[0] != 1 && l.shape[0] > 1) ||
      c.shape[0] != l.shape[0] + 1)
    return refuse("cu_q must have one entry more than kv_len, both contiguous vectors");
  if (p.dims != 2 || p.shape[0] != l.shape[0] || (p.stride[1] != 1 && p.shape[1] > 1))
    return refuse("pages must be [batch x max_pages] with contiguous rows");
  if (l.shape[0] >= (1 << 24) || p.shape[1] >= (1LL << 31)) return refuse("the batch is too large");
  s->cu_q = (const int *)c.ptr;
  s->kv_len = (const int *)l.ptr;
  s->pages = (const int *)p.ptr;
  s->pages_stride = p.stride[0];
  s->batch = (int)l.shape[0];
  s->max_pages = (int)p.shape[1];
  return 0;
}

/* A launch goes to the current device, whatever its pointers' and its stream's device. */
static int check_device(int device) {
  PyObject *v = PyObject_CallNoArgs(current_device);
  if (!v) return -1;
  const long now = PyLong_AsLong(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (now == device) return 0;
  PyErr_Format(PyExc_ValueError, "the tensors are on device %d, and the current device is %ld: use torch.cuda.device(%d)",
               device, now, device);
  return -1;
}

static int read_stream(PyObject *stream, int device, mk_stream_t *s) {
  PyObject *v;
  if (stream == Py_None) {
    PyObject *d = PyLong_FromLong(device);
    v = d ? PyObject_CallOneArg(raw_stream, d) : NULL;
    Py_XDECREF(d);
  } else {
    v = Py_NewRef(stream);         /* a raw handle */
  }
  if (!v) return -1;
  *s = (mk_stream_t)PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

static PyObject *empty_like_rows(PyObject *t, long long tokens, long long heads, long long d, PyObject *dtype) {
  PyObject *shape = d ? Py_BuildValue("(LLL)", tokens, heads, d) : Py_BuildValue("(LL)", tokens, heads);
  PyObject *type = dtype ? Py_NewRef(dtype) : PyObject_GetAttr(t, s_dtype), *device = PyObject_GetAttr(t, s_device);
  PyObject *args[3] = {shape, type, device};
  PyObject *r = shape && type && device ? PyObject_Vectorcall(empty, args, 1, s_kw) : NULL;
  Py_XDECREF(shape);
  Py_XDECREF(type);
  Py_XDECREF(device);
  return r;
}

/* cache(k, v, k_scale, v_scale) -> the bytes of an mk_kv_cache */
static PyObject *bind_cache(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 4, "cache: 4 arguments");
  tensor k, v;
  if (read_tensor(a[0], &k, "k") || read_tensor(a[1], &v, "v")) return NULL;
  NEED(k.dims == 4 && v.dims == 4 && k.device >= 0 && v.device == k.device, "k and v must be 4-D CUDA tensors");
  NEED(k.dtype == v.dtype && (k.dtype == MK_BF16 || k.dtype == MK_F16 || k.dtype == MK_E4M3),
       "unsupported cache types: bf16, fp16 or float8_e4m3fn, the same for k and v");
  mk_kv_cache c;
  for (int i = 0; i < 4; ++i)
    NEED(k.shape[i] == v.shape[i] && (k.stride[i] == v.stride[i] || k.shape[i] <= 1),
         "k and v must have the same shape and strides");
  NEED(k.stride[3] == 1 || k.shape[3] == 1, "the last dimension must be contiguous");
  NEED(k.shape[1] < (1 << 30) && k.shape[2] < (1 << 30) && k.shape[3] < (1 << 30), "the cache is too large");
  float **scale[2] = {&c.k_scale, &c.v_scale};
  for (int i = 0; i < 2; ++i) {
    *scale[i] = NULL;
    if (k.dtype != MK_E4M3) {
      NEED(a[2 + i] == Py_None, "16-bit caches have no scales");
      continue;
    }
    tensor s;
    NEED(a[2 + i] != Py_None, "an 8-bit cache needs k_scale and v_scale: contiguous fp32 [n_pages x heads]");
    if (read_tensor(a[2 + i], &s, "a scale")) return NULL;
    NEED(s.dtype == MK_F32 && s.dims == 2 && s.device == k.device && s.shape[0] == k.shape[0] &&
             s.shape[1] == k.shape[1] && (s.stride[1] == 1 || s.shape[1] <= 1) &&
             (s.stride[0] == s.shape[1] || s.shape[0] <= 1),
         "an 8-bit cache needs k_scale and v_scale: contiguous fp32 [n_pages x heads]");
    *scale[i] = (float *)s.ptr;
  }
  c.k = k.ptr;
  c.v = v.ptr;
  c.page_stride = k.shape[0] > 1 ? k.stride[0] : 0;
  c.head_stride = k.shape[1] > 1 ? k.stride[1] : 0;
  c.slot_stride = k.stride[2];
  c.n_pages = k.shape[0];
  c.dtype = k.dtype;
  c.heads = (int)k.shape[1];
  c.page_size = (int)k.shape[2];
  c.d = (int)k.shape[3];
  return Py_BuildValue("(y#i)", (const char *)&c, (Py_ssize_t)sizeof(c), k.device);
}

typedef mk_status (*rope_fn)(const void *, void *, mk_dtype, long long, int, int, long long, long long, long long,
                             long long, const mk_rotation *, mk_stream_t);
/* rope(fn, x, out, freqs, positions, start, interleaved, inverse, magnitude, stream) -> status */
static PyObject *bind_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 10, "rope: 10 arguments");
  tensor x, y;
  mk_rotation r;
  mk_stream_t s;
  if (read_rows(a[1], &x, "x", NULL, 0) || read_rows(a[2], &y, "out", &x, 1)) return NULL;
  NEED(x.dtype == MK_BF16 || x.dtype == MK_F16 || x.dtype == MK_F32, "unsupported dtype: bf16, fp16 or fp32");
  NEED(x.shape[1] < (1 << 30) && x.shape[2] < (1 << 30), "x is too large");
  if (check_device(x.device) || read_rotation(a[3], a[4], a[5], a[6], a[7], a[8], x.shape[0], x.device, &r) ||
      read_stream(a[9], x.device, &s))
    return NULL;
  rope_fn fn = (rope_fn)PyLong_AsVoidPtr(a[0]);
  if (!fn) return NULL;
  mk_status e;
  Py_BEGIN_ALLOW_THREADS
  e = fn(x.ptr, y.ptr, (mk_dtype)x.dtype, x.shape[0], (int)x.shape[1], (int)x.shape[2], x.stride[0], x.stride[1],
         y.stride[0], y.stride[1], &r, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(e);
}

static int read_cache(PyObject *bytes, PyObject *device, const mk_kv_cache **c, int *dev) {
  if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof(mk_kv_cache)) return refuse("not a cache");
  *c = (const mk_kv_cache *)PyBytes_AS_STRING(bytes);
  *dev = (int)PyLong_AsLong(device);
  return PyErr_Occurred() ? -1 : 0;
}

typedef mk_status (*append_fn)(const mk_kv_cache *, const void *, const void *, mk_dtype, long long, long long, long long,
                               long long, long long, const void *, void *, int, long long, long long, long long,
                               long long, const mk_seq_batch *, const mk_rotation *, void *, size_t, mk_stream_t);
/* append(fn, cache, device, k, v, cu_q, kv_len, pages, q, q_out, freqs, positions, interleaved, magnitude, workspace,
 * stream) -> (status, q_out) */
static PyObject *bind_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 16, "append: 16 arguments");
  const mk_kv_cache *c;
  int dev;
  tensor k, v, q, o, w;
  mk_seq_batch s;
  mk_rotation r;
  mk_stream_t st;
  if (read_cache(a[1], a[2], &c, &dev) || read_rows(a[3], &k, "k", NULL, 0) || read_rows(a[4], &v, "v", &k, 1)) return NULL;
  NEED(k.shape[1] == c->heads && k.shape[2] == c->d, "k and v do not fit the cache's heads and d");
  NEED((k.dtype == MK_BF16 || k.dtype == MK_F16) && (c->dtype == k.dtype || c->dtype == MK_E4M3) && k.device == dev,
       "k and v do not have the cache's type or device");
  if (check_device(dev) || read_seqs(a[5], a[6], a[7], dev, &s)) return NULL;
  const int has_q = a[8] != Py_None, turn = a[10] != Py_None;
  NEED(turn || !has_q, "q is only rotated: give freqs with it");
  if (turn && read_rotation(a[10], a[11], Py_False, a[12], Py_False, a[13], k.shape[0], dev, &r)) return NULL;
  PyObject *out = Py_NewRef(a[9]);
  if (has_q) {
    if (read_rows(a[8], &q, "q", &k, 0)) goto fail;
    if (q.shape[1] >= (1 << 30)) {
      refuse("q is too large");
      goto fail;
    }
    if (out == Py_None) {
      Py_DECREF(out);
      out = empty_like_rows(a[8], q.shape[0], q.shape[1], q.shape[2], NULL);
      if (!out) return NULL;
    }
    if (read_rows(out, &o, "q_out", &q, 1)) goto fail;
  }
  if (read_tensor(a[14], &w, "workspace") || read_stream(a[15], dev, &st)) goto fail;
  {
    append_fn fn = (append_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto fail;
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(c, k.ptr, v.ptr, (mk_dtype)k.dtype, k.shape[0], k.stride[0], k.stride[1], v.stride[0], v.stride[1],
           has_q ? q.ptr : NULL, has_q ? o.ptr : NULL, has_q ? (int)q.shape[1] : 0, has_q ? q.stride[0] : 0,
           has_q ? q.stride[1] : 0, has_q ? o.stride[0] : 0, has_q ? o.stride[1] : 0, &s, turn ? &r : NULL, w.ptr,
           (size_t)w.shape[0], st);
    Py_END_ALLOW_THREADS
    return Py_BuildValue("(iN)", (int)e, has_q ? out : (Py_DECREF(out), Py_NewRef(Py_None)));
  }
fail:
  Py_DECREF(out);
  return NULL;
}

typedef size_t (*size_fn)(long long, int, int, int, int);
typedef mk_status (*attention_fn)(const void *, void *, float *, mk_dtype, long long, int, long long, long long, long long,
                                  long long, const mk_kv_cache *, const mk_seq_batch *, float, int, int, int, int, void *,
                                  size_t, const mk_config *, mk_stream_t);
/* attention(fn, size_fn, get_workspace, q, cache, device, cu_q, kv_len, pages, causal, window, sinks, scale, max_q, out,
 * lse (a tensor, True to make one, or None), config address, stream) -> (status, out, lse) */
static PyObject *bind_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 18, "attention: 18 arguments");
  const mk_kv_cache *c;
  int dev;
  tensor q, o, l, w;
  mk_seq_batch s;
  mk_stream_t st;
  if (read_rows(a[3], &q, "q", NULL, 0) || read_cache(a[4], a[5], &c, &dev)) return NULL;
  NEED((q.dtype == MK_BF16 || q.dtype == MK_F16) && (c->dtype == q.dtype || c->dtype == MK_E4M3) && q.device == dev,
       "q does not have the cache's type or device");
  NEED(c->dtype != MK_E4M3 || q.dtype == MK_BF16, "an 8-bit cache takes bf16 queries");
  NEED(q.shape[2] == c->d, "q's d is not the cache's");
  NEED(q.shape[1] < (1 << 30), "q has too many heads");
  if (check_device(dev) || read_seqs(a[6], a[7], a[8], dev, &s)) return NULL;
  const int causal = PyObject_IsTrue(a[9]);
  const long long window = PyLong_AsLongLong(a[10]), sinks = PyLong_AsLongLong(a[11]), max_q = PyLong_AsLongLong(a[13]);
  const double scale = a[12] == Py_None ? 1.0 / sqrt((double)c->d) : PyFloat_AsDouble(a[12]);
  void *cfg = a[16] == Py_None ? NULL : PyLong_AsVoidPtr(a[16]);
  if (PyErr_Occurred()) return NULL;
  NEED(window <= 0x7fffffff && sinks <= 0x7fffffff && max_q <= 0x7fffffff && window >= -1 && sinks >= -1 && max_q >= -1,
       "window, sinks or max_q is out of range");
  PyObject *out = NULL, *lse = NULL, *ws = NULL, *result = NULL;
  out = a[14] == Py_None ? empty_like_rows(a[3], q.shape[0], q.shape[1], q.shape[2], NULL) : Py_NewRef(a[14]);
  if (!out || read_rows(out, &o, "out", &q, 1)) goto end;
  lse = a[15] == Py_True ? empty_like_rows(a[3], q.shape[0], q.shape[1], 0, dtypes[1]) : Py_NewRef(a[15]);
  if (!lse) goto end;
  l.ptr = NULL;
  if (lse != Py_None) {
    if (read_tensor(lse, &l, "lse")) goto end;
  }
  {
    const size_t need = ((size_fn)PyLong_AsVoidPtr(a[1]))(q.shape[0], (int)q.shape[1], c->heads, c->d, s.batch);
    if (need == 0) {
      result = Py_BuildValue("(iOO)", (int)MK_ERR_INVALID, Py_None, Py_None);
      goto end;
    }
    PyObject *bytes = PyLong_FromSize_t(need);
    ws = bytes ? PyObject_CallOneArg(a[2], bytes) : NULL;
    Py_XDECREF(bytes);
    if (!ws || read_tensor(ws, &w, "workspace") || read_stream(a[17], dev, &st)) goto end;
    attention_fn fn = (attention_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto end;
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(q.ptr, o.ptr, (float *)l.ptr, (mk_dtype)q.dtype, q.shape[0], (int)q.shape[1], q.stride[0], q.stride[1],
           o.stride[0], o.stride[1], c, &s, (float)scale, causal, (int)window, (int)sinks, (int)max_q, w.ptr,
           (size_t)w.shape[0], (const mk_config *)cfg, st);
    Py_END_ALLOW_THREADS
    result = Py_BuildValue("(iOO)", (int)e, out, lse);
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(lse);
  Py_XDECREF(ws);
  return result;
}

/* setup(dtypes in the order of `dtypes`, raw_stream, empty, current_device) */
static PyObject *bind_setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 4 && PyTuple_Check(a[0]) && PyTuple_GET_SIZE(a[0]) == 7, "setup: (7 dtypes, three functions)");
  for (int i = 0; i < 7; ++i) Py_XSETREF(dtypes[i], Py_NewRef(PyTuple_GET_ITEM(a[0], i)));
  Py_XSETREF(raw_stream, Py_NewRef(a[1]));
  Py_XSETREF(empty, Py_NewRef(a[2]));
  Py_XSETREF(current_device, Py_NewRef(a[3]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", (PyCFunction)(void (*)(void))bind_setup, METH_FASTCALL, NULL},
                                {"cache", (PyCFunction)(void (*)(void))bind_cache, METH_FASTCALL, NULL},
                                {"rope", (PyCFunction)(void (*)(void))bind_rope, METH_FASTCALL, NULL},
                                {"append", (PyCFunction)(void (*)(void))bind_append, METH_FASTCALL, NULL},
                                {"attention", (PyCFunction)(void (*)(void))bind_attention, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mkbind", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mkbind(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_device = PyUnicode_InternFromString("device");
  s_kw = Py_BuildValue("(ss)", "dtype", "device");
  return PyModule_Create(&module);
}
