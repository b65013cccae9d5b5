/* mk_bind.c -- the checks and the marshalling of the rotary, cache, paged attention, norm, router
 * and 4-bit weight calls, for Python.  The calls of a decode step take the GPU a few microseconds, less than ctypes and
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
enum { T_I32 = 16, T_I64 = 17, T_F64 = 18, T_OTHER = 19, T_U8 = 20, T_BOOL = 21 };
enum { N_DTYPES = 9 };

static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_get_device, *s_device, *s_kw;
static PyObject *dtypes[N_DTYPES];  /* bf16, f32, f16, e4m3, i32, i64, f64, u8, bool */
static const int dtype_codes[N_DTYPES] = {MK_BF16, MK_F32, MK_F16, MK_E4M3, T_I32, T_I64, T_F64, T_U8, T_BOOL};
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
  for (int i = 0; i < N_DTYPES; ++i)
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

/* The memory of a descriptor's tensors: theirs still, or they have been given other memory (t.data = ..., set_, resize_) and
 * what the descriptor names may be gone. */
static int still_there(PyObject *tensors, const void *const *at, int n, const char *what) {
  if (!PyTuple_Check(tensors) || PyTuple_GET_SIZE(tensors) != n) return refuse("not a descriptor's tensors");
  for (int i = 0; i < n; ++i) {
    PyObject *t = PyTuple_GET_ITEM(tensors, i);
    if (t == Py_None) continue;
    PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!p) return -1;
    const void *now = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    if (now != at[i]) {
      PyErr_Format(PyExc_ValueError, "a tensor of the %s has been given other memory: make another one of it", what);
      return -1;
    }
  }
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

static int read_cache(PyObject *bytes, PyObject *device, PyObject *tensors, const mk_kv_cache **c, int *dev) {
  if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof(mk_kv_cache)) return refuse("not a cache");
  *c = (const mk_kv_cache *)PyBytes_AS_STRING(bytes);
  *dev = (int)PyLong_AsLong(device);
  if (PyErr_Occurred()) return -1;
  const void *const at[4] = {(*c)->k, (*c)->v, (*c)->k_scale, (*c)->v_scale};
  return still_there(tensors, at, 4, "cache");
}

typedef mk_status (*append_fn)(const mk_kv_cache *, const void *, const void *, mk_dtype, long long, long long, long long,
                               long long, long long, const void *, void *, int, long long, long long, long long,
                               long long, const mk_seq_batch *, const mk_rotation *, void *, size_t, mk_stream_t);
/* append(fn, cache, device, k, v, cu_q, kv_len, pages, q, q_out, freqs, positions, interleaved, magnitude, workspace,
 * stream, the cache's tensors) -> (status, q_out) */
static PyObject *bind_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 17, "append: 17 arguments");
  const mk_kv_cache *c;
  int dev;
  tensor k, v, q, o, w;
  mk_seq_batch s;
  mk_rotation r;
  mk_stream_t st;
  if (read_cache(a[1], a[2], a[16], &c, &dev) || read_rows(a[3], &k, "k", NULL, 0) || read_rows(a[4], &v, "v", &k, 1)) return NULL;
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
 * lse (a tensor, True to make one, or None), config address, stream, the cache's tensors) -> (status, out, lse) */
static PyObject *bind_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 19, "attention: 19 arguments");
  const mk_kv_cache *c;
  int dev;
  tensor q, o, l, w;
  mk_seq_batch s;
  mk_stream_t st;
  if (read_rows(a[3], &q, "q", NULL, 0) || read_cache(a[4], a[5], a[18], &c, &dev)) return NULL;
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

/* ------------------------------------------------------------------ norm, router, 4-bit weights */

static PyObject *new_tensor(PyObject *shape, PyObject *dtype, PyObject *device) {      /* steals shape */
  PyObject *args[3] = {shape, dtype, device};
  PyObject *r = shape && device ? PyObject_Vectorcall(empty, args, 1, s_kw) : NULL;
  Py_XDECREF(shape);
  return r;
}
static int pointer_of(PyObject *t, tensor *o) {
  PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!p) return -1;
  o->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return PyErr_Occurred() ? -1 : 0;
}
/* What a new contiguous tensor of like's shape and the given type is (like: three dimensions). */
static int read_new_rows(PyObject *t, tensor *o, const tensor *like, int dtype) {
  *o = *like;
  o->dtype = dtype;
  o->stride[2] = 1;
  o->stride[1] = o->shape[1] > 1 ? o->shape[2] : 0;
  o->stride[0] = o->shape[0] > 1 ? o->shape[1] * o->shape[2] : 0;
  return pointer_of(t, o);
}
static PyObject *dtype_object(int code) {
  for (int i = 0; i < N_DTYPES; ++i)
    if (dtype_codes[i] == code) return dtypes[i];
  return NULL;
}

/* [rows x n] or [tokens x heads x n] rows of a norm, as three dimensions. */
static int read_norm_rows(PyObject *t, tensor *o, const char *name, const tensor *like) {
  if (read_tensor(t, o, name)) return -1;
  if ((o->dims != 2 && o->dims != 3) || o->device < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be a [rows x n] or [tokens x heads x n] CUDA tensor", name);
    return -1;
  }
  if (o->dims == 2) {
    o->shape[2] = o->shape[1];
    o->stride[2] = o->stride[1];
    o->shape[1] = 1;
    o->stride[1] = 0;
  }
  if (o->stride[2] != 1 && o->shape[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", name);
    return -1;
  }
  if (like && (o->device != like->device || o->dims != like->dims || o->shape[0] != like->shape[0] ||
               o->shape[1] != like->shape[1] || o->shape[2] != like->shape[2])) {
    PyErr_Format(PyExc_ValueError, "%s's shape or device is not that of the others", name);
    return -1;
  }
  if (o->shape[1] >= (1 << 30) || o->shape[2] >= (1 << 30)) return refuse("the rows are too large");
  if (o->shape[0] <= 1) o->stride[0] = 0;
  if (o->shape[1] <= 1) o->stride[1] = 0;
  return 0;
}
static mk_rows rows_arg(const tensor *t) {
  mk_rows r = {t->ptr, t->stride[0], t->stride[1]};
  return r;
}
static int read_same_rows(PyObject *t, tensor *o, const char *name, const tensor *like) {
  if (read_norm_rows(t, o, name, like)) return -1;
  if (o->dtype == like->dtype) return 0;
  PyErr_Format(PyExc_ValueError, "%s's type is not that of the others", name);
  return -1;
}

/* A contiguous tensor of the given type and shape (dims of them; -1: any). */
static int read_plain(PyObject *t, tensor *o, const char *name, int dtype, int device, int dims, const long long *shape) {
  if (read_tensor(t, o, name)) return -1;
  int good = o->dtype == dtype && o->device == device && o->dims == dims;
  long long n = 1;
  for (int i = dims - 1; i >= 0 && good; --i) {
    if (shape[i] >= 0 && o->shape[i] != shape[i]) good = 0;
    if (n > 0 && o->shape[i] > 1 && o->stride[i] != n) good = 0;       /* (strides of nothing say nothing) */
    n *= o->shape[i];
  }
  if (good) return 0;
  PyErr_Format(PyExc_ValueError, "%s must be contiguous and have the type, shape and device that the call says", name);
  return -1;
}

static int read_weight(PyObject *w, tensor *o, const tensor *x) {
  o->ptr = NULL;
  o->dtype = x->dtype;
  if (w == Py_None) return 0;
  if (read_tensor(w, o, "weight")) return -1;
  if (o->dims != 1 || o->shape[0] != x->shape[2] || (o->stride[0] != 1 && o->shape[0] > 1) || o->device != x->device ||
      (o->dtype != x->dtype && o->dtype != MK_F32))
    return refuse("weight must be a contiguous [n] vector of the rows' type or fp32, on their device");
  return 0;
}

typedef mk_status (*norm_fn)(const mk_rows *, const mk_rows *, const void *, const mk_rows *, const mk_rows *, float *,
                             mk_dtype, mk_dtype, mk_dtype, long long, int, int, float, mk_stream_t);
/* rms_norm(fn, x, residual, weight, out, scale_out, h_out, e4m3, eps, stream) -> (status, out, scale, h) */
static PyObject *bind_norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 10, "rms_norm: 10 arguments");
  tensor x, r, w, y, h, sc;
  mk_stream_t st;
  if (read_norm_rows(a[1], &x, "x", NULL)) return NULL;
  NEED(x.dtype == MK_BF16 || x.dtype == MK_F16 || x.dtype == MK_F32, "unsupported dtype: bf16, fp16 or fp32");
  NEED(x.shape[2] >= 1, "rows of no elements have no norm");
  const int has_r = a[2] != Py_None, e4m3 = PyObject_IsTrue(a[7]);
  if (has_r && read_same_rows(a[2], &r, "residual", &x)) return NULL;
  NEED(has_r || a[6] == Py_None, "h_out is x + residual: give a residual with it");
  NEED(e4m3 || a[5] == Py_None, "only 8-bit outputs have scales");
  const double eps = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred() || read_weight(a[3], &w, &x) || check_device(x.device) || read_stream(a[9], x.device, &st)) return NULL;
  PyObject *out = NULL, *scale = NULL, *ho = NULL, *result = NULL, *device = PyObject_GetAttr(a[1], s_device);
  const int odt = e4m3 ? MK_E4M3 : x.dtype;
  out = a[4] == Py_None ? new_tensor(PyObject_GetAttr(a[1], s_shape), dtype_object(odt), device) : Py_NewRef(a[4]);
  if (!out || (a[4] == Py_None ? read_new_rows(out, &y, &x, odt) : read_norm_rows(out, &y, "out", &x))) goto end;
  if (y.dtype != odt) {
    refuse("out's type is not the output's");
    goto end;
  }
  sc.ptr = NULL;
  if (e4m3) {
    const long long shape[2] = {x.shape[0], x.shape[1]};
    scale = a[5] == Py_None
                ? new_tensor(x.dims == 3 ? Py_BuildValue("(LL)", shape[0], shape[1]) : Py_BuildValue("(L)", shape[0]), dtypes[1], device)
                : Py_NewRef(a[5]);
    if (!scale || (a[5] == Py_None ? pointer_of(scale, &sc) : read_plain(scale, &sc, "scale_out", MK_F32, x.device, x.dims - 1, shape))) goto end;
  }
  if (has_r) {
    ho = a[6] == Py_None ? new_tensor(PyObject_GetAttr(a[1], s_shape), dtype_object(x.dtype), device) : Py_NewRef(a[6]);
    if (!ho || (a[6] == Py_None ? read_new_rows(ho, &h, &x, x.dtype) : read_same_rows(ho, &h, "h_out", &x))) goto end;
  }
  {
    norm_fn fn = (norm_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto end;
    const mk_rows xr = rows_arg(&x), yr = rows_arg(&y);
    mk_rows rr, hr;
    if (has_r) {
      rr = rows_arg(&r);
      hr = rows_arg(&h);
    }
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(&xr, has_r ? &rr : NULL, w.ptr, &yr, has_r ? &hr : NULL, (float *)sc.ptr, (mk_dtype)x.dtype, (mk_dtype)w.dtype,
           (mk_dtype)odt, x.shape[0], (int)x.shape[1], (int)x.shape[2], (float)eps, st);
    Py_END_ALLOW_THREADS
    result = Py_BuildValue("(iOOO)", (int)e, out, scale ? scale : Py_None, ho ? ho : Py_None);
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(scale);
  Py_XDECREF(ho);
  Py_XDECREF(device);
  return result;
}

/* Scratch of a call: from the given get(bytes), or memory of the call's stream. */
static PyObject *scratch(PyObject *get, size_t bytes, PyObject *device, tensor *o) {
  PyObject *r;
  if (get == Py_None) {
    r = new_tensor(Py_BuildValue("(n)", (Py_ssize_t)bytes), dtype_object(T_U8), device);
    o->shape[0] = (long long)bytes;
    if (r && !pointer_of(r, o)) return r;
  } else {
    PyObject *b = PyLong_FromSize_t(bytes);
    r = b ? PyObject_CallOneArg(get, b) : NULL;
    Py_XDECREF(b);
    if (r && !read_tensor(r, o, "workspace")) return r;
  }
  Py_XDECREF(r);
  return NULL;
}

typedef size_t (*norm_size_fn)(long long, int, int);
typedef mk_status (*norm_grad_fn)(const mk_rows *, const mk_rows *, const mk_rows *, const void *, const mk_rows *, void *,
                                  mk_dtype, mk_dtype, long long, int, int, float, void *, size_t, mk_stream_t);
/* rms_norm_backward(fn, size_fn, get_workspace or None, dy, dh, h, weight, dx, dweight (True to make one, None, or a
 * tensor), eps, stream) -> (status, dx, dweight) */
static PyObject *bind_norm_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 11, "rms_norm_backward: 11 arguments");
  tensor dy, dh, h, w, dx, dw, ws;
  mk_stream_t st;
  if (read_norm_rows(a[5], &h, "h", NULL)) return NULL;
  NEED(h.dtype == MK_BF16 || h.dtype == MK_F16 || h.dtype == MK_F32, "unsupported dtype: bf16, fp16 or fp32");
  NEED(h.shape[2] >= 1, "rows of no elements have no norm");
  if (read_same_rows(a[3], &dy, "dy", &h)) return NULL;
  const int has_dh = a[4] != Py_None;
  if (has_dh && read_same_rows(a[4], &dh, "dh", &h)) return NULL;
  const double eps = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred() || read_weight(a[6], &w, &h) || check_device(h.device) || read_stream(a[10], h.device, &st)) return NULL;
  NEED(w.ptr || a[8] == Py_None, "there is no gradient of a weight without a weight");
  PyObject *out = NULL, *dwo = NULL, *space = NULL, *result = NULL, *device = PyObject_GetAttr(a[5], s_device);
  out = a[7] == Py_None ? new_tensor(PyObject_GetAttr(a[5], s_shape), dtype_object(h.dtype), device) : Py_NewRef(a[7]);
  if (!out || (a[7] == Py_None ? read_new_rows(out, &dx, &h, h.dtype) : read_same_rows(out, &dx, "dx", &h))) goto end;
  dw.ptr = ws.ptr = NULL;
  ws.shape[0] = 0;
  if (a[8] != Py_None) {
    const long long shape[1] = {h.shape[2]};
    dwo = a[8] == Py_True ? new_tensor(Py_BuildValue("(L)", shape[0]), dtype_object(w.dtype), device) : Py_NewRef(a[8]);
    if (!dwo || (a[8] == Py_True ? pointer_of(dwo, &dw) : read_plain(dwo, &dw, "dweight", w.dtype, h.device, 1, shape))) goto end;
    const size_t need = ((norm_size_fn)PyLong_AsVoidPtr(a[1]))(h.shape[0], (int)h.shape[1], (int)h.shape[2]);
    if (need == 0) {
      result = Py_BuildValue("(iOO)", (int)MK_ERR_INVALID, Py_None, Py_None);
      goto end;
    }
    space = scratch(a[2], need, device, &ws);
    if (!space) goto end;
  }
  {
    norm_grad_fn fn = (norm_grad_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto end;
    const mk_rows yr = rows_arg(&dy), hr = rows_arg(&h), xr = rows_arg(&dx);
    mk_rows sr;
    if (has_dh) sr = rows_arg(&dh);
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(&yr, has_dh ? &sr : NULL, &hr, w.ptr, &xr, dw.ptr, (mk_dtype)h.dtype, (mk_dtype)w.dtype, h.shape[0],
           (int)h.shape[1], (int)h.shape[2], (float)eps, ws.ptr, (size_t)ws.shape[0], st);
    Py_END_ALLOW_THREADS
    result = Py_BuildValue("(iOO)", (int)e, out, dwo ? dwo : Py_None);
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(device);
  Py_XDECREF(dwo);
  Py_XDECREF(space);
  return result;
}

/* A [rows x n] matrix with contiguous rows. */
static int read_matrix(PyObject *t, tensor *o, const char *name) {
  if (read_tensor(t, o, name)) return -1;
  if (o->dims != 2 || o->device < 0 || (o->stride[1] != 1 && o->shape[1] > 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA matrix with contiguous rows", name);
    return -1;
  }
  if (o->shape[0] <= 1) o->stride[0] = o->shape[1];
  return 0;
}
static int logits_dtype(const tensor *t) {
  return t->dtype == MK_F32 || t->dtype == MK_BF16 || t->dtype == MK_F16 ? 0 : refuse("logits must be fp32, bf16 or fp16");
}

typedef size_t (*route_size_fn)(long long, int);
typedef mk_status (*route_fn)(const void *, mk_dtype, long long, int, long long, int, int, float, const unsigned char *, int *,
                              float *, int *, int *, float *, float *, void *, size_t, mk_stream_t);
/* route(fn, size_fn, get_workspace or None, logits, topk, normalize, scale, mask, (six outputs or None each), stream)
 * -> (status, topk_idx, gates, counts, tokens, balance_loss, z_loss) */
static PyObject *bind_route(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 10 && PyTuple_Check(a[8]) && PyTuple_GET_SIZE(a[8]) == 6, "route: 10 arguments");
  tensor l, m, ws, t[6];
  mk_stream_t st;
  if (read_matrix(a[3], &l, "logits") || logits_dtype(&l)) return NULL;
  const long long topk = PyLong_AsLongLong(a[4]);
  const int normalize = PyObject_IsTrue(a[5]);
  const double scale = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) return NULL;
  NEED(l.shape[1] >= 1 && l.shape[1] < (1 << 30) && topk >= 1 && topk <= l.shape[1] && topk <= 8,
       "topk must be between 1 and the experts, at most 8");
  m.ptr = NULL;
  if (a[7] != Py_None) {
    const long long shape[1] = {l.shape[0]};
    if (read_plain(a[7], &m, "mask (bool, one for each token)", T_BOOL, l.device, 1, shape)) return NULL;
  }
  if (check_device(l.device) || read_stream(a[9], l.device, &st)) return NULL;
  static const char *names[6] = {"topk_idx", "gates", "counts", "tokens", "balance_loss", "z_loss"};
  static const int types[6] = {T_I32, MK_F32, T_I32, T_I32, MK_F32, MK_F32}, dims[6] = {2, 2, 1, 0, 0, 0};
  const long long pairs[2] = {l.shape[0], topk}, experts[1] = {l.shape[1]};
  PyObject *o[6] = {NULL}, *space = NULL, *result = NULL, *device = PyObject_GetAttr(a[3], s_device);
  for (int i = 0; i < 6; ++i) {
    PyObject *given = PyTuple_GET_ITEM(a[8], i);
    const long long *shape = i < 2 ? pairs : experts;
    if (given != Py_None) o[i] = Py_NewRef(given);
    else
      o[i] = new_tensor(i < 2 ? Py_BuildValue("(LL)", pairs[0], pairs[1]) : i == 2 ? Py_BuildValue("(L)", experts[0]) : PyTuple_New(0),
                        dtype_object(types[i]), device);
    if (!o[i] || (given == Py_None ? pointer_of(o[i], &t[i]) : read_plain(o[i], &t[i], names[i], types[i], l.device, dims[i], shape)))
      goto end;
  }
  ws.ptr = NULL;
  ws.shape[0] = 0;
  if (l.shape[0] > MK_ROUTE_SMALL) {
    const size_t need = ((route_size_fn)PyLong_AsVoidPtr(a[1]))(l.shape[0], (int)l.shape[1]);
    if (need > 0) {                      /* (0: the call refuses the sizes) */
      space = scratch(a[2], need, device, &ws);
      if (!space) goto end;
    }
  }
  {
    route_fn fn = (route_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto end;
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(l.ptr, (mk_dtype)l.dtype, l.shape[0], (int)l.shape[1], l.stride[0], (int)topk, normalize, (float)scale,
           (const unsigned char *)m.ptr, (int *)t[0].ptr, (float *)t[1].ptr, (int *)t[2].ptr, (int *)t[3].ptr,
           (float *)t[4].ptr, (float *)t[5].ptr, ws.ptr, (size_t)ws.shape[0], st);
    Py_END_ALLOW_THREADS
    result = Py_BuildValue("(iOOOOOO)", (int)e, o[0], o[1], o[2], o[3], o[4], o[5]);
  }
end:
  for (int i = 0; i < 6; ++i) Py_XDECREF(o[i]);
  Py_XDECREF(space);
  Py_XDECREF(device);
  return result;
}

typedef mk_status (*route_grad_fn)(const void *, mk_dtype, long long, int, long long, int, int, float, const int *, const int *,
                                   const int *, const float *, const float *, const float *, void *, long long, mk_stream_t);
/* route_backward(fn, logits, topk_idx, counts, tokens, dgates, dbalance, dz, normalize, scale, out, stream)
 * -> (status, dlogits) */
static PyObject *bind_route_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 12, "route_backward: 12 arguments");
  tensor l, idx, counts, tokens, g[3], dl;
  mk_stream_t st;
  if (read_matrix(a[1], &l, "logits") || logits_dtype(&l)) return NULL;
  NEED(l.shape[1] < (1 << 30), "too many experts");
  const long long any[2] = {l.shape[0], -1}, experts[1] = {l.shape[1]};
  if (read_plain(a[2], &idx, "topk_idx", T_I32, l.device, 2, any) ||
      read_plain(a[3], &counts, "counts", T_I32, l.device, 1, experts) ||
      read_plain(a[4], &tokens, "tokens", T_I32, l.device, 0, experts))
    return NULL;
  NEED(idx.shape[1] >= 1 && idx.shape[1] <= 8, "topk_idx has no or too many experts for a token");
  const long long pairs[2] = {l.shape[0], idx.shape[1]};
  static const char *names[3] = {"dgates", "dbalance", "dz"};
  for (int i = 0; i < 3; ++i) {
    g[i].ptr = NULL;
    if (a[5 + i] != Py_None && read_plain(a[5 + i], &g[i], names[i], MK_F32, l.device, i ? 0 : 2, pairs)) return NULL;
  }
  const int normalize = PyObject_IsTrue(a[8]);
  const double scale = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred() || check_device(l.device) || read_stream(a[11], l.device, &st)) return NULL;
  PyObject *device = PyObject_GetAttr(a[1], s_device), *result = NULL;
  PyObject *out = a[10] == Py_None ? new_tensor(PyObject_GetAttr(a[1], s_shape), dtype_object(l.dtype), device) : Py_NewRef(a[10]);
  if (!out) goto end;
  if (a[10] == Py_None) {
    dl = l;
    dl.stride[0] = l.shape[1];
    if (pointer_of(out, &dl)) goto end;
  } else if (read_matrix(out, &dl, "out")) {
    goto end;
  }
  if (dl.dtype != l.dtype || dl.device != l.device || dl.shape[0] != l.shape[0] || dl.shape[1] != l.shape[1]) {
    refuse("out's type, shape or device is not that of the logits");
    goto end;
  }
  {
    route_grad_fn fn = (route_grad_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto end;
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(l.ptr, (mk_dtype)l.dtype, l.shape[0], (int)l.shape[1], l.stride[0], (int)idx.shape[1], normalize, (float)scale,
           (const int *)idx.ptr, (const int *)counts.ptr, (const int *)tokens.ptr, (const float *)g[0].ptr,
           (const float *)g[1].ptr, (const float *)g[2].ptr, dl.ptr, dl.stride[0], st);
    Py_END_ALLOW_THREADS
    result = Py_BuildValue("(iO)", (int)e, out);
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(device);
  return result;
}

/* w4(codes, scales, zeros or None) -> (the bytes of an mk_w4_weight, device) */
static PyObject *bind_w4(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 3, "w4: 3 arguments");
  tensor c, s, z;
  if (read_tensor(a[0], &c, "codes") || read_tensor(a[1], &s, "scales")) return NULL;
  NEED(c.dtype == T_U8 && c.dims == 2 && c.device >= 0, "codes must be a [n x k / 2] uint8 CUDA tensor");
  NEED((c.shape[1] <= 1 || c.stride[1] == 1) && (c.shape[0] <= 1 || c.stride[0] == c.shape[1]), "codes must be contiguous");
  NEED(s.dtype == MK_BF16 || s.dtype == MK_F16, "scales must be bf16 or fp16");
  const long long groups = s.dims == 2 ? s.shape[1] : 0;
  NEED(groups > 0 && 2 * c.shape[1] % groups == 0, "scales must be [n x k / group]");
  const long long group = 2 * c.shape[1] / groups, shape[2] = {c.shape[0], groups};
  NEED(group == 32 || group == 64 || group == 128, "groups must have 32, 64 or 128 weights");
  if (read_plain(a[1], &s, "scales", s.dtype, c.device, 2, shape)) return NULL;
  z.ptr = NULL;
  if (a[2] != Py_None && read_plain(a[2], &z, "zeros", s.dtype, c.device, 2, shape)) return NULL;
  const mk_w4_weight w = {c.ptr, s.ptr, z.ptr, c.shape[0], 2 * c.shape[1], (int)group, s.dtype};
  return Py_BuildValue("(y#i)", (const char *)&w, (Py_ssize_t)sizeof(w), c.device);
}

typedef size_t (*w4_size_fn)(const mk_w4_weight *, long long);
typedef mk_status (*w4_fn)(const void *, long long, const mk_w4_weight *, void *, long long, mk_dtype, mk_dtype, long long,
                           void *, size_t, void *, size_t, const mk_config *, mk_stream_t);
/* w4_gemm(fn, size_fn, get_workspace, x, weight, device, out, fp32, config address, stream, the weight's tensors)
 * -> (status, out) */
static PyObject *bind_w4_gemm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 11, "w4_gemm: 11 arguments");
  tensor x, y, sc, ws;
  mk_stream_t st;
  if (read_matrix(a[3], &x, "x")) return NULL;
  NEED(PyBytes_Check(a[4]) && PyBytes_GET_SIZE(a[4]) == (Py_ssize_t)sizeof(mk_w4_weight), "not a 4-bit weight");
  const mk_w4_weight *w = (const mk_w4_weight *)PyBytes_AS_STRING(a[4]);
  const void *const at[3] = {w->codes, w->scales, w->zeros};
  if (still_there(a[10], at, 3, "4-bit weight")) return NULL;
  const int dev = (int)PyLong_AsLong(a[5]), f32 = PyObject_IsTrue(a[7]);
  void *cfg = a[8] == Py_None ? NULL : PyLong_AsVoidPtr(a[8]);
  if (PyErr_Occurred()) return NULL;
  NEED(x.dtype == w->dtype && x.device == dev, "x does not have the weight's type or device");
  NEED(x.shape[1] == w->k, "x's rows are not as long as the weight's");
  if (check_device(dev) || read_stream(a[9], dev, &st)) return NULL;
  const int odt = f32 ? MK_F32 : x.dtype;
  PyObject *device = PyObject_GetAttr(a[3], s_device), *space = NULL, *status = NULL, *result = NULL;
  PyObject *out = a[6] == Py_None ? new_tensor(Py_BuildValue("(LL)", x.shape[0], w->n), dtype_object(odt), device) : Py_NewRef(a[6]);
  if (!out) goto end;
  if (a[6] == Py_None) {
    y = x;
    y.dtype = odt;
    y.shape[1] = y.stride[0] = w->n;
    if (pointer_of(out, &y)) goto end;
  } else if (read_matrix(out, &y, "out")) {
    goto end;
  }
  if (y.dtype != odt || y.device != dev || y.shape[0] != x.shape[0] || y.shape[1] != w->n) {
    refuse("out's type, shape or device does not fit");
    goto end;
  }
  sc.ptr = ws.ptr = NULL;
  sc.shape[0] = ws.shape[0] = 0;
  {
    const size_t need = ((w4_size_fn)PyLong_AsVoidPtr(a[1]))(w, x.shape[0]);
    if (need > 0) {
      space = scratch(Py_None, need, device, &sc);
      if (!space) goto end;
      status = PyObject_CallFunction(a[2], "i", 256);
      if (!status || read_tensor(status, &ws, "workspace")) goto end;
    }
    w4_fn fn = (w4_fn)PyLong_AsVoidPtr(a[0]);
    if (!fn) goto end;
    mk_status e;
    Py_BEGIN_ALLOW_THREADS
    e = fn(x.ptr, x.stride[0], w, y.ptr, y.stride[0], (mk_dtype)x.dtype, (mk_dtype)odt, x.shape[0], sc.ptr,
           (size_t)sc.shape[0], ws.ptr, (size_t)ws.shape[0], (const mk_config *)cfg, st);
    Py_END_ALLOW_THREADS
    result = Py_BuildValue("(iO)", (int)e, out);
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(space);
  Py_XDECREF(status);
  Py_XDECREF(device);
  return result;
}

/* setup(dtypes in the order of `dtypes`, raw_stream, empty, current_device) */
static PyObject *bind_setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  NEED(n == 4 && PyTuple_Check(a[0]) && PyTuple_GET_SIZE(a[0]) == N_DTYPES, "setup: (9 dtypes, three functions)");
  for (int i = 0; i < N_DTYPES; ++i) Py_XSETREF(dtypes[i], Py_NewRef(PyTuple_GET_ITEM(a[0], i)));
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
                                {"rms_norm", (PyCFunction)(void (*)(void))bind_norm, METH_FASTCALL, NULL},
                                {"rms_norm_backward", (PyCFunction)(void (*)(void))bind_norm_grad, METH_FASTCALL, NULL},
                                {"route", (PyCFunction)(void (*)(void))bind_route, METH_FASTCALL, NULL},
                                {"route_backward", (PyCFunction)(void (*)(void))bind_route_grad, METH_FASTCALL, NULL},
                                {"w4", (PyCFunction)(void (*)(void))bind_w4, METH_FASTCALL, NULL},
                                {"w4_gemm", (PyCFunction)(void (*)(void))bind_w4_gemm, METH_FASTCALL, NULL},
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
