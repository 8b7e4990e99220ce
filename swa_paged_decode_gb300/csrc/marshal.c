/*
 * marshal.c -- the argument marshalling of the cache, shared-prefix and prompt calls
 * as a CPython extension (swa_paged_decode_gb300._marshal): a tensor's own
 * properties (device, dtype, extents, strides), which its pointer cannot
 * carry, are read and checked here, and the library's function is called
 * through its address. Through ctypes and Python these checks took longer
 * than the launch they precede (a cache write 8.5 us of host time, 3 of them
 * the launch). No torch headers: tensors are asked through their Python
 * methods. Every function returns the library's status, or kBadTensor.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "dsa_decode.h"

enum { kBadTensor = -1000, kMaxDims = 3 };

static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr;
/* torch dtypes, and torch's current device and raw stream functions */
static PyObject *t_u8, *t_i32, *t_i64, *t_bf16, *t_f16, *t_f32, *f_device, *f_stream;

typedef struct {
  void *ptr;
  PyObject *dtype; /* borrowed: torch's dtypes live as long as torch */
  long dev;
  Py_ssize_t nd;
  long long shape[kMaxDims], stride[kMaxDims];
} tensor;

static int as_ll(PyObject *o, long long *v) {
  *v = PyLong_AsLongLong(o);
  return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

/* -1: a Python error is set; 1: more dims than any argument has. */
static int get(PyObject *t, tensor *o) {
  PyObject *p = PyObject_GetAttr(t, s_dtype);
  if (!p) return -1;
  o->dtype = p;
  Py_DECREF(p);
  p = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!p) return -1;
  o->dev = PyLong_AsLong(p);
  Py_DECREF(p);
  p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!p) return -1;
  o->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  PyObject *sh = PyObject_GetAttr(t, s_shape), *st = sh ? PyObject_CallMethodNoArgs(t, s_stride) : NULL;
  int rc = -1;
  if (sh && st) {
    if (!PyTuple_Check(sh) || !PyTuple_Check(st) || PyTuple_GET_SIZE(sh) != PyTuple_GET_SIZE(st)) {
      PyErr_SetString(PyExc_TypeError, "not a tensor");
    } else {
      o->nd = PyTuple_GET_SIZE(sh);
      rc = o->nd > kMaxDims ? 1 : 0;
      for (Py_ssize_t i = 0; rc == 0 && i < o->nd; ++i)
        if (as_ll(PyTuple_GET_ITEM(sh, i), &o->shape[i]) || as_ll(PyTuple_GET_ITEM(st, i), &o->stride[i])) rc = -1;
    }
  }
  Py_XDECREF(sh);
  Py_XDECREF(st);
  return PyErr_Occurred() ? -1 : rc;
}

static int contiguous(const tensor *t) {
  long long n = 1;
  for (Py_ssize_t i = t->nd - 1; i >= 0; --i) {
    if (t->shape[i] == 0) return 1;
    if (t->shape[i] != 1 && t->stride[i] != n) return 0;
    n *= t->shape[i];
  }
  return 1;
}

/* One call's state: the current device (asked for with the first tensor that
 * is on one), and whether an argument failed (bad) or a Python error is set
 * (err). */
typedef struct {
  long dev;
  int bad, err;
} call;

/* A number that the library takes as int32; another one is not cut to one. */
static int32_t as_i32(call *c, PyObject *o) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (PyErr_Occurred()) c->err = 1;
  if (over || v < INT32_MIN || v > INT32_MAX) c->bad = 1;
  return c->err || c->bad ? 0 : (int32_t)v;
}

static int read_tensor(call *c, PyObject *o, tensor *t) {
  if (c->bad || c->err) return 0;
  const int rc = get(o, t);
  if (rc < 0) {
    c->err = 1;
    return 0;
  }
  if (rc == 0 && t->dev >= 0 && c->dev < 0) {
    PyObject *p = PyObject_CallNoArgs(f_device);
    if (p) c->dev = PyLong_AsLong(p);
    Py_XDECREF(p);
    if (PyErr_Occurred()) {
      c->err = 1;
      return 0;
    }
  }
  if (rc > 0 || t->dev < 0 || t->dev != c->dev) c->bad = 1;
  return !c->bad;
}

/* A contiguous tensor of this dtype and shape (a negative extent: any); None
 * gives NULL where it may (opt). `n0`: receives the first extent. */
static void *vec(call *c, PyObject *o, int opt, PyObject *dtype, Py_ssize_t nd, long long a, long long b, long long d,
                 long long *n0) {
  tensor t;
  if (o == Py_None) {
    if (!opt) c->bad = 1;
    return NULL;
  }
  if (!read_tensor(c, o, &t)) return NULL;
  const long long want[kMaxDims] = {a, b, d};
  int ok = t.dtype == dtype && t.nd == nd && contiguous(&t);
  for (Py_ssize_t i = 0; ok && i < nd; ++i) ok = want[i] < 0 || t.shape[i] == want[i];
  if (!ok) {
    c->bad = 1;
    return NULL;
  }
  if (n0) *n0 = t.shape[0];
  return t.ptr;
}

static int record_bytes(int32_t fmt) {
  switch (fmt) {
    case DSA_REC_FP8_528: case DSA_REC_FP8_528_UE8M0: return 528;
    case DSA_REC_NVFP4_288: return 288;
    case DSA_REC_MODEL1_584: return 584;
    case DSA_REC_V32_656: return 656;
  }
  return 0; /* the library says what it does not know */
}

static void cache(call *c, PyObject *data, PyObject *page, PyObject *fmt, dsa_cache_desc *d) {
  tensor t;
  const int32_t pg = as_i32(c, page), f = as_i32(c, fmt);
  if (!read_tensor(c, data, &t)) return;
  if (t.dtype != t_u8 || t.nd != 2 || t.stride[1] != 1 || t.shape[1] < (long long)pg * record_bytes(f)) {
    c->bad = 1;
    return;
  }
  d->base = t.ptr;
  d->num_pages = t.shape[0];
  d->page_stride_bytes = t.stride[0];
  d->page_size = pg;
  d->format = f;
}

/* Dense rows [n, dims of the format]. */
static void *rows(call *c, PyObject *o, long long n, const dsa_cache_desc *d, long long *stride, int32_t *type) {
  tensor t;
  const long long dims = d->format == DSA_REC_V32_656 ? 576 : 512;
  if (!read_tensor(c, o, &t)) return NULL;
  *type = t.dtype == t_bf16 ? DSA_TYPE_BF16 : t.dtype == t_f16 ? DSA_TYPE_F16 : t.dtype == t_f32 ? DSA_TYPE_F32 : -1;
  if (*type < 0 || t.nd != 2 || t.shape[0] != n || t.shape[1] != dims || (n > 0 && t.stride[1] != 1)) {
    c->bad = 1;
    return NULL;
  }
  *stride = n > 1 ? t.stride[0] : dims;
  return t.ptr;
}

/* The raw stream given, or the current one of the device. */
static dsa_stream_t stream_of(call *c, PyObject *o) {
  if (c->bad || c->err) return NULL;
  PyObject *p = o;
  if (o == Py_None) {
    PyObject *d = PyLong_FromLong(c->dev);
    p = d ? PyObject_CallOneArg(f_stream, d) : NULL;
    Py_XDECREF(d);
  } else {
    Py_INCREF(p);
  }
  if (!p) {
    c->err = 1;
    return NULL;
  }
  void *s = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  if (PyErr_Occurred()) c->err = 1;
  return (dsa_stream_t)s;
}

static int want_args(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
  return -1;
}

#define DSA_CALL(rc, expr)                             \
  do {                                                 \
    if (c.err) return NULL;                            \
    if (c.bad) return PyLong_FromLong(kBadTensor);     \
    Py_BEGIN_ALLOW_THREADS rc = (expr);                \
    Py_END_ALLOW_THREADS                               \
  } while (0)

typedef dsa_status (*write_fn)(const dsa_cache_desc *, const int32_t *, int64_t, const void *, int64_t, int32_t,
                               const float *, float, const int64_t *, const float *, int64_t, int32_t, int32_t *,
                               dsa_stream_t);
typedef dsa_status (*read_fn)(const dsa_cache_desc *, const int32_t *, int64_t, void *, int64_t, int32_t,
                              dsa_stream_t);
typedef dsa_status (*prefix_fn)(const dsa_prefix_plan_t *, void *, size_t, const void *, int64_t, int64_t,
                                const dsa_cache_desc *, const int32_t *, const int32_t *, const float *,
                                const int64_t *, const float *, int64_t, int32_t, float, const void *, const float *,
                                void *, float *, dsa_stream_t);

typedef dsa_status (*chunk_fn)(const dsa_chunk_plan_t *, void *, size_t, const void *, int64_t, int64_t,
                               const dsa_cache_desc *, const int32_t *, int64_t, const int32_t *, const int32_t *,
                               int32_t, const float *, const int64_t *, const float *, int64_t, int32_t, float,
                               const void *, const float *, void *, float *, dsa_stream_t);

typedef dsa_status (*weights_fn)(const dsa_weights_plan_t *, void *, size_t, const void *, int64_t, int64_t,
                                 const dsa_cache_desc *, const int32_t *, int64_t, const int32_t *, const int32_t *,
                                 int32_t, float, const float *, const float *, const float *, int64_t, float *, int64_t,
                                 dsa_stream_t);
typedef dsa_status (*qk_fn)(int32_t, int32_t, int32_t, int32_t, const void *, int64_t, int64_t, const float *, int64_t,
                            void *, int64_t, int64_t, const void *, int64_t, const float *, const dsa_cache_desc *,
                            const int32_t *, float, const int64_t *, const float *, int64_t, int32_t, int32_t *,
                            dsa_stream_t);
typedef dsa_status (*evict_fn)(int32_t, int32_t, const int32_t *, int64_t, const int32_t *, const float *, int64_t,
                               int32_t, int32_t, int32_t, int32_t *, int64_t, float *, int64_t, int32_t *, int32_t *,
                               int64_t, int32_t *, dsa_stream_t);

/* (address, data, page_size, fmt, slots, rows, norm_weight, norm_eps,
 *  positions, cos_sin, rope_style, device_status, stream) */
static PyObject *cache_write(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  dsa_cache_desc d = {0};
  long long n = 0, stride = 0, table = 0;
  int32_t type = 0;
  dsa_status rc;
  if (want_args(na, 13)) return NULL;
  write_fn f = (write_fn)PyLong_AsVoidPtr(a[0]);
  const float eps = (float)PyFloat_AsDouble(a[7]);
  const int32_t style = as_i32(&c, a[10]);
  if (PyErr_Occurred()) return NULL;
  cache(&c, a[1], a[2], a[3], &d);
  const int32_t *slots = vec(&c, a[4], 0, t_i32, 1, -1, -1, -1, &n);
  void *r = rows(&c, a[5], n, &d, &stride, &type);
  const float *w = vec(&c, a[6], 1, t_f32, 1, 512, -1, -1, NULL);
  const int64_t *pos = vec(&c, a[8], 1, t_i64, 1, n, -1, -1, NULL);
  const float *cs = vec(&c, a[9], 1, t_f32, 2, -1, 64, -1, &table);
  int32_t *status = vec(&c, a[11], 1, t_i32, 1, 1, -1, -1, NULL);
  dsa_stream_t st = stream_of(&c, a[12]);
  DSA_CALL(rc, f(&d, slots, n, r, stride, type, w, eps, pos, cs, table, style, status, st));
  return PyLong_FromLong(rc);
}

/* (address, data, page_size, fmt, slots, rows, stream) */
static PyObject *cache_read(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  dsa_cache_desc d = {0};
  long long n = 0, stride = 0;
  int32_t type = 0;
  dsa_status rc;
  if (want_args(na, 7)) return NULL;
  read_fn f = (read_fn)PyLong_AsVoidPtr(a[0]);
  if (PyErr_Occurred()) return NULL;
  cache(&c, a[1], a[2], a[3], &d);
  const int32_t *slots = vec(&c, a[4], 0, t_i32, 1, -1, -1, -1, &n);
  void *r = rows(&c, a[5], n, &d, &stride, &type);
  dsa_stream_t st = stream_of(&c, a[6]);
  DSA_CALL(rc, f(&d, slots, n, r, stride, type, st));
  return PyLong_FromLong(rc);
}

/* (address, plan address, workspace, q, data, page_size, fmt, slots, length,
 *  sink, positions, cos_sin, rope_style, scale, tail_out, tail_lse, out, lse,
 *  stream) */
static PyObject *prefix_run(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  dsa_cache_desc d = {0};
  long long ws_bytes = 0, table = 0;
  tensor q = {0};
  dsa_status rc;
  if (want_args(na, 19)) return NULL;
  prefix_fn f = (prefix_fn)PyLong_AsVoidPtr(a[0]);
  const dsa_prefix_plan_t *plan = PyLong_AsVoidPtr(a[1]);
  const int32_t style = as_i32(&c, a[12]);
  const float scale = (float)PyFloat_AsDouble(a[13]);
  if (PyErr_Occurred()) return NULL;
  const long long T = plan->num_tokens, H = plan->num_heads, D = plan->d_qk;
  void *ws = vec(&c, a[2], 0, t_u8, 1, -1, -1, -1, &ws_bytes);
  if (read_tensor(&c, a[3], &q) &&
      (q.dtype != t_bf16 || q.nd != 3 || q.shape[0] != T || q.shape[1] != H || q.shape[2] != D ||
       (T > 0 && q.stride[2] != 1)))
    c.bad = 1;
  cache(&c, a[4], a[5], a[6], &d);
  const int32_t *slots = vec(&c, a[7], 0, t_i32, 1, plan->width, -1, -1, NULL);
  const int32_t *length = vec(&c, a[8], 0, t_i32, 1, 1, -1, -1, NULL);
  const float *sink = vec(&c, a[9], 1, t_f32, 1, H, -1, -1, NULL);
  const int64_t *pos = vec(&c, a[10], 1, t_i64, 1, T, -1, -1, NULL);
  const float *cs = vec(&c, a[11], 1, t_f32, 2, -1, 64, -1, &table);
  const void *tail = vec(&c, a[14], 1, t_bf16, 3, T, H, 512, NULL);
  const float *tail_lse = vec(&c, a[15], 1, t_f32, 2, T, H, -1, NULL);
  void *out = vec(&c, a[16], 0, t_bf16, 3, T, H, 512, NULL);
  float *lse = vec(&c, a[17], 0, t_f32, 2, T, H, -1, NULL);
  dsa_stream_t st = stream_of(&c, a[18]);
  const long long sh = H > 1 ? q.stride[1] : D, sq = T > 1 ? q.stride[0] : H * sh;
  DSA_CALL(rc, f(plan, ws, (size_t)ws_bytes, q.ptr, sq, sh, &d, slots, length, sink, pos, cs, table, style,
                 scale, tail, tail_lse, out, lse, st));
  return PyLong_FromLong(rc);
}

/* read_tensor, None being no tensor. */
static int given(call *c, PyObject *o, tensor *t) {
  if (o == Py_None) c->bad = 1;
  return read_tensor(c, o, t);
}

/* Queries [T, H, D] of a dtype, any token and head strides. */
static void *queries(call *c, PyObject *o, PyObject *dtype, long long T, long long H, long long D, long long *st,
                     long long *sh) {
  tensor t;
  if (!given(c, o, &t)) return NULL;
  if ((dtype && t.dtype != dtype) || t.nd != 3 || t.shape[0] != T || t.shape[1] != H || t.shape[2] != D ||
      (T > 0 && t.stride[2] != 1)) {
    c->bad = 1;
    return NULL;
  }
  *sh = H > 1 ? t.stride[1] : D;
  *st = T > 1 ? t.stride[0] : H * *sh;
  return t.ptr;
}

/* Lists [B, width] of a dtype (`exact`: else of width or more), any list
 * stride. */
static void *lists_of(call *c, PyObject *o, PyObject *dtype, long long B, long long width, int exact, long long *stride) {
  tensor t;
  if (!given(c, o, &t)) return NULL;
  if (t.dtype != dtype || t.nd != 2 || t.shape[0] != B || (exact ? t.shape[1] != width : t.shape[1] < width) ||
      (B > 0 && t.shape[1] > 1 && t.stride[1] != 1)) {
    c->bad = 1;
    return NULL;
  }
  *stride = B > 1 ? t.stride[0] : t.shape[1];
  return t.ptr;
}
static void *lists(call *c, PyObject *o, PyObject *dtype, long long B, long long width, long long *stride) {
  return lists_of(c, o, dtype, B, width, 1, stride);
}

/* (address, plan address, workspace, q, data, page_size, fmt, slots, lengths,
 *  starts, window, sink, positions, cos_sin, rope_style, scale, tail_out,
 *  tail_lse, out, lse, stream) */
static PyObject *chunk_run(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  dsa_cache_desc d = {0};
  long long ws_bytes = 0, table = 0, st = 0, sh = 0, ls = 0;
  dsa_status rc;
  if (want_args(na, 21)) return NULL;
  chunk_fn f = (chunk_fn)PyLong_AsVoidPtr(a[0]);
  const dsa_chunk_plan_t *plan = PyLong_AsVoidPtr(a[1]);
  const int32_t window = as_i32(&c, a[10]), style = as_i32(&c, a[14]);
  const float scale = (float)PyFloat_AsDouble(a[15]);
  if (PyErr_Occurred()) return NULL;
  const long long T = plan->num_tokens, B = plan->num_seqs, H = plan->num_heads;
  void *ws = vec(&c, a[2], 0, t_u8, 1, -1, -1, -1, &ws_bytes);
  const void *q = queries(&c, a[3], t_bf16, T, H, plan->d_qk, &st, &sh);
  cache(&c, a[4], a[5], a[6], &d);
  const int32_t *slots = lists(&c, a[7], t_i32, B, plan->width, &ls);
  const int32_t *lengths = vec(&c, a[8], 0, t_i32, 1, B, -1, -1, NULL);
  const int32_t *starts = vec(&c, a[9], 0, t_i32, 1, B + 1, -1, -1, NULL);
  const float *sink = vec(&c, a[11], 1, t_f32, 1, H, -1, -1, NULL);
  const int64_t *pos = vec(&c, a[12], 1, t_i64, 1, T, -1, -1, NULL);
  const float *cs = vec(&c, a[13], 1, t_f32, 2, -1, 64, -1, &table);
  const void *tail = vec(&c, a[16], 1, t_bf16, 3, T, H, 512, NULL);
  const float *tail_lse = vec(&c, a[17], 1, t_f32, 2, T, H, -1, NULL);
  void *out = vec(&c, a[18], 0, t_bf16, 3, T, H, 512, NULL);
  float *lse = vec(&c, a[19], 0, t_f32, 2, T, H, -1, NULL);
  dsa_stream_t stream = stream_of(&c, a[20]);
  DSA_CALL(rc, f(plan, ws, (size_t)ws_bytes, q, st, sh, &d, slots, ls, lengths, starts, window, sink, pos, cs, table,
                 style, scale, tail, tail_lse, out, lse, stream));
  return PyLong_FromLong(rc);
}

/* (address, plan address, workspace, q, data, page_size, fmt, slots, lengths,
 *  starts, window, scale, sink, lse, scores_in, scores_out, stream) */
static PyObject *weights_run(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  dsa_cache_desc d = {0};
  long long ws_bytes = 0, st = 0, sh = 0, ls = 0, is = 0, os = 0;
  dsa_status rc;
  if (want_args(na, 17)) return NULL;
  weights_fn f = (weights_fn)PyLong_AsVoidPtr(a[0]);
  const dsa_weights_plan_t *plan = PyLong_AsVoidPtr(a[1]);
  const int32_t window = as_i32(&c, a[10]);
  const float scale = (float)PyFloat_AsDouble(a[11]);
  if (PyErr_Occurred()) return NULL;
  const long long T = plan->num_tokens, B = plan->num_seqs, H = plan->num_heads, width = plan->width;
  void *ws = vec(&c, a[2], 0, t_u8, 1, -1, -1, -1, &ws_bytes);
  const void *q = queries(&c, a[3], t_bf16, T, H, plan->d_qk, &st, &sh);
  cache(&c, a[4], a[5], a[6], &d);
  const int32_t *slots = lists(&c, a[7], t_i32, B, width, &ls);
  const int32_t *lengths = vec(&c, a[8], 0, t_i32, 1, B, -1, -1, NULL);
  const int32_t *starts = vec(&c, a[9], 0, t_i32, 1, B + 1, -1, -1, NULL);
  const float *sink = vec(&c, a[12], 1, t_f32, 1, H, -1, -1, NULL);
  const float *lse = vec(&c, a[13], 0, t_f32, 2, T, H, -1, NULL);
  const float *in = a[14] == Py_None ? NULL : lists(&c, a[14], t_f32, B, width, &is);
  float *out = lists(&c, a[15], t_f32, B, width, &os);
  dsa_stream_t stream = stream_of(&c, a[16]);
  DSA_CALL(rc, f(plan, ws, (size_t)ws_bytes, q, st, sh, &d, slots, ls, lengths, starts, window, scale, sink, lse, in, is,
                 out, os, stream));
  return PyLong_FromLong(rc);
}

/* (address, q, out, q_weight, keys, key_weight, data, page_size, fmt, slots,
 *  eps, positions, cos_sin, rope_style, device_status, stream); data None: no
 *  keys */
static PyObject *qk_norm(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  dsa_cache_desc d = {0};
  tensor q, w;
  long long st = 0, sh = 0, ot = 0, oh = 0, wh = 0, ks = 0, table = 0, T = 0, H = 0, D = 0;
  int32_t type = -1, ktype = -1;
  dsa_status rc;
  if (want_args(na, 16)) return NULL;
  qk_fn f = (qk_fn)PyLong_AsVoidPtr(a[0]);
  const float eps = (float)PyFloat_AsDouble(a[10]);
  const int32_t style = as_i32(&c, a[13]);
  if (PyErr_Occurred()) return NULL;
  const int with_keys = a[6] != Py_None;
  void *out = NULL, *k = NULL;
  const float *qw = NULL, *kw = NULL;
  const int32_t *slots = NULL;
  if (given(&c, a[1], &q)) {
    type = q.dtype == t_bf16 ? DSA_TYPE_BF16 : q.dtype == t_f16 ? DSA_TYPE_F16 : q.dtype == t_f32 ? DSA_TYPE_F32 : -1;
    if (type < 0 || q.nd != 3 || q.shape[0] > INT32_MAX || q.shape[1] > INT32_MAX || (q.shape[2] != 512 && q.shape[2] != 576) ||
        (q.shape[0] > 0 && q.stride[2] != 1)) {
      c.bad = 1;
    } else {
      T = q.shape[0];
      H = q.shape[1];
      D = q.shape[2];
      sh = H > 1 ? q.stride[1] : D;
      st = T > 1 ? q.stride[0] : H * sh;
    }
  }
  if (!c.bad && !c.err) out = queries(&c, a[2], t_bf16, T, H, D, &ot, &oh);
  if (a[3] != Py_None && read_tensor(&c, a[3], &w)) { /* [512], or [H, 512] */
    if (w.dtype != t_f32 || w.nd < 1 || w.nd > 2 || w.shape[w.nd - 1] != 512 || w.stride[w.nd - 1] != 1 ||
        (w.nd == 2 && w.shape[0] != H)) {
      c.bad = 1;
    } else {
      qw = w.ptr;
      wh = w.nd == 2 ? (H > 1 ? w.stride[0] : 512) : 0;
    }
  }
  if (with_keys) {
    cache(&c, a[6], a[7], a[8], &d);
    slots = vec(&c, a[9], 0, t_i32, 1, T, -1, -1, NULL);
    if (a[4] == Py_None) c.bad = 1;
    k = rows(&c, a[4], T, &d, &ks, &ktype);
    kw = vec(&c, a[5], 1, t_f32, 1, 512, -1, -1, NULL);
    if (!c.bad && (ktype != type || (d.format == DSA_REC_V32_656) != (D == 576))) c.bad = 1;
  } else if (a[4] != Py_None || a[5] != Py_None || a[9] != Py_None) {
    c.bad = 1;
  }
  const int64_t *pos = vec(&c, a[11], 1, t_i64, 1, T, -1, -1, NULL);
  const float *cs = vec(&c, a[12], 1, t_f32, 2, -1, 64, -1, &table);
  int32_t *status = vec(&c, a[14], 1, t_i32, 1, 1, -1, -1, NULL);
  dsa_stream_t stream = stream_of(&c, a[15]);
  DSA_CALL(rc, f((int32_t)T, (int32_t)H, (int32_t)D, type, q.ptr, st, sh, qw, wh, out, ot, oh, k, ks, kw,
                 with_keys ? &d : NULL, slots, eps, pos, cs, table, style, status, stream));
  return PyLong_FromLong(rc);
}

/* (address, slots, lengths, scores, budget, keep_first, keep_last, kept_slots,
 *  kept_scores, kept_lengths, freed, freed_counts, stream) */
static PyObject *evict(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  call c = {-1, 0, 0};
  tensor t;
  long long B = 0, width = 0, s1 = 0, s2 = 0, s3 = 0, s4 = 0, s5 = 0;
  dsa_status rc;
  if (want_args(na, 13)) return NULL;
  evict_fn f = (evict_fn)PyLong_AsVoidPtr(a[0]);
  const int32_t budget = as_i32(&c, a[4]), first = as_i32(&c, a[5]), last = as_i32(&c, a[6]);
  if (PyErr_Occurred()) return NULL;
  if (given(&c, a[1], &t)) {
    if (t.nd != 2 || t.shape[0] > INT32_MAX || t.shape[1] > INT32_MAX) c.bad = 1;
    else B = t.shape[0], width = t.shape[1];
  }
  const long long most = budget < width ? budget : width;
  const int32_t *slots = lists(&c, a[1], t_i32, B, width, &s1);
  const int32_t *lengths = vec(&c, a[2], 0, t_i32, 1, B, -1, -1, NULL);
  const float *scores = lists(&c, a[3], t_f32, B, width, &s2);
  int32_t *kept = lists_of(&c, a[7], t_i32, B, most, 0, &s3);
  float *kept_scores = lists_of(&c, a[8], t_f32, B, most, 0, &s4);
  int32_t *kept_lengths = vec(&c, a[9], 0, t_i32, 1, B, -1, -1, NULL), *freed = NULL, *counts = NULL;
  if (a[10] != Py_None || a[11] != Py_None) {
    freed = lists_of(&c, a[10], t_i32, B, width - most, 0, &s5);
    counts = vec(&c, a[11], 0, t_i32, 1, B, -1, -1, NULL);
  }
  dsa_stream_t stream = stream_of(&c, a[12]);
  DSA_CALL(rc, f((int32_t)B, (int32_t)width, slots, s1, lengths, scores, s2, budget, first, last, kept, s3, kept_scores,
                 s4, kept_lengths, freed, s5, counts, stream));
  return PyLong_FromLong(rc);
}

/* setup(uint8, int32, int64, bfloat16, float16, float32, current device, raw stream) */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  PyObject **to[8] = {&t_u8, &t_i32, &t_i64, &t_bf16, &t_f16, &t_f32, &f_device, &f_stream};
  if (want_args(na, 8)) return NULL;
  for (int i = 0; i < 8; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*to[i], a[i]);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {"cache_write", (PyCFunction)(void (*)(void))cache_write, METH_FASTCALL, NULL},
    {"cache_read", (PyCFunction)(void (*)(void))cache_read, METH_FASTCALL, NULL},
    {"prefix_run", (PyCFunction)(void (*)(void))prefix_run, METH_FASTCALL, NULL},
    {"chunk_run", (PyCFunction)(void (*)(void))chunk_run, METH_FASTCALL, NULL},
    {"weights_run", (PyCFunction)(void (*)(void))weights_run, METH_FASTCALL, NULL},
    {"qk_norm", (PyCFunction)(void (*)(void))qk_norm, METH_FASTCALL, NULL},
    {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_shape || !s_stride || !s_get_device || !s_data_ptr) return NULL;
  PyObject *m = PyModule_Create(&module);
  if (m) PyModule_AddIntConstant(m, "BAD_TENSOR", kBadTensor);
  return m;
}
