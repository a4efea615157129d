/*
 * binding.c -- CPython side of the calls whose kernels take a few
 * microseconds: pkv_append_rope, pkv_append_rope_fp8, pkv_decode_attn_fp8,
 * pkv_decode_append_attn_fp8, pkv_expand_fp8, pkv_tree_attn, pkv_tree_attn_fp8,
 * pkv_keep_nodes and pkv_copy_pages. It reads the torch tensors' attributes, checks them and makes
 * the C call. Written against the CPython API alone (no torch headers): a
 * tensor is asked for its dtype, device, strides and address like any object.
 * In Python, with ctypes, the same checks and call take 8.7 us
 * (decode_attn_fp8) and 12.4 us (append_rope_fp8) of host time on a Grace core,
 * longer than the kernels of a decode step; the launch itself is 2.4 us of it.
 *
 * Each function returns the C call's status; refusals that a tensor's own
 * attributes show raise TypeError or ValueError, and nothing is launched.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "pkv.h"

/* Attribute names and torch objects, looked up once. */
static PyObject *s_dtype, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_shape, *s_stride, *s_tensor, *s_cuda_stream,
    *s_device, *s_index;
static PyObject *t_bf16, *t_i32, *t_i64, *t_f32, *t_e4m3, *t_e8m0;
static PyObject *f_raw_stream, *f_get_device, *f_exchange_device;

typedef struct {
  void* ptr;
  int nd;
  long long shape[5];
} Tensor;

static long as_long(PyObject* o) { /* steals o; -1 with an exception set on failure */
  if (o == NULL) return -1;
  const long v = PyLong_AsLong(o);
  Py_DECREF(o);
  return v;
}

/* Up to 5 entries of a tuple of ints (a shape or strides); *nd is its length. Steals `t`. */
static int read_ints(PyObject* t, const char* name, int* nd, long long* v) {
  if (t == NULL) return -1;
  if (!PyTuple_Check(t)) {
    Py_DECREF(t);
    PyErr_Format(PyExc_TypeError, "%s is not a tensor", name);
    return -1;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(t);
  *nd = (int)n;
  for (Py_ssize_t i = 0; i < n && i < 5; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (v[i] == -1 && PyErr_Occurred()) {
      Py_DECREF(t);
      return -1;
    }
  }
  Py_DECREF(t);
  return 0;
}

static int read_ptr(PyObject* t, void** ptr) {
  PyObject* o = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (o == NULL) return -1;
  *ptr = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return *ptr == NULL && PyErr_Occurred() ? -1 : 0;
}

/* Type and device of `t`; *dev < 0: any CUDA device, and *dev becomes its index. */
static int check_place(PyObject* t, const char* name, PyObject* dtype, long* dev) {
  if (t == NULL || t == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s is required", name);
    return -1;
  }
  PyObject* have = PyObject_GetAttr(t, s_dtype);
  if (have == NULL) return -1;
  const int same = have == dtype;
  if (!same) PyErr_Format(PyExc_TypeError, "%s: expected %S, got %S", name, dtype, have);
  Py_DECREF(have);
  if (!same) return -1;
  const long d = as_long(PyObject_CallMethodNoArgs(t, s_get_device));
  if (d == -1 && PyErr_Occurred()) return -1;
  if (d < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor (the library has no CPU path)", name);
    return -1;
  }
  if (*dev < 0) *dev = d;
  if (d != *dev) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, expected cuda:%ld", name, d, *dev);
    return -1;
  }
  return 0;
}

/* A contiguous tensor of `nd` dimensions (nd < 0: any number). */
static int get_tensor(PyObject* t, const char* name, PyObject* dtype, long* dev, int nd, Tensor* out) {
  if (check_place(t, name, dtype, dev) != 0) return -1;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (c == NULL) return -1;
  Py_DECREF(c);
  if (c != Py_True) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return -1;
  }
  if (read_ints(PyObject_GetAttr(t, s_shape), name, &out->nd, out->shape) != 0) return -1;
  if (nd >= 0 && out->nd != nd) {
    PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, got %d", name, nd, out->nd);
    return -1;
  }
  return read_ptr(t, &out->ptr);
}

/* Rows of the new tokens, [n, heads, d] with a token's rows contiguous and tokens any distance apart (*stride). */
static int get_rows(PyObject* t, const char* name, long* dev, long long n, long long heads, long long d, Tensor* out,
                    long long* stride) {
  if (check_place(t, name, t_bf16, dev) != 0) return -1;
  long long st[5];
  int nd;
  if (read_ints(PyObject_GetAttr(t, s_shape), name, &out->nd, out->shape) != 0) return -1;
  if (out->nd != 3 || out->shape[0] != n || out->shape[1] != heads || out->shape[2] != d) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, n, heads, d);
    return -1;
  }
  if (read_ints(PyObject_CallMethodNoArgs(t, s_stride), name, &nd, st) != 0) return -1;
  if (st[2] != 1 || (st[1] != d && heads > 1)) {
    PyErr_Format(PyExc_ValueError, "%s: the rows of a token must be contiguous", name);
    return -1;
  }
  *stride = st[0];
  return read_ptr(t, &out->ptr);
}

static int same_shape(const Tensor* a, const Tensor* b) {
  if (a->nd != b->nd) return 0;
  for (int i = 0; i < a->nd && i < 5; ++i)
    if (a->shape[i] != b->shape[i]) return 0;
  return 1;
}

static long long numel(const Tensor* t) {
  long long n = 1;
  for (int i = 0; i < t->nd && i < 4; ++i) n *= t->shape[i];
  return t->nd > 4 ? -1 : n;
}

static int bad_shape(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  return -1;
}

/* sizes that a C call takes as int32 */
static int fits_i32(long long a, long long b, long long c) {
  const long long top = 0x7fffffffLL;
  if (a <= top && b <= top && c <= top) return 0;
  PyErr_SetString(PyExc_ValueError, "a size is beyond 2^31 - 1");
  return -1;
}

static const char kPools[] = "pools are [num_pages, num_kv_heads, page_size, head_dim]";

/* The pools of a bf16 cache (scales NULL) or an 8-bit one: their device and descriptor. */
static int get_cache(PyObject* k, PyObject* v, PyObject* scales, long* dev, Tensor* tk, Tensor* tv, Tensor* ts,
                     pkv_cache_desc* d) {
  PyObject* dtype = scales == NULL ? t_bf16 : t_e4m3;
  if (get_tensor(k, "k_pages", dtype, dev, 4, tk) != 0 || get_tensor(v, "v_pages", dtype, dev, 4, tv) != 0) return -1;
  if (!same_shape(tk, tv)) return bad_shape(kPools);
  if (fits_i32(tk->shape[0], tk->shape[1], tk->shape[2]) != 0 || fits_i32(tk->shape[3], 0, 0) != 0) return -1;
  ts->ptr = NULL;
  if (scales != NULL) {
    if (get_tensor(scales, "kv_scales", t_e8m0, dev, 4, ts) != 0) return -1;
    if (ts->shape[0] != tk->shape[0] || ts->shape[1] != tk->shape[1] || ts->shape[2] != 2 || ts->shape[3] != tk->shape[2])
      return bad_shape("kv_scales must be [num_pages, num_kv_heads, 2, page_size] of the pools' sizes");
  }
  d->num_pages = (int32_t)tk->shape[0];
  d->num_kv_heads = (int32_t)tk->shape[1];
  d->page_size = (int32_t)tk->shape[2];
  d->head_dim = (int32_t)tk->shape[3];
  d->num_q_heads = d->num_kv_heads;
  return 0;
}

/* A Workspace's tensor (its first dimension is its size in bytes), or none. */
static int get_workspace(PyObject* w, long dev, void** ptr, size_t* bytes) {
  *ptr = NULL;
  *bytes = 0;
  if (w == Py_None) return 0;
  PyObject* t = PyObject_GetAttr(w, s_tensor);
  if (t == NULL) return -1;
  int rc = -1;
  Tensor s;
  const long d = as_long(PyObject_CallMethodNoArgs(t, s_get_device));
  if (d == -1 && PyErr_Occurred()) goto done;
  if (d != dev) {
    PyErr_Format(PyExc_ValueError, "the workspace is on device %ld, expected cuda:%ld", d, dev);
    goto done;
  }
  if (read_ints(PyObject_GetAttr(t, s_shape), "workspace", &s.nd, s.shape) != 0) goto done;
  *bytes = (size_t)numel(&s);
  rc = read_ptr(t, ptr);
done:
  Py_DECREF(t);
  return rc;
}

/* The stream to use on `dev`: `stream`, or the device's current one. */
static int get_stream(PyObject* stream, long dev, pkv_stream_t* out) {
  PyObject* o;
  if (stream == Py_None) {
    PyObject* i = PyLong_FromLong(dev);
    if (i == NULL) return -1;
    o = PyObject_CallOneArg(f_raw_stream, i);
    Py_DECREF(i);
  } else {
    PyObject* d = PyObject_GetAttr(stream, s_device);
    if (d == NULL) return -1;
    const long i = as_long(PyObject_GetAttr(d, s_index));
    Py_DECREF(d);
    if (i == -1 && PyErr_Occurred()) return -1;
    if (i != dev) {
      PyErr_Format(PyExc_ValueError, "the stream is on cuda:%ld, the tensors are on cuda:%ld", i, dev);
      return -1;
    }
    o = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (o == NULL) return -1;
  *out = (pkv_stream_t)PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* Make `dev` current; *back is the device to return to, -1 if it was current already. */
static int enter_device(long dev, long* back) {
  *back = -1;
  const long now = as_long(PyObject_CallNoArgs(f_get_device));
  if (now == -1 && PyErr_Occurred()) return -1;
  if (now == dev) return 0;
  PyObject* i = PyLong_FromLong(dev);
  if (i == NULL) return -1;
  *back = as_long(PyObject_CallOneArg(f_exchange_device, i));
  Py_DECREF(i);
  return *back == -1 && PyErr_Occurred() ? -1 : 0;
}

static PyObject* leave_device(long back, int rc) {
  if (back >= 0) {
    PyObject* i = PyLong_FromLong(back);
    PyObject* o = i == NULL ? NULL : PyObject_CallOneArg(f_exchange_device, i);
    Py_XDECREF(i);
    if (o == NULL) return NULL;
    Py_DECREF(o);
  }
  return PyLong_FromLong(rc);
}

static int count_args(const char* name, Py_ssize_t have, Py_ssize_t want) {
  if (have == want) return 0;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, have);
  return -1;
}

/* A table [max_pos, hd] or None: its pointer and rows. */
static int get_table(PyObject* t, long* dev, long long hd, void** ptr, long long* max_pos) {
  *ptr = NULL;
  *max_pos = 0;
  if (t == Py_None) return 0;
  Tensor table;
  if (get_tensor(t, "cos_sin", t_f32, dev, 2, &table) != 0) return -1;
  if (table.shape[1] != hd || table.shape[0] < 1) return bad_shape("cos_sin must be [max_pos, head_dim], not empty");
  *ptr = table.ptr;
  *max_pos = table.shape[0];
  return fits_i32(*max_pos, 0, 0);
}

/* Norm weights [hd] or None. */
static int get_weight(PyObject* t, const char* name, long* dev, long long hd, void** ptr) {
  *ptr = NULL;
  if (t == Py_None) return 0;
  Tensor w;
  if (get_tensor(t, name, t_bf16, dev, 1, &w) != 0) return -1;
  if (w.shape[0] != hd) {
    PyErr_Format(PyExc_ValueError, "%s must be [head_dim]", name);
    return -1;
  }
  *ptr = w.ptr;
  return 0;
}

/* (k_new, v_new, positions, slot_mapping, cos_sin, k_pages, v_pages, kv_scales or None, workspace, q, q_out, q_weight,
 * k_weight, eps, stream); an 8-bit append where fp8 */
static PyObject* append_any(PyObject* const* a, Py_ssize_t n_args, int fp8) {
  if (count_args("append_rope", n_args, 15) != 0) return NULL;
  long dev = -1, back;
  Tensor kp, vp, sc, slots, k, v, q, q_out, pos;
  pkv_cache_desc d;
  if (get_cache(a[5], a[6], fp8 ? a[7] : NULL, &dev, &kp, &vp, &sc, &d) != 0) return NULL;
  if (get_tensor(a[3], "slot_mapping", t_i32, &dev, -1, &slots) != 0) return NULL;
  const long long n = numel(&slots), hd = d.head_dim;
  long long ks, vs, qs = 0;
  if (n < 0 || fits_i32(n, 0, 0) != 0) return n < 0 ? (bad_shape("slot_mapping must be [n]"), NULL) : NULL;
  if (get_rows(a[0], "k_new", &dev, n, d.num_kv_heads, hd, &k, &ks) != 0) return NULL;
  if (get_rows(a[1], "v_new", &dev, n, d.num_kv_heads, hd, &v, &vs) != 0) return NULL;
  q.ptr = q_out.ptr = NULL;
  if (a[9] != Py_None) {
    if (a[10] == Py_None) return bad_shape("q and q_out come together"), NULL;
    if (get_tensor(a[10], "q_out", t_bf16, &dev, 3, &q_out) != 0) return NULL;
    if (fits_i32(q_out.shape[1], 0, 0) != 0) return NULL;
    if (get_rows(a[9], "q", &dev, n, q_out.shape[1], hd, &q, &qs) != 0) return NULL;
    if (!same_shape(&q, &q_out)) return bad_shape("q_out must have q's shape"), NULL;
    if (q.ptr == q_out.ptr && n > 1 && qs != q_out.shape[1] * hd)
      return bad_shape("q_out may be q itself only where q is contiguous"), NULL;
    d.num_q_heads = (int32_t)q_out.shape[1];
  } else if (a[10] != Py_None || a[11] != Py_None) {
    return bad_shape("q_out and q_weight come with q"), NULL;
  }
  void *table, *qw, *kw;
  long long max_pos;
  if (get_table(a[4], &dev, hd, &table, &max_pos) != 0) return NULL;
  pos.ptr = NULL;
  if (table != NULL) {
    if (get_tensor(a[2], "positions", t_i32, &dev, -1, &pos) != 0) return NULL;
    if (numel(&pos) != n) return bad_shape("positions and slot_mapping differ in length"), NULL;
  }
  if (get_weight(a[11], "q_weight", &dev, hd, &qw) != 0 || get_weight(a[12], "k_weight", &dev, hd, &kw) != 0) return NULL;
  const double eps = PyFloat_AsDouble(a[13]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  void* ws;
  size_t ws_bytes;
  pkv_stream_t stream;
  if (get_workspace(a[8], dev, &ws, &ws_bytes) != 0 || get_stream(a[14], dev, &stream) != 0) return NULL;
  if (enter_device(dev, &back) != 0) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fp8 ? pkv_append_rope_fp8(q.ptr, qs, k.ptr, ks, v.ptr, vs, pos.ptr, slots.ptr, (int32_t)n, table,
                                 (int32_t)max_pos, qw, kw, (float)eps, q_out.ptr, kp.ptr, vp.ptr, sc.ptr,
                                 &d, stream, ws, ws_bytes)
           : pkv_append_rope(q.ptr, qs, k.ptr, ks, v.ptr, vs, pos.ptr, slots.ptr, (int32_t)n, table,
                             (int32_t)max_pos, qw, kw, (float)eps, q_out.ptr, kp.ptr, vp.ptr, &d, stream,
                             ws, ws_bytes);
  Py_END_ALLOW_THREADS;
  return leave_device(back, rc);
}

static PyObject* append_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return append_any(a, n, 0);
}

static PyObject* append_rope_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return append_any(a, n, 1);
}

/* What a decode call takes besides its cache: q, out, block table and lengths, checked against each other. */
static int get_step(PyObject* q, PyObject* out, PyObject* table, PyObject* lens, long* dev, pkv_cache_desc* d, Tensor* tq,
                    Tensor* to, Tensor* bt, Tensor* sl) {
  if (get_tensor(q, "q", t_bf16, dev, 3, tq) != 0 || get_tensor(out, "out", t_bf16, dev, 3, to) != 0 ||
      get_tensor(table, "block_table", t_i32, dev, 2, bt) != 0 || get_tensor(lens, "seq_lens", t_i32, dev, -1, sl) != 0)
    return -1;
  if (tq->shape[2] != d->head_dim || !same_shape(tq, to) || bt->shape[0] != tq->shape[0] || numel(sl) != tq->shape[0])
    return bad_shape("shape mismatch");
  if (fits_i32(tq->shape[0], tq->shape[1], bt->shape[1]) != 0) return -1;
  d->num_q_heads = (int32_t)tq->shape[1];
  return 0;
}

static int get_flags(PyObject* o, uint32_t* flags) {
  const unsigned long f = PyLong_AsUnsignedLong(o);
  if (f == (unsigned long)-1 && PyErr_Occurred()) return -1;
  *flags = (uint32_t)f;
  return 0;
}

/* (q, k_pages, v_pages, kv_scales, block_table, seq_lens, out, scale, workspace, stream, flags) */
static PyObject* decode_attn_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (count_args("decode_attn_fp8", n_args, 11) != 0) return NULL;
  long dev = -1, back;
  Tensor kp, vp, sc, q, bt, sl, out;
  pkv_cache_desc d;
  uint32_t flags;
  if (get_cache(a[1], a[2], a[3], &dev, &kp, &vp, &sc, &d) != 0) return NULL;
  if (get_step(a[0], a[6], a[4], a[5], &dev, &d, &q, &out, &bt, &sl) != 0) return NULL;
  const double scale = PyFloat_AsDouble(a[7]);
  if ((scale == -1.0 && PyErr_Occurred()) || get_flags(a[10], &flags) != 0) return NULL;
  void* ws;
  size_t ws_bytes;
  pkv_stream_t stream;
  if (get_workspace(a[8], dev, &ws, &ws_bytes) != 0 || get_stream(a[9], dev, &stream) != 0) return NULL;
  if (enter_device(dev, &back) != 0) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pkv_decode_attn_fp8(q.ptr, kp.ptr, vp.ptr, sc.ptr, bt.ptr, sl.ptr, out.ptr, (float)scale, stream, &d,
                           (int32_t)q.shape[0], (int32_t)bt.shape[1], ws, ws_bytes, flags);
  Py_END_ALLOW_THREADS;
  return leave_device(back, rc);
}

/* (q, k_new, v_new, k_pages, v_pages, kv_scales, block_table, seq_lens, cos_sin, out, scale, workspace, q_weight,
 * k_weight, eps, stream, flags) */
static PyObject* decode_append_attn_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (count_args("decode_append_attn_fp8", n_args, 17) != 0) return NULL;
  long dev = -1, back;
  Tensor kp, vp, sc, q, k, v, bt, sl, out;
  pkv_cache_desc d;
  uint32_t flags;
  if (get_cache(a[3], a[4], a[5], &dev, &kp, &vp, &sc, &d) != 0) return NULL;
  if (get_step(a[0], a[9], a[6], a[7], &dev, &d, &q, &out, &bt, &sl) != 0) return NULL;
  if (get_tensor(a[1], "k_new", t_bf16, &dev, 3, &k) != 0 || get_tensor(a[2], "v_new", t_bf16, &dev, 3, &v) != 0)
    return NULL;
  if (!same_shape(&k, &v) || k.shape[0] != q.shape[0] || k.shape[1] != d.num_kv_heads || k.shape[2] != d.head_dim)
    return bad_shape("k_new and v_new are [batch, num_kv_heads, head_dim]"), NULL;
  void *table, *qw, *kw, *ws;
  long long max_pos;
  if (get_table(a[8], &dev, d.head_dim, &table, &max_pos) != 0 ||
      get_weight(a[12], "q_weight", &dev, d.head_dim, &qw) != 0 || get_weight(a[13], "k_weight", &dev, d.head_dim, &kw) != 0)
    return NULL;
  const double scale = PyFloat_AsDouble(a[10]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  const double eps = PyFloat_AsDouble(a[14]);
  if ((eps == -1.0 && PyErr_Occurred()) || get_flags(a[16], &flags) != 0) return NULL;
  size_t ws_bytes;
  pkv_stream_t stream;
  if (get_workspace(a[11], dev, &ws, &ws_bytes) != 0 || get_stream(a[15], dev, &stream) != 0) return NULL;
  if (enter_device(dev, &back) != 0) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pkv_decode_append_attn_fp8(q.ptr, k.ptr, v.ptr, kp.ptr, vp.ptr, sc.ptr, bt.ptr, sl.ptr, table, (int32_t)max_pos, qw,
                                  kw, (float)eps, out.ptr, (float)scale, stream, &d, (int32_t)q.shape[0],
                                  (int32_t)bt.shape[1], ws, ws_bytes, flags);
  Py_END_ALLOW_THREADS;
  return leave_device(back, rc);
}

/* (k_pages, v_pages, kv_scales, block_table, seq_lens, k_out, v_out, out_block_table, workspace, stream) */
static PyObject* expand_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (count_args("expand_fp8", n_args, 10) != 0) return NULL;
  long dev = -1, back;
  Tensor kp, vp, sc, bt, sl, ko, vo, ot;
  pkv_cache_desc d;
  if (get_cache(a[0], a[1], a[2], &dev, &kp, &vp, &sc, &d) != 0) return NULL;
  if (get_tensor(a[5], "k_out", t_bf16, &dev, 4, &ko) != 0 || get_tensor(a[6], "v_out", t_bf16, &dev, 4, &vo) != 0 ||
      get_tensor(a[3], "block_table", t_i32, &dev, 2, &bt) != 0 ||
      get_tensor(a[7], "out_block_table", t_i32, &dev, 2, &ot) != 0 ||
      get_tensor(a[4], "seq_lens", t_i32, &dev, -1, &sl) != 0)
    return NULL;
  if (!same_shape(&ko, &vo) || ko.shape[1] != kp.shape[1] || ko.shape[2] != kp.shape[2] || ko.shape[3] != kp.shape[3])
    return bad_shape("k_out and v_out are [pages, num_kv_heads, page_size, head_dim] of the cache's geometry"), NULL;
  if (!same_shape(&bt, &ot) || numel(&sl) != bt.shape[0]) return bad_shape("shape mismatch"), NULL;
  if (fits_i32(bt.shape[0], bt.shape[1], ko.shape[0]) != 0) return NULL;
  void* ws;
  size_t ws_bytes;
  pkv_stream_t stream;
  if (get_workspace(a[8], dev, &ws, &ws_bytes) != 0 || get_stream(a[9], dev, &stream) != 0) return NULL;
  if (enter_device(dev, &back) != 0) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pkv_expand_fp8(kp.ptr, vp.ptr, sc.ptr, bt.ptr, sl.ptr, (int32_t)bt.shape[0], (int32_t)bt.shape[1], ko.ptr, vo.ptr,
                      ot.ptr, (int32_t)ko.shape[0], &d, stream, ws, ws_bytes);
  Py_END_ALLOW_THREADS;
  return leave_device(back, rc);
}

/* (q, k_pages, v_pages, kv_scales or None, block_table, prefix_lens, cu_nodes, tree_mask or None, out, scale, max_nodes,
 * workspace, stream) */
static PyObject* tree_any(PyObject* const* a, Py_ssize_t n_args, int fp8) {
  if (count_args("tree_attn", n_args, 13) != 0) return NULL;
  long dev = -1, back;
  Tensor kp, vp, sc, q, out, bt, pl, cu, mask;
  pkv_cache_desc d;
  if (get_cache(a[1], a[2], fp8 ? a[3] : NULL, &dev, &kp, &vp, &sc, &d) != 0) return NULL;
  if (get_tensor(a[0], "q", t_bf16, &dev, 3, &q) != 0 || get_tensor(a[8], "out", t_bf16, &dev, 3, &out) != 0 ||
      get_tensor(a[4], "block_table", t_i32, &dev, 2, &bt) != 0 ||
      get_tensor(a[5], "prefix_lens", t_i32, &dev, -1, &pl) != 0 || get_tensor(a[6], "cu_nodes", t_i32, &dev, -1, &cu) != 0)
    return NULL;
  if (q.shape[2] != d.head_dim || !same_shape(&q, &out) || numel(&pl) != bt.shape[0] || numel(&cu) != bt.shape[0] + 1)
    return bad_shape("shape mismatch"), NULL;
  mask.ptr = NULL;
  if (a[7] != Py_None) {
    if (get_tensor(a[7], "tree_mask", t_i64, &dev, -1, &mask) != 0) return NULL;
    if (numel(&mask) != q.shape[0]) return bad_shape("tree_mask must be [total_nodes]"), NULL;
  }
  if (fits_i32(q.shape[0], q.shape[1], bt.shape[0]) != 0 || fits_i32(bt.shape[1], 0, 0) != 0) return NULL;
  d.num_q_heads = (int32_t)q.shape[1];
  const double scale = PyFloat_AsDouble(a[9]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  const long max_nodes = PyLong_AsLong(a[10]);
  if ((max_nodes == -1 && PyErr_Occurred()) || fits_i32(max_nodes, 0, 0) != 0) return NULL;
  if (max_nodes < 0) return bad_shape("max_nodes is negative"), NULL;
  void* ws;
  size_t ws_bytes;
  pkv_stream_t stream;
  if (get_workspace(a[11], dev, &ws, &ws_bytes) != 0 || get_stream(a[12], dev, &stream) != 0) return NULL;
  if (enter_device(dev, &back) != 0) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fp8 ? pkv_tree_attn_fp8(q.ptr, kp.ptr, vp.ptr, sc.ptr, bt.ptr, pl.ptr, cu.ptr, mask.ptr, (int32_t)bt.shape[0],
                               (int32_t)q.shape[0], (int32_t)max_nodes, out.ptr, (float)scale, stream, &d,
                               (int32_t)bt.shape[1], ws, ws_bytes)
           : pkv_tree_attn(q.ptr, kp.ptr, vp.ptr, bt.ptr, pl.ptr, cu.ptr, mask.ptr, (int32_t)bt.shape[0],
                           (int32_t)q.shape[0], (int32_t)max_nodes, out.ptr, (float)scale, stream, &d,
                           (int32_t)bt.shape[1], ws, ws_bytes);
  Py_END_ALLOW_THREADS;
  return leave_device(back, rc);
}

static PyObject* tree_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return tree_any(a, n, 0);
}

static PyObject* tree_attn_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return tree_any(a, n, 1);
}

/* The pools of one kind of all layers: a tensor of 4 dimensions (one layer), one of 5 (all layers, stacked) or a list or
 * tuple of the former. *first is the shape of one pool; ptrs (PyMem) holds *n addresses. */
static int get_layers(PyObject* o, const char* name, PyObject* dtype, long* dev, Tensor* first, void*** ptrs, long long* n) {
  const int many = PyList_Check(o) || PyTuple_Check(o);
  Tensor t;
  *ptrs = NULL;
  if (!many) {
    if (get_tensor(o, name, dtype, dev, -1, &t) != 0) return -1;
    if (t.nd != 4 && t.nd != 5) {
      PyErr_Format(PyExc_ValueError, "%s must have 4 dimensions, or 5 for the pools of all layers, got %d", name, t.nd);
      return -1;
    }
    *n = t.nd == 5 ? t.shape[0] : 1;
    first->nd = 4;
    long long bytes = dtype == t_bf16 ? 2 : 1;
    for (int i = 0; i < 4; ++i) bytes *= first->shape[i] = t.shape[i + t.nd - 4];
    if (fits_i32(*n, 0, 0) != 0) return -1;
    if ((*ptrs = PyMem_Malloc((size_t)(*n + 1) * sizeof(void*))) == NULL) return PyErr_NoMemory(), -1;
    for (long long i = 0; i < *n; ++i) (*ptrs)[i] = (char*)t.ptr + i * bytes;
    return 0;
  }
  *n = PySequence_Fast_GET_SIZE(o);
  if (fits_i32(*n, 0, 0) != 0) return -1;
  if ((*ptrs = PyMem_Malloc((size_t)(*n + 1) * sizeof(void*))) == NULL) return PyErr_NoMemory(), -1;
  first->nd = 0;
  for (long long i = 0; i < *n; ++i) {
    if (i >= PySequence_Fast_GET_SIZE(o)) return bad_shape("the list of pools changed its length");
    PyObject* pool = PySequence_Fast_GET_ITEM(o, i);
    Py_INCREF(pool);
    const int rc = get_tensor(pool, name, dtype, dev, 4, &t);
    Py_DECREF(pool);
    if (rc != 0) return -1;
    if (i == 0) *first = t;
    if (!same_shape(first, &t)) {
      PyErr_Format(PyExc_ValueError, "%s: the layers' pools differ in shape", name);
      return -1;
    }
    (*ptrs)[i] = t.ptr;
  }
  return 0;
}

typedef struct {
  void** p[3]; /* K, V, scales or NULL */
  long long n;
  pkv_cache_desc d;
} Layers;

static void free_layers(Layers* l) {
  for (int i = 0; i < 3; ++i) PyMem_Free(l->p[i]);
}

static int get_all_layers(PyObject* k, PyObject* v, PyObject* scales, long* dev, Layers* l) {
  Tensor tk, tv, ts;
  long long nv, ns;
  const int fp8 = scales != Py_None;
  memset(l, 0, sizeof *l);
  if (get_layers(k, "k_pages", fp8 ? t_e4m3 : t_bf16, dev, &tk, &l->p[0], &l->n) != 0 ||
      get_layers(v, "v_pages", fp8 ? t_e4m3 : t_bf16, dev, &tv, &l->p[1], &nv) != 0)
    return -1;
  if (l->n < 1) return bad_shape("there are no pools");
  if (nv != l->n || !same_shape(&tk, &tv)) return bad_shape(kPools);
  if (fp8) {
    if (get_layers(scales, "kv_scales", t_e8m0, dev, &ts, &l->p[2], &ns) != 0) return -1;
    if (ns != l->n || ts.shape[0] != tk.shape[0] || ts.shape[1] != tk.shape[1] || ts.shape[2] != 2 || ts.shape[3] != tk.shape[2])
      return bad_shape("kv_scales must be [num_pages, num_kv_heads, 2, page_size] of the pools' sizes, for each layer");
  }
  if (fits_i32(tk.shape[0], tk.shape[1], tk.shape[2]) != 0 || fits_i32(tk.shape[3], 0, 0) != 0) return -1;
  l->d.num_pages = (int32_t)tk.shape[0];
  l->d.num_q_heads = l->d.num_kv_heads = (int32_t)tk.shape[1];
  l->d.page_size = (int32_t)tk.shape[2];
  l->d.head_dim = (int32_t)tk.shape[3];
  return 0;
}

/* (path, path_lens, prefix_lens, block_table, k_pages, v_pages, kv_scales or None, workspace, stream) */
static PyObject* keep_nodes(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (count_args("keep_nodes", n_args, 9) != 0) return NULL;
  long dev = -1, back;
  Tensor path, n, pl, bt;
  Layers l;
  void* ws;
  size_t ws_bytes;
  pkv_stream_t stream;
  PyObject* done = NULL;
  if (get_all_layers(a[4], a[5], a[6], &dev, &l) != 0) goto end;
  if (get_tensor(a[0], "path", t_i32, &dev, 2, &path) != 0 || get_tensor(a[1], "path_lens", t_i32, &dev, -1, &n) != 0 ||
      get_tensor(a[2], "prefix_lens", t_i32, &dev, -1, &pl) != 0 || get_tensor(a[3], "block_table", t_i32, &dev, 2, &bt) != 0)
    goto end;
  if (numel(&n) != path.shape[0] || numel(&pl) != path.shape[0] || bt.shape[0] != path.shape[0]) {
    bad_shape("shape mismatch");
    goto end;
  }
  if (fits_i32(path.shape[0], path.shape[1], bt.shape[1]) != 0) goto end;
  if (get_workspace(a[7], dev, &ws, &ws_bytes) != 0 || get_stream(a[8], dev, &stream) != 0) goto end;
  if (enter_device(dev, &back) != 0) goto end;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pkv_keep_nodes(path.ptr, n.ptr, pl.ptr, bt.ptr, (int32_t)path.shape[0], (int32_t)path.shape[1], (int32_t)bt.shape[1],
                      l.p[0], l.p[1], l.p[2], (int32_t)l.n, &l.d, stream, ws, ws_bytes);
  Py_END_ALLOW_THREADS;
  done = leave_device(back, rc);
end:
  free_layers(&l);
  return done;
}

/* (src, dst, k_pages, v_pages, kv_scales or None, workspace, stream) */
static PyObject* copy_pages(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (count_args("copy_pages", n_args, 7) != 0) return NULL;
  long dev = -1, back;
  Tensor src, dst;
  Layers l;
  void* ws;
  size_t ws_bytes;
  pkv_stream_t stream;
  PyObject* done = NULL;
  if (get_all_layers(a[2], a[3], a[4], &dev, &l) != 0) goto end;
  if (get_tensor(a[0], "src", t_i32, &dev, 1, &src) != 0 || get_tensor(a[1], "dst", t_i32, &dev, 1, &dst) != 0) goto end;
  if (src.shape[0] != dst.shape[0]) {
    bad_shape("src and dst differ in length");
    goto end;
  }
  if (fits_i32(src.shape[0], 0, 0) != 0) goto end;
  if (get_workspace(a[5], dev, &ws, &ws_bytes) != 0 || get_stream(a[6], dev, &stream) != 0) goto end;
  if (enter_device(dev, &back) != 0) goto end;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pkv_copy_pages(src.ptr, dst.ptr, (int32_t)src.shape[0], l.p[0], l.p[1], l.p[2], (int32_t)l.n, &l.d, stream, ws, ws_bytes);
  Py_END_ALLOW_THREADS;
  done = leave_device(back, rc);
end:
  free_layers(&l);
  return done;
}

static PyMethodDef methods[] = {
    {"append_rope", (PyCFunction)(void (*)(void))append_rope, METH_FASTCALL, NULL},
    {"append_rope_fp8", (PyCFunction)(void (*)(void))append_rope_fp8, METH_FASTCALL, NULL},
    {"decode_attn_fp8", (PyCFunction)(void (*)(void))decode_attn_fp8, METH_FASTCALL, NULL},
    {"decode_append_attn_fp8", (PyCFunction)(void (*)(void))decode_append_attn_fp8, METH_FASTCALL, NULL},
    {"expand_fp8", (PyCFunction)(void (*)(void))expand_fp8, METH_FASTCALL, NULL},
    {"tree_attn", (PyCFunction)(void (*)(void))tree_attn, METH_FASTCALL, NULL},
    {"tree_attn_fp8", (PyCFunction)(void (*)(void))tree_attn_fp8, METH_FASTCALL, NULL},
    {"keep_nodes", (PyCFunction)(void (*)(void))keep_nodes, METH_FASTCALL, NULL},
    {"copy_pages", (PyCFunction)(void (*)(void))copy_pages, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Checks and calls of libpkv's short kernels.", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  const struct {
    PyObject** at;
    const char* text;
  } names[] = {{&s_dtype, "dtype"},       {&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"},
               {&s_data_ptr, "data_ptr"}, {&s_shape, "shape"},           {&s_stride, "stride"},
               {&s_tensor, "tensor"},     {&s_cuda_stream, "cuda_stream"}, {&s_device, "device"},
               {&s_index, "index"}};
  for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
    if ((*names[i].at = PyUnicode_InternFromString(names[i].text)) == NULL) return NULL;
  PyObject* torch = PyImport_ImportModule("torch");
  if (torch == NULL) return NULL;
  PyObject* c = PyObject_GetAttrString(torch, "_C");
  const struct {
    PyObject** at;
    PyObject* of;
    const char* text;
  } objects[] = {{&t_bf16, torch, "bfloat16"},
                 {&t_i32, torch, "int32"},
                 {&t_i64, torch, "int64"},
                 {&t_f32, torch, "float32"},
                 {&t_e4m3, torch, "float8_e4m3fn"},
                 {&t_e8m0, torch, "float8_e8m0fnu"},
                 {&f_raw_stream, c, "_cuda_getCurrentRawStream"},
                 {&f_get_device, c, "_cuda_getDevice"},
                 {&f_exchange_device, c, "_cuda_exchangeDevice"}};
  int ok = c != NULL;
  for (size_t i = 0; ok && i < sizeof objects / sizeof objects[0]; ++i)
    ok = (*objects[i].at = PyObject_GetAttrString(objects[i].of, objects[i].text)) != NULL;
  Py_XDECREF(c);
  Py_DECREF(torch);
  return ok ? PyModule_Create(&module) : NULL;
}
