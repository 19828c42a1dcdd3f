/* The calls of a decoding step from Python: reads the tensors' pointers,
 * shapes and strides and makes one library call.
 *
 * A step makes several such calls of a few microseconds of device work each.
 * Through ctypes one takes 8.5 to 10 microseconds of host time, most of it
 * looking at tensors and converting arguments one by one in the interpreter;
 * here it takes 4.5 to 5.3.  Checks that need the tensors (CUDA,
 * type, shape, contiguity) raise ValueError; all others are the library's,
 * whose status is returned. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "layoutmove.h"

static PyObject *n_is_cuda, *n_shape, *n_dtype, *n_stride, *n_data_ptr;
static PyObject *t_bf16, *t_f16, *t_f32, *t_i8, *t_i32, *t_i64;

static int64_t wrong(const char* what, const char* wanted) {
  if (!PyErr_Occurred())
    PyErr_Format(PyExc_ValueError, "%s: %s is wanted", what, wanted);
  return -1;
}

/* lm_elem of a dtype, 0 for any other. */
static int elem_of(PyObject* dtype) {
  return dtype == t_bf16 ? LM_BF16
         : dtype == t_f16 ? LM_F16
         : dtype == t_f32 ? LM_F32
                          : 0;
}

typedef struct {
  char* data;
  int dims;
  int64_t size[4], stride[4];
  PyObject* dtype; /* a singleton of torch's, borrowed */
} tensor;

static int ints(PyObject* tuple, int64_t* out) {
  Py_ssize_t i, n;
  if (!tuple || !PyTuple_Check(tuple)) return -1;
  n = PyTuple_GET_SIZE(tuple);
  for (i = 0; i < n && i < 4; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

/* A CUDA tensor of 1 to 4 dimensions. */
static int look(PyObject* o, const char* what, tensor* t) {
  PyObject *a = PyObject_GetAttr(o, n_is_cuda), *b;
  const int cuda = a == Py_True;
  if (!a) PyErr_Clear(); /* no tensor at all, None among others */
  Py_XDECREF(a);
  if (!cuda) return (int)wrong(what, "a CUDA tensor");
  a = PyObject_GetAttr(o, n_shape);
  b = PyObject_CallMethodNoArgs(o, n_stride);
  t->dims = ints(a, t->size);
  if (ints(b, t->stride) != t->dims) t->dims = -1;
  Py_XDECREF(a);
  Py_XDECREF(b);
  if (t->dims < 1 || t->dims > 4)
    return (int)wrong(what, "a tensor of 1 to 4 dimensions");
  t->dtype = PyObject_GetAttr(o, n_dtype);
  if (!t->dtype) return -1;
  Py_DECREF(t->dtype);
  a = PyObject_CallMethodNoArgs(o, n_data_ptr);
  if (!a) return -1;
  t->data = (char*)(uintptr_t)PyLong_AsUnsignedLongLong(a);
  Py_DECREF(a);
  return PyErr_Occurred() ? -1 : 0;
}

static int64_t count(const tensor* t) {
  int64_t n = 1;
  int i;
  for (i = 0; i < t->dims; ++i) n *= t->size[i];
  return n;
}

static int dense(const tensor* t) {
  int64_t n = 1;
  int i;
  for (i = t->dims - 1; i >= 0; --i) {
    if (t->size[i] != 1 && t->stride[i] != n) return 0;
    n *= t->size[i];
  }
  return 1;
}

/* [tokens, heads, dim], dim contiguous and (unless 0) `dim` long, of dtype
 * `elem` (0: any of lm_elem). */
static int rows(PyObject* o, const char* what, int64_t dim, int elem,
                tensor* t, lm_rows* r) {
  if (look(o, what, t)) return -1;
  if (t->dims != 3 || t->size[2] != dim ||
      (dim > 1 && t->stride[2] != 1))
    return (int)wrong(what, "[tokens, heads, dim] with a contiguous dim of "
                            "the plan's");
  if (!elem_of(t->dtype) || (elem && elem_of(t->dtype) != elem))
    return (int)wrong(what, "the plan's (or the other tensor's) type");
  r->data = t->data;
  r->token_stride = t->stride[0];
  r->head_stride = t->stride[1];
  r->capacity = t->size[0] && t->size[1]
                    ? (t->size[0] - 1) * t->stride[0] +
                          (t->size[1] - 1) * t->stride[1] + dim
                    : 0;
  return 0;
}

static int vector(PyObject* o, const char* what, int64_t n, PyObject* dtype,
                  tensor* t) {
  if (look(o, what, t)) return -1;
  if (t->dims != 1 || t->size[0] != n || !dense(t) ||
      (t->dtype != dtype && !(dtype == NULL && (t->dtype == t_i32 ||
                                                t->dtype == t_i64))))
    return (int)wrong(what, dtype == t_i32   ? "a contiguous int32 vector, "
                                               "one per sequence,"
                            : dtype == t_i64 ? "a contiguous int64 vector, "
                                               "one per token,"
                                             : "a contiguous int32 or int64 "
                                               "vector, one per token,");
  return 0;
}

typedef struct {
  void* pos;
  int bytes;
  float* table;
  int64_t rows;
} turn;

static int turn_of(PyObject* pos, PyObject* table, int64_t tokens,
                   int64_t rotary, turn* out) {
  tensor p, t;
  if (vector(pos, "positions", tokens, NULL, &p) || look(table, "table", &t))
    return -1;
  if (t.dtype != t_f32 || !dense(&t) || count(&t) != t.size[0] * rotary)
    return (int)wrong("table", "a contiguous float32 CUDA tensor [positions, "
                               "rotary_dim]");
  out->pos = p.data;
  out->bytes = p.dtype == t_i64 ? 8 : 4;
  out->table = (float*)t.data;
  out->rows = t.size[0];
  return 0;
}

static int want(Py_ssize_t n, Py_ssize_t args, const char* name) {
  if (n == args) return 0;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, args);
  return -1;
}

#define PTR(i) ((void*)(uintptr_t)PyLong_AsUnsignedLongLong(a[i]))
#define I64(i) PyLong_AsLongLong(a[i])

/* rope(plan, head_dim, rotary_dim, x, positions, table, out, inverse,
 * stream) */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  tensor x, o;
  lm_rows xr, orr;
  turn t;
  int rc, elem, inverse;
  void *plan, *stream;
  int64_t dim;
  (void)self;
  if (want(n, 9, "rope")) return NULL;
  plan = PTR(0);
  dim = I64(1);
  if (rows(a[3], "x", dim, 0, &x, &xr)) return NULL;
  elem = elem_of(x.dtype);
  if (rows(a[6], "out", dim, elem, &o, &orr)) return NULL;
  if (o.size[0] != x.size[0] || o.size[1] != x.size[1]) {
    wrong("out", "x's shape");
    return NULL;
  }
  if (turn_of(a[4], a[5], x.size[0], I64(2), &t)) return NULL;
  inverse = PyObject_IsTrue(a[7]);
  stream = PTR(8);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lm_rope(plan, elem, &xr, &orr, x.size[0],
               x.size[1] > INT32_MAX ? -1 : (int)x.size[1], t.pos, t.bytes,
               t.table, t.rows, inverse, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* kv_write(plan, cache, heads, dim, elem, k, v, slots, rope, rotary_dim,
 * positions, table, stream); rope 0: keys are not turned */
static PyObject* py_kv_write(PyObject* self, PyObject* const* a,
                             Py_ssize_t n) {
  tensor k, v, s;
  lm_rows kr, vr;
  turn t = {NULL, 0, NULL, 0};
  int rc, elem;
  void *plan, *cache, *rope, *stream;
  int64_t heads, dim;
  (void)self;
  if (want(n, 13, "kv_write")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  heads = I64(2);
  dim = I64(3);
  elem = (int)I64(4);
  if (rows(a[5], "k", dim, elem, &k, &kr) ||
      rows(a[6], "v", dim, elem, &v, &vr))
    return NULL;
  if (k.size[1] != heads || v.size[1] != heads || v.size[0] != k.size[0]) {
    wrong("k and v", "the plan's heads, and as many tokens in each,");
    return NULL;
  }
  if (vector(a[7], "slots", k.size[0], t_i64, &s)) return NULL;
  rope = PTR(8);
  if (rope && turn_of(a[10], a[11], k.size[0], I64(9), &t)) return NULL;
  stream = PTR(12);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lm_kv_write(plan, cache, &kr, &vr, k.size[0], (int64_t*)s.data, rope,
                   t.pos, t.bytes, t.table, t.rows, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

static int page_table(PyObject* o, int64_t seqs, tensor* t) {
  if (look(o, "page_table", t)) return -1;
  if (t->dims != 2 || t->size[0] != seqs || t->dtype != t_i32 ||
      (t->size[1] > 1 && t->stride[1] != 1))
    return (int)wrong("page_table", "an int32 tensor [sequences, pages] with "
                                    "contiguous rows");
  return 0;
}

/* kv_read(plan, cache, heads, dim, page_table, lens, starts, k_out, v_out,
 * stream) */
static PyObject* py_kv_read(PyObject* self, PyObject* const* a,
                            Py_ssize_t n) {
  tensor k, v, p, l, s;
  lm_rows kr, vr;
  int rc, elem;
  void *plan, *cache, *stream;
  int64_t heads, dim;
  (void)self;
  if (want(n, 10, "kv_read")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  heads = I64(2);
  dim = I64(3);
  if (rows(a[7], "k_out", dim, 0, &k, &kr)) return NULL;
  elem = elem_of(k.dtype);
  if (rows(a[8], "v_out", dim, elem, &v, &vr)) return NULL;
  if (k.size[1] != heads || v.size[1] != heads || v.size[0] != k.size[0]) {
    wrong("k_out and v_out", "the plan's heads, and as many rows in each,");
    return NULL;
  }
  if (look(a[5], "lens", &l) ||
      vector(a[5], "lens", l.size[0], t_i32, &l) ||
      vector(a[6], "starts (one more than lens)", l.size[0] + 1, t_i32, &s) ||
      page_table(a[4], l.size[0], &p))
    return NULL;
  stream = PTR(9);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = l.size[0] > INT32_MAX
           ? LM_E_INVALID
           : lm_kv_read(plan, cache, (int32_t*)p.data, p.stride[0],
                        (int)l.size[0], p.size[1], (int32_t*)l.data,
                        (int32_t*)s.data, elem, &kr, &vr, k.size[0], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* A workspace's address and bytes; None: none. */
static int space(PyObject* o, char** data, int64_t* bytes) {
  tensor w;
  PyObject* b;
  *data = NULL;
  *bytes = 0;
  if (o == Py_None) return 0;
  if (look(o, "workspace", &w)) return -1;
  if (w.dims != 1 || !dense(&w))
    return (int)wrong("workspace", "a contiguous vector");
  b = PyObject_GetAttrString(o, "nbytes");
  if (!b) return -1;
  *bytes = PyLong_AsLongLong(b);
  Py_DECREF(b);
  *data = w.data;
  return PyErr_Occurred() ? -1 : 0;
}

/* A contiguous tensor of a type. */
static int buffer(PyObject* o, const char* what, PyObject* dtype,
                  const char* wanted, tensor* t) {
  if (look(o, what, t)) return -1;
  if (t->dtype != dtype || !dense(t)) return (int)wrong(what, wanted);
  return 0;
}

/* lse [sequences, query heads]; None: none. */
static int lse_of(PyObject* o, const tensor* q, char** data) {
  tensor e;
  *data = NULL;
  if (o == Py_None) return 0;
  if (look(o, "lse", &e)) return -1;
  if (e.dtype != t_f32 || !dense(&e) || count(&e) != q->size[0] * q->size[1])
    return (int)wrong("lse",
                      "a contiguous float32 tensor [sequences, query heads]");
  *data = e.data;
  return 0;
}

/* kv_attend(plan, cache, heads, dim, elem, q, page_table, lens, out,
 * workspace, lse, scale, window, weights, stream); workspace, lse and weights
 * may be None, the page table have a dimension for the key heads */
static PyObject* py_kv_attend(PyObject* self, PyObject* const* a,
                              Py_ssize_t n) {
  tensor q, o, p, l, m;
  lm_rows qr, orr;
  int rc, elem;
  void *plan, *cache, *stream;
  int64_t heads, dim, window, ws_bytes, by_head = 0, n_weights = 0;
  double scale;
  char *ws, *lse, *weights = NULL;
  (void)self;
  if (want(n, 15, "kv_attend")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  heads = I64(2);
  dim = I64(3);
  elem = (int)I64(4);
  if (rows(a[5], "q", dim, elem, &q, &qr) ||
      rows(a[8], "out", dim, elem, &o, &orr))
    return NULL;
  if (o.size[0] != q.size[0] || o.size[1] != q.size[1]) {
    wrong("out", "q's shape");
    return NULL;
  }
  if (vector(a[7], "lens", q.size[0], t_i32, &l) || look(a[6], "page_table", &p))
    return NULL;
  if (p.dims == 3) {
    if (p.size[0] != q.size[0] || p.size[1] != heads || p.dtype != t_i32 ||
        (p.size[2] > 1 && p.stride[2] != 1)) {
      wrong("page_table", "an int32 tensor [sequences, key heads, pages] with "
                          "contiguous rows");
      return NULL;
    }
    by_head = p.stride[1];
    p.size[1] = p.size[2];
    /* (of heads and sequences that share pages, a stride may be 0) */
    if (p.size[0] > 1 && p.stride[0] < p.size[1]) {
      wrong("page_table", "rows of its own for every sequence");
      return NULL;
    }
  } else if (page_table(a[6], q.size[0], &p)) {
    return NULL;
  }
  if (space(a[9], &ws, &ws_bytes) || lse_of(a[10], &q, &lse)) return NULL;
  if (a[13] != Py_None) {
    if (buffer(a[13], "weights", t_f32,
               "a contiguous float32 tensor [pages, key heads, page_tokens]",
               &m))
      return NULL;
    weights = m.data;
    n_weights = count(&m);
  }
  scale = PyFloat_AsDouble(a[11]);
  window = I64(12);
  stream = PTR(14);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = q.size[0] > INT32_MAX || q.size[1] > INT32_MAX
           ? LM_E_INVALID
           : lm_kv_attend_weigh(plan, cache, &qr, &orr, (int)q.size[0],
                                (int)q.size[1], (int32_t*)p.data, p.stride[0],
                                by_head, p.size[1], (int32_t*)l.data, window,
                                (float)scale, (float*)lse, (float*)weights,
                                n_weights, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* kv_attend_shared(plan, cache, dim, elem, q, shared_table, shared_lens,
 * starts, page_table, lens, out, workspace, lse, scale, stream); lse may be
 * None */
static PyObject* py_kv_attend_shared(PyObject* self, PyObject* const* a,
                                     Py_ssize_t n) {
  tensor q, o, p, l, t, sl, st;
  lm_rows qr, orr;
  int rc, elem;
  void *plan, *cache, *stream;
  int64_t dim, ws_bytes;
  double scale;
  char *ws, *lse;
  (void)self;
  if (want(n, 15, "kv_attend_shared")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  dim = I64(2);
  elem = (int)I64(3);
  if (rows(a[4], "q", dim, elem, &q, &qr) ||
      rows(a[10], "out", dim, elem, &o, &orr))
    return NULL;
  if (o.size[0] != q.size[0] || o.size[1] != q.size[1]) {
    wrong("out", "q's shape");
    return NULL;
  }
  if (look(a[6], "shared_lens", &sl) ||
      vector(a[6], "shared_lens", sl.size[0], t_i32, &sl) ||
      vector(a[7], "starts (one more than shared_lens)", sl.size[0] + 1, t_i32,
             &st) ||
      page_table(a[5], sl.size[0], &t) ||
      vector(a[9], "lens", q.size[0], t_i32, &l) ||
      page_table(a[8], q.size[0], &p) || space(a[11], &ws, &ws_bytes) ||
      lse_of(a[12], &q, &lse))
    return NULL;
  scale = PyFloat_AsDouble(a[13]);
  stream = PTR(14);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = q.size[0] > INT32_MAX || q.size[1] > INT32_MAX ||
               sl.size[0] > INT32_MAX
           ? LM_E_INVALID
           : lm_kv_attend_shared(
                 plan, cache, &qr, &orr, (int)q.size[0], (int)q.size[1],
                 (int32_t*)t.data, t.stride[0], (int)sl.size[0], t.size[1],
                 (int32_t*)sl.data, (int32_t*)st.data, (int32_t*)p.data,
                 p.stride[0], p.size[1], (int32_t*)l.data, (float)scale,
                 (float*)lse, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* bounds [pages, heads, 2, dim] int8 and scale [pages, heads] float32 */
static int bounds_of(PyObject* bo, PyObject* so, int64_t heads, int64_t dim,
                     lm_kv_bounds* out, int64_t* pages) {
  tensor b, s;
  if (buffer(bo, "bounds", t_i8,
             "a contiguous int8 tensor [pages, key heads, 2, dim]", &b) ||
      buffer(so, "bound_scale", t_f32,
             "a contiguous float32 tensor [pages, key heads]", &s))
    return -1;
  if (b.dims != 4 || b.size[1] != heads || b.size[2] != 2 ||
      b.size[3] != dim)
    return (int)wrong("bounds", "[pages, key heads, 2, dim]");
  if (s.dims != 2 || s.size[0] != b.size[0] || s.size[1] != heads)
    return (int)wrong("bound_scale", "[pages, key heads]");
  out->data = (int8_t*)b.data;
  out->scale = (float*)s.data;
  out->capacity = count(&b);
  out->scale_capacity = count(&s);
  *pages = b.size[0];
  return 0;
}

/* kv_bound(plan, cache, heads, dim, pages, counts, bounds, bound_scale,
 * stream) */
static PyObject* py_kv_bound(PyObject* self, PyObject* const* a,
                             Py_ssize_t n) {
  tensor p, c;
  lm_kv_bounds b;
  int rc;
  void *plan, *cache, *stream;
  int64_t pages;
  (void)self;
  if (want(n, 9, "kv_bound")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  if (look(a[4], "pages", &p) ||
      vector(a[4], "pages", p.size[0], t_i32, &p) ||
      vector(a[5], "counts", p.size[0], t_i32, &c) ||
      bounds_of(a[6], a[7], I64(2), I64(3), &b, &pages))
    return NULL;
  stream = PTR(8);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lm_kv_bound(plan, cache, (int32_t*)p.data, (int32_t*)c.data, p.size[0],
                   &b, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* kv_select(plan, heads, dim, elem, q, bounds, bound_scale, page_table, lens,
 * selected, selected_lens, workspace, first, last, stream) */
static PyObject* py_kv_select(PyObject* self, PyObject* const* a,
                              Py_ssize_t n) {
  tensor q, p, l, s, sl;
  lm_rows qr;
  lm_kv_bounds b;
  int rc;
  void *plan, *stream;
  int64_t heads, dim, pages, ws_bytes, first, last;
  char* ws;
  (void)self;
  if (want(n, 15, "kv_select")) return NULL;
  plan = PTR(0);
  heads = I64(1);
  dim = I64(2);
  if (rows(a[4], "q", dim, (int)I64(3), &q, &qr) ||
      bounds_of(a[5], a[6], heads, dim, &b, &pages) ||
      page_table(a[7], q.size[0], &p) ||
      vector(a[8], "lens", q.size[0], t_i32, &l) ||
      buffer(a[9], "selected", t_i32,
             "a contiguous int32 tensor [sequences, key heads, pages]", &s) ||
      vector(a[10], "selected_lens", q.size[0], t_i32, &sl) ||
      space(a[11], &ws, &ws_bytes))
    return NULL;
  if (s.dims != 3 || s.size[0] != q.size[0] || s.size[1] != heads) {
    wrong("selected", "[sequences, key heads, pages]");
    return NULL;
  }
  first = I64(12);
  last = I64(13);
  stream = PTR(14);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = q.size[0] > INT32_MAX || q.size[1] > INT32_MAX ||
               s.size[2] > INT32_MAX || first > INT32_MAX ||
               last > INT32_MAX || first < 0 || last < 0
           ? LM_E_INVALID
           : lm_kv_select(plan, pages, &b, &qr, (int)q.size[0],
                          (int)q.size[1], (int32_t*)p.data, p.stride[0],
                          p.size[1], (int32_t*)l.data, (int)s.size[2],
                          (int)first, (int)last, (int32_t*)s.data,
                          (int32_t*)sl.data, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* kv_evict(plan, cache, weights, page_table, lens, kept_table, kept_lens,
 * keep, recent, workspace, stream) */
static PyObject* py_kv_evict(PyObject* self, PyObject* const* a,
                             Py_ssize_t n) {
  tensor m, p, l, k, kl;
  int rc;
  void *plan, *cache, *stream;
  int64_t ws_bytes, keep, recent;
  char* ws;
  (void)self;
  if (want(n, 11, "kv_evict")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  if (buffer(a[2], "weights", t_f32,
             "a contiguous float32 tensor [pages, key heads, page_tokens]",
             &m) ||
      look(a[4], "lens", &l) || vector(a[4], "lens", l.size[0], t_i32, &l) ||
      page_table(a[3], l.size[0], &p) || page_table(a[5], l.size[0], &k) ||
      vector(a[6], "kept_lens", l.size[0], t_i32, &kl) ||
      space(a[9], &ws, &ws_bytes))
    return NULL;
  keep = I64(7);
  recent = I64(8);
  stream = PTR(10);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = l.size[0] > INT32_MAX || keep < 1 || keep > INT32_MAX || recent < 0 ||
               recent > keep
           ? LM_E_INVALID
           : lm_kv_evict(plan, cache, (float*)m.data, count(&m),
                         (int32_t*)p.data, p.stride[0], (int)l.size[0],
                         p.size[1], (int32_t*)l.data, (int32_t*)k.data,
                         k.stride[0], k.size[1], (int32_t*)kl.data, (int)keep,
                         (int)recent, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"kv_write", (PyCFunction)(void (*)(void))py_kv_write, METH_FASTCALL,
     NULL},
    {"kv_read", (PyCFunction)(void (*)(void))py_kv_read, METH_FASTCALL, NULL},
    {"kv_attend", (PyCFunction)(void (*)(void))py_kv_attend, METH_FASTCALL,
     NULL},
    {"kv_attend_shared", (PyCFunction)(void (*)(void))py_kv_attend_shared,
     METH_FASTCALL, NULL},
    {"kv_bound", (PyCFunction)(void (*)(void))py_kv_bound, METH_FASTCALL,
     NULL},
    {"kv_select", (PyCFunction)(void (*)(void))py_kv_select, METH_FASTCALL,
     NULL},
    {"kv_evict", (PyCFunction)(void (*)(void))py_kv_evict, METH_FASTCALL,
     NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", NULL,
                                    -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycall(void) {
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return NULL;
  n_is_cuda = PyUnicode_InternFromString("is_cuda");
  n_shape = PyUnicode_InternFromString("shape");
  n_dtype = PyUnicode_InternFromString("dtype");
  n_stride = PyUnicode_InternFromString("stride");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  t_bf16 = PyObject_GetAttrString(torch, "bfloat16");
  t_f16 = PyObject_GetAttrString(torch, "float16");
  t_f32 = PyObject_GetAttrString(torch, "float32");
  t_i8 = PyObject_GetAttrString(torch, "int8");
  t_i32 = PyObject_GetAttrString(torch, "int32");
  t_i64 = PyObject_GetAttrString(torch, "int64");
  Py_DECREF(torch);
  if (!n_data_ptr || !n_is_cuda || !n_shape || !n_dtype || !n_stride ||
      !t_bf16 || !t_f16 || !t_f32 || !t_i8 || !t_i32 || !t_i64)
    return NULL;
  return PyModule_Create(&module);
}
