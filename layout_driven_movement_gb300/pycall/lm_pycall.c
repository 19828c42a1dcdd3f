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
static PyObject *t_bf16, *t_f16, *t_f32, *t_i32, *t_i64;

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
  int64_t size[3], stride[3];
  PyObject* dtype; /* a singleton of torch's, borrowed */
} tensor;

static int ints(PyObject* tuple, int64_t* out) {
  Py_ssize_t i, n;
  if (!tuple || !PyTuple_Check(tuple)) return -1;
  n = PyTuple_GET_SIZE(tuple);
  for (i = 0; i < n && i < 3; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

/* A CUDA tensor of 1 to 3 dimensions. */
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
  if (t->dims < 1 || t->dims > 3)
    return (int)wrong(what, "a tensor of 1 to 3 dimensions");
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

/* kv_attend(plan, cache, dim, elem, q, page_table, lens, out, workspace,
 * lse, scale, window, stream); workspace and lse may be None */
static PyObject* py_kv_attend(PyObject* self, PyObject* const* a,
                              Py_ssize_t n) {
  tensor q, o, p, l, w, e;
  lm_rows qr, orr;
  int rc, elem;
  void *plan, *cache, *stream;
  int64_t dim, window, ws_bytes = 0;
  double scale;
  char *ws = NULL, *lse = NULL;
  (void)self;
  if (want(n, 13, "kv_attend")) return NULL;
  plan = PTR(0);
  cache = PTR(1);
  dim = I64(2);
  elem = (int)I64(3);
  if (rows(a[4], "q", dim, elem, &q, &qr) ||
      rows(a[7], "out", dim, elem, &o, &orr))
    return NULL;
  if (o.size[0] != q.size[0] || o.size[1] != q.size[1]) {
    wrong("out", "q's shape");
    return NULL;
  }
  if (vector(a[6], "lens", q.size[0], t_i32, &l) ||
      page_table(a[5], q.size[0], &p))
    return NULL;
  if (a[8] != Py_None) {
    if (look(a[8], "workspace", &w)) return NULL;
    if (w.dims != 1 || !dense(&w)) {
      wrong("workspace", "a contiguous vector");
      return NULL;
    }
    ws = w.data;
    {
      PyObject* b = PyObject_GetAttrString(a[8], "nbytes");
      if (!b) return NULL;
      ws_bytes = PyLong_AsLongLong(b);
      Py_DECREF(b);
    }
  }
  if (a[9] != Py_None) {
    if (look(a[9], "lse", &e)) return NULL;
    if (e.dtype != t_f32 || !dense(&e) || count(&e) != q.size[0] * q.size[1]) {
      wrong("lse", "a contiguous float32 tensor [sequences, query heads]");
      return NULL;
    }
    lse = e.data;
  }
  scale = PyFloat_AsDouble(a[10]);
  window = I64(11);
  stream = PTR(12);
  if (PyErr_Occurred()) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = q.size[0] > INT32_MAX || q.size[1] > INT32_MAX
           ? LM_E_INVALID
           : lm_kv_attend(plan, cache, &qr, &orr, (int)q.size[0],
                          (int)q.size[1], (int32_t*)p.data, p.stride[0],
                          p.size[1], (int32_t*)l.data, window, (float)scale,
                          (float*)lse, ws, ws_bytes, stream);
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
  t_i32 = PyObject_GetAttrString(torch, "int32");
  t_i64 = PyObject_GetAttrString(torch, "int64");
  Py_DECREF(torch);
  if (!n_data_ptr || !n_is_cuda || !n_shape || !n_dtype || !n_stride ||
      !t_bf16 || !t_f16 || !t_f32 || !t_i32 || !t_i64)
    return NULL;
  return PyModule_Create(&module);
}
