/* The 8-bit cache's calls from Python without a ctypes round trip: a CPython extension that checks the
 * tensors of a call, reads their pointers, sizes and strides, and calls the C ABI (include/pkv.h) with the
 * GIL released.  Small calls are bound by this: a decode of four sequences took 12.5 us from Python with the
 * checks there and ctypes (2.4 us for its 28 arguments), most of it not the launch.
 *
 * Each function returns the entry point's status, or -1 if a check fails; ops.py then says what is wrong. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "pkv.h"

static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_is_contiguous;
static PyObject *dt_bf16, *dt_i32, *dt_f32, *dt_int8, *dt_e4m3;

typedef int (*append_fn)(void*, int64_t, int64_t, const void*, int64_t, int64_t, const void*, int64_t, int64_t,
                         const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*, int64_t, void*, void*,
                         float*, float*, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int, double, void*);
typedef int (*read_fn)(const void*, const void*, const float*, const float*, int64_t, int64_t, const int32_t*, int64_t,
                       int64_t, const int32_t*, const int32_t*, int64_t, void*, int64_t, int64_t, void*, int64_t,
                       int64_t, int64_t, int64_t, int64_t, int, void*);
typedef int (*attention_fn)(const void*, int64_t, int64_t, const void*, const void*, const float*, const float*, int64_t,
                            int64_t, const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*, int64_t, void*,
                            int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int, float, void*, size_t, void*,
                            const pkv_attention_options*);
static append_fn f_append;
static read_fn f_read;
static attention_fn f_attention;

typedef struct {
  void* ptr;
  int64_t size[4], stride[4];
} Tensor;

static int int_of(PyObject* o, long long* v) { /* steals o */
  if (!o) return 0;
  *v = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return !(*v == -1 && PyErr_Occurred());
}

static int tuple_of(PyObject* o, int n, int64_t* v) { /* steals o */
  if (!o) return 0;
  int ok = PyTuple_Check(o) && PyTuple_GET_SIZE(o) == n;
  for (int i = 0; ok && i < n; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
    ok = !(v[i] == -1 && PyErr_Occurred());
  }
  Py_DECREF(o);
  return ok;
}

/* A tensor of `nd` dimensions on device `dev`, of type `dt` (NULL: any, returned in *got); contiguous, or with
 * its strides read. */
static int tensor_of(PyObject* t, int nd, PyObject* dt, PyObject** got, int strides, long dev, Tensor* o) {
  PyObject* x = PyObject_GetAttr(t, s_dtype);
  if (!x) return 0;
  if (got) *got = x; /* (a type object lives on: only compared) */
  const int same = dt == NULL || x == dt;
  Py_DECREF(x);
  long long v;
  if (!same || !int_of(PyObject_CallMethodNoArgs(t, s_get_device), &v) || v != dev) return 0;
  if (!tuple_of(PyObject_GetAttr(t, s_shape), nd, o->size)) return 0;
  if (strides) {
    if (!tuple_of(PyObject_CallMethodNoArgs(t, s_stride), nd, o->stride)) return 0;
  } else {
    x = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!x) return 0;
    const int yes = x == Py_True;
    Py_DECREF(x);
    if (!yes) return 0;
  }
  if (!int_of(PyObject_CallMethodNoArgs(t, s_data_ptr), &v)) return 0;
  o->ptr = (void*)(intptr_t)v;
  return 1;
}

typedef struct {
  Tensor k, v, ks, vs, table, ctx, start;
  int format;
  int64_t seqs, table_stride, max_blocks;
} Cache;

/* k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, start_loc = a[0 .. 6] */
static int cache_of(PyObject* const* a, PyObject* max_blocks, long dev, Cache* c) {
  PyObject* dt = NULL;
  if (!tensor_of(a[0], 4, NULL, &dt, 0, dev, &c->k)) return 0;
  c->format = dt == dt_int8 ? PKV_Q8_INT8 : dt == dt_e4m3 ? PKV_Q8_E4M3 : 0;
  if (!c->format || !tensor_of(a[1], 4, dt, NULL, 0, dev, &c->v)) return 0;
  for (int i = 0; i < 4; ++i)
    if (c->v.size[i] != c->k.size[i]) return 0;
  if (!tensor_of(a[2], 2, dt_f32, NULL, 0, dev, &c->ks) || !tensor_of(a[3], 2, dt_f32, NULL, 0, dev, &c->vs)) return 0;
  if (c->ks.size[0] != c->k.size[0] || c->ks.size[1] != c->k.size[2] || c->vs.size[0] != c->k.size[0] ||
      c->vs.size[1] != c->k.size[2])
    return 0;
  if (!tensor_of(a[4], 2, dt_i32, NULL, 1, dev, &c->table) || !tensor_of(a[5], 1, dt_i32, NULL, 0, dev, &c->ctx) ||
      !tensor_of(a[6], 1, dt_i32, NULL, 0, dev, &c->start))
    return 0;
  c->seqs = c->ctx.size[0];
  const int64_t width = c->table.size[1];
  if (c->table.size[0] != c->seqs || c->start.size[0] != c->seqs + 1) return 0;
  if (c->table.stride[1] != 1 && width > 1) return 0;
  c->table_stride = c->seqs > 1 ? c->table.stride[0] : width; /* (a single row's stride is never used) */
  c->max_blocks = width;
  if (max_blocks != Py_None) {
    c->max_blocks = PyLong_AsLongLong(max_blocks);
    if (PyErr_Occurred() || c->max_blocks > width) return 0;
  }
  return 1;
}

/* [rows, heads, d] bf16 with contiguous rows; sizes as given where not negative */
static int rows_of(PyObject* t, int64_t rows, int64_t heads, int64_t d, long dev, Tensor* o) {
  return tensor_of(t, 3, dt_bf16, NULL, 1, dev, o) && o->stride[2] == 1 && (rows < 0 || o->size[0] == rows) &&
         (heads < 0 || o->size[1] == heads) && (d < 0 || o->size[2] == d);
}

static PyObject* refused(void) {
  PyErr_Clear();
  return PyLong_FromLong(-1);
}

/* append(q, k, v, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start_loc, rope_theta,
 *        max_blocks_per_seq, stream, device) */
static PyObject* call_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Tensor q, k, v;
  Cache c;
  if (n != 14) return refused();
  const long dev = PyLong_AsLong(a[13]);
  const double theta = PyFloat_AsDouble(a[10]);
  void* stream = PyLong_AsVoidPtr(a[12]);
  if (PyErr_Occurred() || !cache_of(a + 3, a[11], dev, &c) || !rows_of(a[0], -1, -1, c.k.size[3], dev, &q) ||
      !rows_of(a[1], q.size[0], c.k.size[2], c.k.size[3], dev, &k) ||
      !rows_of(a[2], q.size[0], c.k.size[2], c.k.size[3], dev, &v))
    return refused();
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f_append(q.ptr, q.stride[0], q.stride[1], k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1],
                c.table.ptr, c.table_stride, c.max_blocks, c.ctx.ptr, c.start.ptr, c.seqs, c.k.ptr, c.v.ptr, c.ks.ptr,
                c.vs.ptr, q.size[0], q.size[1], c.k.size[2], c.k.size[3], c.k.size[0], c.k.size[1], c.format, theta, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* read(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, read_start_loc, k_out, v_out,
 *      max_blocks_per_seq, stream, device) */
static PyObject* call_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Tensor k, v;
  Cache c;
  if (n != 12) return refused();
  const long dev = PyLong_AsLong(a[11]);
  void* stream = PyLong_AsVoidPtr(a[10]);
  if (PyErr_Occurred() || !cache_of(a, a[9], dev, &c) || !rows_of(a[7], -1, c.k.size[2], c.k.size[3], dev, &k) ||
      !rows_of(a[8], k.size[0], c.k.size[2], c.k.size[3], dev, &v))
    return refused();
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f_read(c.k.ptr, c.v.ptr, c.ks.ptr, c.vs.ptr, c.k.size[0], c.k.size[1], c.table.ptr, c.table_stride, c.max_blocks,
              c.ctx.ptr, c.start.ptr, c.seqs, k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1], k.size[0],
              c.k.size[2], c.k.size[3], c.format, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start_loc, out, workspace, scale,
 *           max_blocks_per_seq, options, stream, device); options: the address of a pkv_attention_options, or 0 */
static PyObject* call_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Tensor q, o, w;
  Cache c;
  if (n != 15) return refused();
  const long dev = PyLong_AsLong(a[14]);
  const double scale = PyFloat_AsDouble(a[10]);
  const pkv_attention_options* opt = PyLong_AsVoidPtr(a[12]);
  void* stream = PyLong_AsVoidPtr(a[13]);
  PyObject* wt = NULL;
  if (PyErr_Occurred() || !cache_of(a + 1, a[11], dev, &c) || !rows_of(a[0], -1, -1, c.k.size[3], dev, &q) ||
      !rows_of(a[8], q.size[0], q.size[1], q.size[2], dev, &o) || !tensor_of(a[9], 1, NULL, &wt, 0, dev, &w))
    return refused();
  int st;
  Py_BEGIN_ALLOW_THREADS;
  /* (a workspace of wider elements than bytes counts as its elements: never more than it holds) */
  st = f_attention(q.ptr, q.stride[0], q.stride[1], c.k.ptr, c.v.ptr, c.ks.ptr, c.vs.ptr, c.k.size[0], c.k.size[1],
                   c.table.ptr, c.table_stride, c.max_blocks, c.ctx.ptr, c.start.ptr, c.seqs, o.ptr, o.stride[0],
                   o.stride[1], q.size[0], q.size[1], c.k.size[2], c.k.size[3], c.format, (float)scale, w.ptr,
                   (size_t)w.size[0], stream, opt);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* bind(bfloat16, int32, float32, int8, float8_e4m3fn, addresses of the three entry points) */
static PyObject* bind(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long pa, pr, pt;
  PyObject *b, *i, *f, *c, *e;
  if (!PyArg_ParseTuple(args, "OOOOOKKK", &b, &i, &f, &c, &e, &pa, &pr, &pt)) return NULL;
  Py_INCREF(b), Py_INCREF(i), Py_INCREF(f), Py_INCREF(c), Py_INCREF(e);
  dt_bf16 = b, dt_i32 = i, dt_f32 = f, dt_int8 = c, dt_e4m3 = e;
  f_append = (append_fn)(uintptr_t)pa;
  f_read = (read_fn)(uintptr_t)pr;
  f_attention = (attention_fn)(uintptr_t)pt;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, NULL},
                                {"append", (PyCFunction)(void (*)(void))call_append, METH_FASTCALL, NULL},
                                {"read", (PyCFunction)(void (*)(void))call_read, METH_FASTCALL, NULL},
                                {"attention", (PyCFunction)(void (*)(void))call_attention, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__q8call(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device || !s_is_contiguous) return NULL;
  return PyModule_Create(&module);
}
