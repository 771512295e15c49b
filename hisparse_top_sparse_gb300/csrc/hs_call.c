/*
 * The binding's short way for calls that take microseconds: a tensor's checks and
 * the C call of one Python function in one native call. Each function here answers
 * with the C call's status, or with None where an argument is not plainly what it
 * takes (another device or type, a pinned tensor, a stream object, anything wrong):
 * the Python function then goes its own way, which checks argument by argument
 * and says what is the matter. Nothing is decided here that the long way would
 * decide otherwise.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "hisparse.h"

static PyObject *s_dtype, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_shape, *s_stride;
static PyObject *t_f32, *t_bf16, *t_i32, *t_i64, *t_u8;      /* torch dtypes */
static PyObject *f_device, *f_stream;                        /* current device, its current stream */

typedef int (*quant_fn)(const void *, int32_t, int64_t, int64_t, void *, int64_t, const int32_t *,
                        const int32_t *, int32_t, uint32_t *, hs_stream_t);
typedef int (*dequant_fn)(const void *, int64_t, void *, int32_t, int64_t, int64_t, const int32_t *,
                          const int32_t *, int32_t, uint32_t *, hs_stream_t);
typedef int (*attend_fn)(const void *, const void *, int64_t, const int32_t *, int32_t, int32_t, int32_t,
                         float, void *, float *, void *, size_t, uint32_t *, hs_stream_t);
typedef int (*rope_fn)(const void *, int64_t, int64_t, int64_t, void *, int64_t, int64_t, int64_t,
                       int32_t, const int32_t *, const int32_t *, const int32_t *, int32_t, int32_t,
                       int32_t, int32_t, int32_t, int32_t, const int64_t *, float, int32_t, uint32_t *,
                       hs_stream_t);

/* Every helper answers 1, or 0 (no Python error left set) where the long way is to be taken. */

static int lost(void) {
  PyErr_Clear();
  return 0;
}

static int whole(PyObject *o, int64_t *to) {
  if (!o || !PyLong_Check(o)) return 0;
  *to = PyLong_AsLongLong(o);
  return *to == -1 && PyErr_Occurred() ? lost() : 1;
}

static int method_whole(PyObject *t, PyObject *name, int64_t *to) {
  PyObject *r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return lost();
  const int ok = whole(r, to);
  Py_DECREF(r);
  return ok;
}

static int numbers(PyObject *t, PyObject *name, int call, int64_t *to, int most) {
  /* the numbers of a tuple, how many; -1: none */
  PyObject *r = call ? PyObject_CallMethodNoArgs(t, name) : PyObject_GetAttr(t, name);
  if (!r) {
    PyErr_Clear();
    return -1;
  }
  int n = -1;
  if (PyTuple_Check(r) && PyTuple_GET_SIZE(r) <= most) {
    n = (int)PyTuple_GET_SIZE(r);
    for (int i = 0; i < n; ++i)
      if (!whole(PyTuple_GET_ITEM(r, i), to + i)) {
        n = -1;
        break;
      }
  }
  Py_DECREF(r);
  return n;
}

/* a tensor's type: the dtype's borrowed identity (torch keeps its dtypes) */
static PyObject *type_of(PyObject *t) {
  PyObject *d = PyObject_GetAttr(t, s_dtype);
  if (!d) {
    PyErr_Clear();
    return NULL;
  }
  Py_DECREF(d);
  return d;
}

static int here(PyObject *t, int64_t device) {
  int64_t d;
  return method_whole(t, s_get_device, &d) && d == device;
}

static int contiguous(PyObject *t) {
  PyObject *r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!r) return lost();
  Py_DECREF(r);
  return r == Py_True;
}

/* pointer of a contiguous tensor of the device and the type (an empty one: NULL) */
static int on(PyObject *t, PyObject *type, int64_t device, void **to) {
  int64_t p;
  if (type_of(t) != type || !here(t, device) || !contiguous(t) || !method_whole(t, s_data_ptr, &p)) return 0;
  *to = (void *)(uintptr_t)p;
  return 1;
}

/* the same for int32 [n]; None: a NULL list (n as it was) */
static int list(PyObject *t, int64_t device, void **to, int64_t *n) {
  *to = NULL;
  if (t == Py_None) return 1;
  return on(t, t_i32, device, to) && numbers(t, s_shape, 0, n, 1) == 1;
}

static int word(PyObject *t, int64_t device, void **to) {
  int64_t n = 1;
  return list(t, device, to, &n) && n == 1;
}

static int device_and_stream(PyObject *stream, int64_t *device, hs_stream_t *to) {
  PyObject *d = PyObject_CallNoArgs(f_device);
  if (!d) return lost();
  int64_t s;
  int ok = whole(d, device);
  if (ok && stream == Py_None) {
    PyObject *r = PyObject_CallOneArg(f_stream, d);
    if (!r) {
      Py_DECREF(d);
      return lost();
    }
    ok = whole(r, &s);
    Py_DECREF(r);
  } else if (ok) {
    ok = whole(stream, &s);
  }
  Py_DECREF(d);
  if (ok) *to = (hs_stream_t)(uintptr_t)s;
  return ok;
}

static int real(PyObject *o, float *to) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return 0;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return lost();
  *to = (float)v;
  return 1;
}

static int wide_type(PyObject *t, int32_t *to) {
  PyObject *d = type_of(t);
  *to = d == t_f32 ? HS_LOGITS_F32 : HS_LOGITS_BF16;
  return d == t_f32 || d == t_bf16;
}

static int small(int64_t v) { return v >= 0 && v <= INT32_MAX; }

/* bf16 / f32 rows of 576 values, the rows any distance apart */
static int wide_rows(PyObject *t, int64_t device, void **p, int32_t *type, int64_t *stride, int64_t *rows) {
  int64_t s[2], st[2], a;
  if (!here(t, device) || !wide_type(t, type) || numbers(t, s_shape, 0, s, 2) != 2 ||
      numbers(t, s_stride, 1, st, 2) != 2 || s[1] != HS_LATENT_DIM || (s[0] > 0 && st[1] != 1) ||
      !method_whole(t, s_data_ptr, &a))
    return 0;
  *p = (void *)(uintptr_t)a;
  *stride = s[0] > 1 ? st[0] : HS_LATENT_DIM;
  *rows = s[0];
  return 1;
}

static int cache_rows(PyObject *t, int64_t device, int64_t row_bytes, void **p, int64_t *rows) {
  int64_t s[2];
  if (!on(t, t_u8, device, p) || numbers(t, s_shape, 0, s, 2) != 2 || s[1] != row_bytes) return 0;
  *rows = s[0];
  return 1;
}

static PyObject *answer(int rc) { return PyLong_FromLong(rc); }

/* (address, row_bytes, source, destination, src_slots, dst_slots, status, stream) */
static PyObject *rows_call(PyObject *const *a, Py_ssize_t n_args, int quant) {
  int64_t addr, row_bytes, device, stride, wide_n, cache_n, n = -1, m = -1;
  int32_t type;
  void *wide, *cache, *ss, *ds, *st;
  hs_stream_t stream;
  if (n_args != 8 || !whole(a[0], &addr) || !whole(a[1], &row_bytes) ||
      !device_and_stream(a[7], &device, &stream) ||
      !wide_rows(quant ? a[2] : a[3], device, &wide, &type, &stride, &wide_n) ||
      !cache_rows(quant ? a[3] : a[2], device, row_bytes, &cache, &cache_n) ||
      !list(a[4], device, &ss, &n) || !list(a[5], device, &ds, &m) || !word(a[6], device, &st))
    Py_RETURN_NONE;
  const int64_t src_rows = quant ? wide_n : cache_n, dst_rows = quant ? cache_n : wide_n;
  if (a[4] == Py_None) n = a[5] == Py_None ? src_rows : m;
  if ((a[5] != Py_None && m != n) || !small(n) || (a[4] == Py_None && n > src_rows) ||
      (a[5] == Py_None && n > dst_rows))
    Py_RETURN_NONE;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  if (quant)
    rc = ((quant_fn)(uintptr_t)addr)(wide, type, stride, wide_n, cache, cache_n, ss, ds, (int32_t)n, st, stream);
  else
    rc = ((dequant_fn)(uintptr_t)addr)(cache, cache_n, wide, type, stride, wide_n, ss, ds, (int32_t)n, st, stream);
  Py_END_ALLOW_THREADS
  return answer(rc);
}

static PyObject *call_quant(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(a, n, 1); }
static PyObject *call_dequant(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(a, n, 0); }

/* (address, row_bytes, q, kv, idx, scale, out, lse, workspace, status, stream) */
static PyObject *call_attend(PyObject *self, PyObject *const *a, Py_ssize_t n_args) {
  int64_t addr, row_bytes, device, q[3], o[3], i[2], l[2], rows, bytes = 0;
  float scale;
  void *pq, *pkv, *pi, *po, *pl = NULL, *pw = NULL, *st;
  hs_stream_t stream;
  if (n_args != 11 || !whole(a[0], &addr) || !whole(a[1], &row_bytes) ||
      !device_and_stream(a[10], &device, &stream) || !on(a[2], t_bf16, device, &pq) ||
      numbers(a[2], s_shape, 0, q, 3) != 3 || q[2] != HS_LATENT_DIM || !small(q[0]) || !small(q[1]) ||
      !cache_rows(a[3], device, row_bytes, &pkv, &rows) || !on(a[4], t_i32, device, &pi) ||
      numbers(a[4], s_shape, 0, i, 2) != 2 || i[0] != q[0] || !small(i[1]) || !real(a[5], &scale) ||
      !on(a[6], t_bf16, device, &po) || numbers(a[6], s_shape, 0, o, 3) != 3 || o[0] != q[0] ||
      o[1] != q[1] || o[2] != HS_VALUE_DIM || !word(a[9], device, &st))
    Py_RETURN_NONE;
  if (a[7] != Py_None && (!on(a[7], t_f32, device, &pl) || numbers(a[7], s_shape, 0, l, 2) != 2 ||
                          l[0] != q[0] || l[1] != q[1]))
    Py_RETURN_NONE;
  if (a[8] != Py_None) {
    if (!on(a[8], t_u8, device, &pw) || numbers(a[8], s_shape, 0, &bytes, 1) != 1) Py_RETURN_NONE;
  }
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = ((attend_fn)(uintptr_t)addr)(pq, pkv, rows, pi, (int32_t)q[0], (int32_t)q[1], (int32_t)i[1], scale, po,
                                    pl, pw, (size_t)bytes, st, stream);
  Py_END_ALLOW_THREADS
  return answer(rc);
}

/* rows [rows][heads][dims] or [rows][dims], dims contiguous */
static int heads_of(PyObject *t, int64_t device, void **p, int64_t s[3], int64_t st[3]) {
  int64_t a;
  const int n = here(t, device) ? numbers(t, s_shape, 0, s, 3) : -1;
  if (n < 2 || numbers(t, s_stride, 1, st, 3) != n || (st[n - 1] != 1 && s[n - 1] > 1) ||
      !method_whole(t, s_data_ptr, &a))
    return 0;
  if (n == 2) {
    s[2] = s[1];
    s[1] = 1;
    st[1] = 0;
  }
  *p = (void *)(uintptr_t)a;
  return 1;
}

/* (address, src, dst, positions, freqs, factor, rot_off, layout, inverse, src_slots, dst_slots,
    status, stream) */
static PyObject *call_rope(PyObject *self, PyObject *const *a, Py_ssize_t n_args) {
  int64_t addr, device, s[3], ss[3], d[3], ds[3], n, pairs, off, layout, k = -1, m = -1;
  float factor;
  int32_t type, type_d;
  void *ps, *pd, *pp, *pf, *ls, *ld, *st;
  hs_stream_t stream;
  if (n_args != 13 || !whole(a[0], &addr) || !device_and_stream(a[12], &device, &stream) ||
      !heads_of(a[1], device, &ps, s, ss) || !heads_of(a[2], device, &pd, d, ds) || !wide_type(a[1], &type) ||
      !wide_type(a[2], &type_d) || type != type_d || s[1] != d[1] || s[2] != d[2] || !small(s[1]) || !small(s[2]) ||
      a[3] == Py_None || !list(a[3], device, &pp, &n) || !small(n) || !on(a[4], t_i64, device, &pf) ||
      numbers(a[4], s_shape, 0, &pairs, 1) != 1 || pairs > 1 << 20 || !real(a[5], &factor) || !whole(a[6], &off) ||
      !whole(a[7], &layout) || (off > INT32_MAX || off < -1) || (layout > 2 || layout < -1) ||
      (a[8] != Py_True && a[8] != Py_False) || !list(a[9], device, &ls, &k) || !list(a[10], device, &ld, &m) ||
      !word(a[11], device, &st))
    Py_RETURN_NONE;
  if (a[9] != Py_None ? k != n : n > s[0] || (a[10] == Py_None && n < s[0])) Py_RETURN_NONE;
  if (a[10] != Py_None ? m != n : n > d[0]) Py_RETURN_NONE;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = ((rope_fn)(uintptr_t)addr)(ps, ss[0], ss[1], s[0], pd, ds[0], ds[1], d[0], type, ls, ld, pp, (int32_t)n,
                                  (int32_t)s[1], (int32_t)s[2], (int32_t)off, (int32_t)(2 * pairs),
                                  (int32_t)layout, pf, factor, a[8] == Py_True, st, stream);
  Py_END_ALLOW_THREADS
  return answer(rc);
}

/* (float32, bfloat16, int32, int64, uint8, current device, current raw stream of a device) */
static PyObject *call_setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  PyObject **const to[] = {&t_f32, &t_bf16, &t_i32, &t_i64, &t_u8, &f_device, &f_stream};
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "setup takes 7 arguments");
    return NULL;
  }
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*to[i], a[i]);
  }
  Py_RETURN_NONE;
}

#define FAST(f) ((PyCFunction)(void (*)(void))(f))
static PyMethodDef methods[] = {{"setup", FAST(call_setup), METH_FASTCALL, NULL},
                                {"quant", FAST(call_quant), METH_FASTCALL, NULL},
                                {"dequant", FAST(call_dequant), METH_FASTCALL, NULL},
                                {"attend", FAST(call_attend), METH_FASTCALL, NULL},
                                {"rope", FAST(call_rope), METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__call(void) {
  struct {
    PyObject **to;
    const char *name;
  } const names[] = {{&s_dtype, "dtype"},       {&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"},
                     {&s_data_ptr, "data_ptr"}, {&s_shape, "shape"},           {&s_stride, "stride"}};
  for (unsigned i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
