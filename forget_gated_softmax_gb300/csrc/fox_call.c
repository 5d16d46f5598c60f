/* The serving calls of libfox.so for Python: fox_cache_append_low, fox_decode and those of the 4-bit cache, with plain
 * numbers (addresses, sizes, strides), which the binding has checked. A step of generation is some microseconds of GPU time; ctypes
 * takes two of them to convert a dozen arguments, these functions a tenth of that. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/fox.h"

typedef fox_status (*append_fn)(const fox_cache*, const fox_batch*, int, const void*, int64_t, const void*, int64_t,
                                const float*, int64_t, const fox_rotary*, float*, void*, size_t, void*);
typedef fox_status (*decode_fn)(const fox_cache*, const fox_batch*, int, const void*, int64_t, float, int, void*, float*,
                                void*, size_t, void*);
typedef fox_status (*append4_fn)(const fox_cache4*, const fox_batch*, int, const void*, int64_t, const void*, int64_t,
                                 const float*, int64_t, const fox_rotary*, void*, size_t, void*);
typedef fox_status (*decode4_fn)(const fox_cache4*, const fox_batch*, int, const void*, int64_t, float, int, void*, float*,
                                 void*, size_t, void*);
typedef fox_status (*read4_fn)(const fox_cache4*, const fox_batch*, int, void*, int64_t, void*, int64_t, void*, size_t, void*);
static append_fn g_append;
static decode_fn g_decode;
static append4_fn g_append4;
static decode4_fn g_decode4;
static read4_fn g_read4;

static void* ptr(PyObject* x) { return (void*)(uintptr_t)PyLong_AsUnsignedLongLong(x); }
static int64_t num(PyObject* x) { return (int64_t)PyLong_AsLongLong(x); }
static int small(PyObject* x) {
  const int overflow = 0x7fffffff;
  const long long v = PyLong_AsLongLong(x);
  if (!PyErr_Occurred() && (v > overflow || v < -overflow)) PyErr_SetString(PyExc_OverflowError, "does not fit an int");
  return (int)v;
}

static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes 5 addresses");
  append_fn f = (append_fn)ptr(a[0]);
  decode_fn g = (decode_fn)ptr(a[1]);
  append4_fn f4 = (append4_fn)ptr(a[2]);
  decode4_fn g4 = (decode4_fn)ptr(a[3]);
  read4_fn r4 = (read4_fn)ptr(a[4]);
  if (PyErr_Occurred()) return NULL;
  g_append = f;
  g_decode = g;
  g_append4 = f4;
  g_decode4 = g4;
  g_read4 = r4;
  Py_RETURN_NONE;
}

/* cache, batch, rows, k, k_stride, v, v_stride, z, z_stride, ws, ws_bytes, stream[, cos, sin, positions, dim, pairs, q,
 * q_stride, q_out][, g_low] */
static PyObject* append_to(PyObject* const* a, Py_ssize_t n, int four) {
  const Py_ssize_t m = !four && (n == 13 || n == 21) ? n - 1 : n;  /* without g_low */
  if ((m != 12 && m != 20) || !(four ? g_append4 != NULL : g_append != NULL))
    return PyErr_Format(PyExc_TypeError, "append takes 12 or 20 numbers, and perhaps one more, after bind; append4 12 or 20");
  const void* c = ptr(a[0]);
  const fox_batch* b = (const fox_batch*)ptr(a[1]);
  const int rows = small(a[2]);
  const void *k = ptr(a[3]), *v = ptr(a[5]);
  const float* z = (const float*)ptr(a[7]);
  const int64_t ks = num(a[4]), vs = num(a[6]), zs = num(a[8]);
  void *ws = ptr(a[9]), *stream = ptr(a[11]);
  const size_t bytes = (size_t)PyLong_AsUnsignedLongLong(a[10]);
  fox_rotary r = {0};
  float* low = m < n ? (float*)ptr(a[m]) : NULL;
  if (m == 20) {
    r.cos = (const float*)ptr(a[12]);
    r.sin = (const float*)ptr(a[13]);
    r.max_pos = small(a[14]);
    r.dim = small(a[15]);
    r.pairs = small(a[16]);
    r.q = ptr(a[17]);
    r.q_stride = num(a[18]);
    r.q_out = ptr(a[19]);
  }
  if (PyErr_Occurred()) return NULL;
  fox_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = four ? g_append4((const fox_cache4*)c, b, rows, k, ks, v, vs, z, zs, m == 20 ? &r : NULL, ws, bytes, stream)
            : g_append((const fox_cache*)c, b, rows, k, ks, v, vs, z, zs, m == 20 ? &r : NULL, low, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)st);
}
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return append_to(a, n, 0);
}
static PyObject* append4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return append_to(a, n, 1);
}

/* cache, batch, rows, q, q_stride, scale, bias_from_j, o, lse, ws, ws_bytes, stream */
static PyObject* decode_over(PyObject* const* a, Py_ssize_t n, int four) {
  if (n != 12 || !(four ? g_decode4 != NULL : g_decode != NULL))
    return PyErr_Format(PyExc_TypeError, "decode and decode4 take 12 numbers, after bind");
  const void* c = ptr(a[0]);
  const fox_batch* b = (const fox_batch*)ptr(a[1]);
  const int rows = small(a[2]), from_j = small(a[6]);
  const void* q = ptr(a[3]);
  const int64_t qs = num(a[4]);
  const float scale = (float)PyFloat_AsDouble(a[5]);
  void *o = ptr(a[7]), *lse = ptr(a[8]), *ws = ptr(a[9]), *stream = ptr(a[11]);
  const size_t bytes = (size_t)PyLong_AsUnsignedLongLong(a[10]);
  if (PyErr_Occurred()) return NULL;
  fox_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = four ? g_decode4((const fox_cache4*)c, b, rows, q, qs, scale, from_j, o, (float*)lse, ws, bytes, stream)
            : g_decode((const fox_cache*)c, b, rows, q, qs, scale, from_j, o, (float*)lse, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)st);
}
static PyObject* decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return decode_over(a, n, 0);
}
static PyObject* decode4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return decode_over(a, n, 1);
}

/* cache, batch, rows, k, k_stride, v, v_stride, ws, ws_bytes, stream */
static PyObject* read4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 10 || !g_read4) return PyErr_Format(PyExc_TypeError, "read4 takes 10 numbers, after bind");
  const fox_cache4* c = (const fox_cache4*)ptr(a[0]);
  const fox_batch* b = (const fox_batch*)ptr(a[1]);
  const int rows = small(a[2]);
  void *k = ptr(a[3]), *v = ptr(a[5]), *ws = ptr(a[7]), *stream = ptr(a[9]);
  const int64_t ks = num(a[4]), vs = num(a[6]);
  const size_t bytes = (size_t)PyLong_AsUnsignedLongLong(a[8]);
  if (PyErr_Occurred()) return NULL;
  fox_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_read4(c, b, rows, k, ks, v, vs, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)st);
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, "bind(fox_cache_append_low, fox_decode, fox_cache4_append, fox_cache4_decode, fox_cache4_read): their addresses"},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, "fox_cache_append_low; returns its status"},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, "fox_decode; returns its status"},
    {"append4", (PyCFunction)(void (*)(void))append4, METH_FASTCALL, "fox_cache4_append; returns its status"},
    {"decode4", (PyCFunction)(void (*)(void))decode4, METH_FASTCALL, "fox_cache4_decode; returns its status"},
    {"read4", (PyCFunction)(void (*)(void))read4, METH_FASTCALL, "fox_cache4_read; returns its status"},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_foxcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__foxcall(void) { return PyModule_Create(&module); }
