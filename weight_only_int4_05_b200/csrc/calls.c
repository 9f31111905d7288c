/*
 * calls.c -- the 8-bit operators' entry points as CPython functions (module _calls).
 *
 * Argument marshalling alone, for calls whose kernels take a few microseconds: a foreign-function call with 7 to 17 arguments
 * costs 0.8 to 1.7 us, this one 0.17 (0.06 of it for the lock).  Each function takes the C arguments in order (addresses as whole numbers, None for
 * NULL) and returns the status code.  Linked against libawq_w4a16.so beside it; no torch type appears.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

#include "awq_w4a16.h"

static void* as_ptr(PyObject* o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }

static int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if ((v > INT_MAX || v < INT_MIN) && !PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "argument does not fit an int");
  return (int)v;
}

static int count_ok(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
  return 0;
}

#define P(i) as_ptr(a[i])
#define I(i) as_int(a[i])
/* The arguments are converted before the call and an error among them refuses it.  The call itself runs without the
 * interpreter's lock: a launch may wait for room in the stream's queue, and a host function in that stream for the lock. */
#define CALL(expr)                     \
  do {                                 \
    long status;                       \
    if (PyErr_Occurred()) return NULL; \
    Py_BEGIN_ALLOW_THREADS             \
    status = (long)(expr);             \
    Py_END_ALLOW_THREADS               \
    return PyLong_FromLong(status);    \
  } while (0)

static PyObject* py_fp8_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!count_ok(n, 7)) return NULL;
  void *x = P(0), *codes = P(4), *scales = P(5), *st = P(6);
  const int dt = I(1), R = I(2), K = I(3);
  CALL(fp8_quantize(x, dt, R, K, codes, scales, st));
}

static PyObject* py_w8a8_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!count_ok(n, 10)) return NULL;
  void *xc = P(0), *xs = P(1), *wc = P(2), *ws = P(3), *y = P(4), *st = P(9);
  const int dt = I(5), M = I(6), N = I(7), K = I(8);
  CALL(w8a8_gemm(xc, xs, wc, ws, y, dt, M, N, K, st));
}

static PyObject* py_w8a8_linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!count_ok(n, 11)) return NULL;
  void *x = P(0), *wc = P(2), *ws = P(3), *y = P(4), *work = P(8), *st = P(10);
  const int dt = I(1), M = I(5), N = I(6), K = I(7);
  const size_t bytes = PyLong_AsSize_t(a[9]);
  CALL(w8a8_linear(x, dt, wc, ws, y, M, N, K, work, bytes, st));
}

static PyObject* py_moe_route(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!count_ok(n, 14)) return NULL;
  void *logits = P(0), *bias = P(2), *ids = P(11), *weights = P(12), *st = P(13);
  const int dt = I(1), M = I(3), E = I(4), topk = I(5), score = I(6), groups = I(7), topk_groups = I(8), renorm = I(9);
  const float scale = (float)PyFloat_AsDouble(a[10]);
  CALL(moe_route(logits, dt, bias, M, E, topk, score, groups, topk_groups, renorm, scale, ids, weights, st));
}

static PyObject* py_w8a8_moe(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!count_ok(n, 18)) return NULL;
  void *x = P(0), *ids = P(2), *weights = P(3), *gc = P(4), *gs = P(5), *dc = P(6), *ds = P(7), *y = P(8);
  const int dt = I(1), M = I(9), E = I(10), topk = I(11), K = I(12), width = I(13), N = I(14);
  void *work = P(15), *st = P(17);
  const size_t bytes = PyLong_AsSize_t(a[16]);
  CALL(w8a8_moe(x, dt, ids, weights, gc, gs, dc, ds, y, M, E, topk, K, width, N, work, bytes, st));
}

#define FUNCTION(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef functions[] = {FUNCTION(fp8_quantize), FUNCTION(w8a8_gemm), FUNCTION(w8a8_linear), FUNCTION(moe_route),
                                  FUNCTION(w8a8_moe), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, functions, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
