/* rssm_call.c -- the binding's fast path into librssm.
 *
 * A decode step's small calls are bound by the host.  For the operators that
 * such a step makes most of, this module takes the arguments that api.py has
 * checked -- integers, addresses as integers, floats -- and makes the C call;
 * marshalling 15 to 22 arguments through ctypes takes 1.5 to 2.5 us, here a
 * tenth of that.  It computes nothing.  device() says where a call's tensors are
 * (a loop over them in Python took 0.9 us longer for a step).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "rssm.h"

static void *as_ptr(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }
#define P(i) as_ptr(args[i])
static int32_t as_i32(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v != (int32_t)v) PyErr_SetString(PyExc_OverflowError, "an argument is outside 32 bits");
  return (int32_t)v;
}
#define I32(i) as_i32(args[i])
#define I64(i) ((int64_t)PyLong_AsLongLong(args[i]))
#define F32(i) ((float)PyFloat_AsDouble(args[i]))

/* arguments are read first: a value of another kind raises before the call */
#define TAKE(n)                                                                        \
  if (nargs != (n)) {                                                                  \
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", (n), nargs);       \
    return NULL;                                                                       \
  }
/* other threads run meanwhile: a launch may wait (for room in the queue, or behind a host callback that needs the lock) */
#define GIVE(call)                                                                     \
  do {                                                                                 \
    long status;                                                                       \
    if (PyErr_Occurred()) return NULL;                                                 \
    Py_BEGIN_ALLOW_THREADS status = (long)(call);                                      \
    Py_END_ALLOW_THREADS return PyLong_FromLong(status);                               \
  } while (0)

static PyObject *delta_step(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(21)
  const rssm_delta_cache *c = P(0);
  const void *q = P(1), *k = P(3), *v = P(5);
  const int64_t qs = I64(2), ks = I64(4), vs = I64(6);
  const float *g = P(7), *beta = P(8);
  const float scale = F32(9);
  const int32_t l2 = I32(10);
  const int32_t *slots = P(11), *acc = P(12), *cu = P(13);
  const int32_t batch = I32(14), T = I32(15);
  const int64_t tokens = I64(16);
  void *out = P(17), *scratch = P(18);
  const int64_t bytes = I64(19);
  void *stream = P(20);
  GIVE(rssm_delta_step(c, q, qs, k, ks, v, vs, g, beta, scale, l2, slots, acc, cu, batch, T, tokens, out, scratch,
                       (size_t)bytes, stream));
}

static PyObject *delta_prefill(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(20)
  const rssm_delta_cache *c = P(0);
  const void *q = P(1), *k = P(3), *v = P(5);
  const int64_t qs = I64(2), ks = I64(4), vs = I64(6);
  const float *g = P(7), *beta = P(8);
  const float scale = F32(9);
  const int32_t l2 = I32(10);
  const int32_t *slots = P(11), *cu = P(12), *initial = P(13);
  const int32_t batch = I32(14);
  const int64_t tokens = I64(15);
  void *out = P(16), *scratch = P(17);
  const int64_t bytes = I64(18);
  void *stream = P(19);
  GIVE(rssm_delta_prefill(c, q, qs, k, ks, v, vs, g, beta, scale, l2, slots, cu, initial, batch, tokens, out, scratch,
                          (size_t)bytes, stream));
}

static PyObject *verify(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(17)
  const void *target = P(0), *draft = P(2);
  const int64_t ts = I64(1), ds = I64(3);
  const int32_t dtype = I32(4), vocab = I32(5);
  const int32_t *tokens = P(6);
  const float *u = P(7), *un = P(8);
  const int32_t *cu = P(9);
  const int32_t batch = I32(10), T = I32(11);
  const int64_t ntok = I64(12);
  int32_t *acc = P(13), *next = P(14);
  uint32_t *word = P(15);
  void *stream = P(16);
  GIVE(rssm_verify(target, ts, draft, ds, dtype, vocab, tokens, u, un, cu, batch, T, ntok, acc, next, word, stream));
}

static PyObject *gated_norm(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(15)
  const void *x = P(0), *z = P(2);
  const int64_t xs = I64(1), zs = I64(3);
  const int32_t dtype = I32(4);
  const float *w = P(5);
  const int32_t shared = I32(6);
  const int64_t rows = I64(7);
  const int32_t dim = I32(8), group = I32(9);
  const float eps = F32(10);
  const int32_t first = I32(11);
  void *out = P(12);
  const int64_t os = I64(13);
  void *stream = P(14);
  GIVE(rssm_gated_norm(x, xs, z, zs, dtype, w, shared, rows, dim, group, eps, first, out, os, stream));
}

static PyObject *residual_norm(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(18)
  const void *x = P(0), *r = P(2);
  const int64_t xs = I64(1), rs = I64(3);
  const int32_t dtype = I32(4), rdtype = I32(5);
  const float *post = P(6), *scale = P(7);
  const float alpha = F32(8);
  const float *w = P(9);
  const int64_t rows = I64(10);
  const int32_t dim = I32(11);
  const float eps = F32(12);
  void *ro = P(13);
  const int64_t ros = I64(14);
  void *out = P(15);
  const int64_t os = I64(16);
  void *stream = P(17);
  GIVE(rssm_residual_norm(x, xs, r, rs, dtype, rdtype, post, scale, alpha, w, rows, dim, eps, ro, ros, out, os, stream));
}

static PyObject *get_device_name;

/* device(tensor or None, ...): the CUDA device that all tensors are on; -1 if one is not on any, or on another one */
static PyObject *device(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  long all = -1;
  int any = 0;
  for (Py_ssize_t i = 0; i < nargs; ++i) {
    if (args[i] == Py_None) continue;
    PyObject *r = PyObject_CallMethodNoArgs(args[i], get_device_name);
    if (!r) return NULL;
    const long d = PyLong_AsLong(r);
    Py_DECREF(r);
    if (d == -1 && PyErr_Occurred()) return NULL;
    if (any && d != all) return PyLong_FromLong(-1);
    any = 1;
    all = d;
  }
  return PyLong_FromLong(all);
}

static PyMethodDef methods[] = {
    {"device", (PyCFunction)(void (*)(void))device, METH_FASTCALL, NULL},
    {"rssm_delta_step", (PyCFunction)(void (*)(void))delta_step, METH_FASTCALL, NULL},
    {"rssm_delta_prefill", (PyCFunction)(void (*)(void))delta_prefill, METH_FASTCALL, NULL},
    {"rssm_verify", (PyCFunction)(void (*)(void))verify, METH_FASTCALL, NULL},
    {"rssm_gated_norm", (PyCFunction)(void (*)(void))gated_norm, METH_FASTCALL, NULL},
    {"rssm_residual_norm", (PyCFunction)(void (*)(void))residual_norm, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "C calls into librssm with checked arguments", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__call(void) {
  get_device_name = PyUnicode_InternFromString("get_device");
  return get_device_name ? PyModule_Create(&module) : NULL;
}
