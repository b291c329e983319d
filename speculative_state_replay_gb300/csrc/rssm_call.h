/* rssm_call.h -- how the binding's C modules take their arguments and give a call's status. */
#ifndef RSSM_CALL_H
#define RSSM_CALL_H

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

#endif /* RSSM_CALL_H */
