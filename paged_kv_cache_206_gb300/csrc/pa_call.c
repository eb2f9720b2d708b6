/*
 * A Python module of one function: call(address, *arguments) -> int calls a C
 * function that takes pointers and 64-bit integers and returns an int. Arguments
 * are Python integers, or None for NULL. ctypes does the same in ten times the time
 * (3 to 5 us for the 13 to 24 arguments of the serving calls, as long as the
 * launches themselves take).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#define MAX_ARGS 24
typedef uint64_t u;

static PyObject* call(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  u v[MAX_ARGS + 1];
  int r = 0;
  (void)self;
  if (n < 1 || n > MAX_ARGS + 1) {
    PyErr_SetString(PyExc_TypeError, "call() takes an address and at most 24 arguments");
    return NULL;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (args[i] == Py_None) {
      v[i] = 0;
      continue;
    }
    v[i] = PyLong_AsUnsignedLongLongMask(args[i]);
    if (v[i] == (u)-1 && PyErr_Occurred()) return NULL;
  }
  const uintptr_t f = (uintptr_t)v[0];
  const u* a = v + 1;
  int known = 1;
  Py_BEGIN_ALLOW_THREADS;
  switch (n - 1) {
    case 13:
      r = ((int (*)(u, u, u, u, u, u, u, u, u, u, u, u, u))f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8],
                                                              a[9], a[10], a[11], a[12]);
      break;
    case 14:
      r = ((int (*)(u, u, u, u, u, u, u, u, u, u, u, u, u, u))f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8],
                                                                 a[9], a[10], a[11], a[12], a[13]);
      break;
    case 15:
      r = ((int (*)(u, u, u, u, u, u, u, u, u, u, u, u, u, u, u))f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7],
                                                                    a[8], a[9], a[10], a[11], a[12], a[13], a[14]);
      break;
    case 23:
      r = ((int (*)(u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u))f)(
          a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13], a[14], a[15], a[16],
          a[17], a[18], a[19], a[20], a[21], a[22]);
      break;
    case 24:
      r = ((int (*)(u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u, u))f)(
          a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13], a[14], a[15], a[16],
          a[17], a[18], a[19], a[20], a[21], a[22], a[23]);
      break;
    default: known = 0;
  }
  Py_END_ALLOW_THREADS;
  if (!known) {
    PyErr_SetString(PyExc_TypeError, "call() of a number of arguments that no serving call has");
    return NULL;
  }
  return PyLong_FromLong(r);
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(address, *arguments) -> int"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_call", NULL, 0, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_pa_call(void) { return PyModule_Create(&module); }
