/* Descriptors of torch tensors for the Python binding: reads a tensor's address, type,
 * shape and strides through its own attributes and writes the library's tp_tensor.
 * A call's descriptors are most of a small call's issue time: 0.9 us a tensor when
 * they are packed by interpreted code, and a one-token projection has eighteen.
 *
 * Only what needs no words is taken here: a CUDA tensor of a type that the library
 * knows, not empty, with unit column stride. Everything else (and every error) is
 * left to the caller, which gets a false result and no exception. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "tpgqa.h"

static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_stride, *s_data_ptr;
static PyObject *known[3]; /* by tp_dtype: the type objects, which live as long as torch does */

/* The long long items of a tuple attribute or result (a reference that this takes). */
static int items(PyObject *t, long long *out, Py_ssize_t n) {
  int ok = t != NULL && PyTuple_Check(t) && PyTuple_GET_SIZE(t) == n;
  for (Py_ssize_t i = 0; ok && i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    ok = out[i] >= 0; /* -1 with an exception, too */
  }
  Py_XDECREF(t);
  return ok;
}

static int describe(PyObject *t, Py_ssize_t dims, tp_tensor *d) {
  PyObject *v = PyObject_GetAttr(t, s_dtype);
  int type = 0;
  while (type < 3 && (v == NULL || v != known[type])) ++type;
  Py_XDECREF(v);
  if (type == 3) return 0;
  v = PyObject_GetAttr(t, s_is_cuda);
  const int cuda = v == Py_True;
  Py_XDECREF(v);
  long long shape[2] = {1, 1}, stride[2] = {1, 1};
  if (!cuda || !items(PyObject_GetAttr(t, s_shape), shape + 2 - dims, dims)) return 0;
  if (shape[0] == 0 || shape[1] == 0) return 0;
  if (!items(PyObject_CallMethodNoArgs(t, s_stride), stride + 2 - dims, dims) || stride[1] != 1) return 0;
  v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  const unsigned long long ptr = v != NULL && PyLong_Check(v) ? PyLong_AsUnsignedLongLong(v) : 0;
  Py_XDECREF(v);
  if (ptr == 0 || ptr == ~0ull) return 0; /* the latter with an exception */
  memset(d, 0, sizeof(*d));
  d->ptr = (void *)(uintptr_t)ptr;
  d->dtype = type;
  d->rows = shape[0];
  d->cols = shape[1];
  /* the pitch of a single row is free */
  d->ld = shape[0] > 1 || stride[0] > shape[1] ? stride[0] : shape[1];
  return 1;
}

static PyObject *truth(int ok) {
  if (!ok) PyErr_Clear();
  return PyBool_FromLong(ok);
}
static tp_tensor *address(PyObject *v) { return (tp_tensor *)PyLong_AsVoidPtr(v); }

static PyObject *py_matrix(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "matrix(tensor, address)");
  tp_tensor *to = address(args[1]);
  if (to == NULL) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "a null address");
  return truth(describe(args[0], 2, to));
}

static PyObject *py_row(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "row(tensor, address)");
  tp_tensor *to = address(args[1]);
  if (to == NULL) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "a null address");
  return truth(describe(args[0], 1, to));
}

static PyObject *py_matrices(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 3) return PyErr_Format(PyExc_TypeError, "matrices(sequence, count, address)");
  const Py_ssize_t count = PyLong_AsSsize_t(args[1]);
  tp_tensor *to = address(args[2]);
  if (PyErr_Occurred()) return NULL;
  Py_ssize_t done = 0;
  if (to != NULL && (PyList_Check(args[0]) || PyTuple_Check(args[0]))) {
    /* attributes run the tensor's own code, so the sequence's length is read anew each time */
    while (done < count && done < PySequence_Fast_GET_SIZE(args[0])) {
      PyObject *t = PySequence_Fast_GET_ITEM(args[0], done);
      Py_INCREF(t);
      const int ok = describe(t, 2, to + done);
      Py_DECREF(t);
      if (!ok) {
        PyErr_Clear();
        break;
      }
      ++done;
    }
  }
  return PyLong_FromSsize_t(done);
}

static PyObject *py_dtypes(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 3) return PyErr_Format(PyExc_TypeError, "dtypes(f32, bf16, e4m3)");
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(args[i]);
    Py_XSETREF(known[i], args[i]);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"dtypes", (PyCFunction)(void (*)(void))py_dtypes, METH_FASTCALL, "dtypes(f32, bf16, e4m3): the type objects of TP_F32, TP_BF16, TP_E4M3"},
    {"matrix", (PyCFunction)(void (*)(void))py_matrix, METH_FASTCALL, "matrix(tensor, address) -> whether it was described there"},
    {"row", (PyCFunction)(void (*)(void))py_row, METH_FASTCALL, "row(tensor, address): a 1-D tensor as a matrix of one row"},
    {"matrices", (PyCFunction)(void (*)(void))py_matrices, METH_FASTCALL, "matrices(sequence, count, address) -> how many of the first were described"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_describe", "Descriptors of torch tensors.", -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__describe(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_is_cuda || !s_shape || !s_stride || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
