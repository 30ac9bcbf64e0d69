/* Descriptors of torch tensors for the Python binding: reads a tensor's address, type,
 * shape and strides through its own attributes and writes the library's tp_tensor.
 * A call's descriptors are most of a small call's issue time: 0.9 us a tensor when
 * they are packed by interpreted code, and a one-token projection has eighteen.
 *
 * Built with describe_torch.cpp, where torch's headers are, plain tensors are read without their attributes. That
 * holds for the torch of these headers alone: with any other at run time (reads_torch) the attributes are used.
 *
 * Only what needs no words is taken here: a CUDA tensor of a type that the library
 * knows, not empty, with unit column stride. Everything else (and every error) is
 * left to the caller, which gets a false result and no exception. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "tpgqa.h"

static int with_torch; /* whether the torch that runs is the one of the headers */
#ifdef TP_WITH_TORCH /* describe_torch.cpp */
#include "torch_version.h"
int tp_describe_torch(PyObject *t, long dims, int device, tp_tensor *d);
unsigned long long tp_address_torch(PyObject *t, int type, long long n, int device, unsigned long long *bytes);
#endif

static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_stride, *s_data_ptr;
static PyObject *known[4]; /* by tp_dtype: the type objects, which live as long as torch does */

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

/* device: the GPU on which the tensor must lie (another one's, or one not known, is left to the caller), -1: any. */
static int describe(PyObject *t, Py_ssize_t dims, int device, tp_tensor *d) {
#ifdef TP_WITH_TORCH
  const int done = with_torch ? tp_describe_torch(t, (long)dims, device, d) : -1;
  if (done >= 0) return done;
#endif
  if (device >= 0) return 0;
  PyObject *v = PyObject_GetAttr(t, s_dtype);
  int type = 0;
  while (type < 4 && (v == NULL || v != known[type])) ++type;
  Py_XDECREF(v);
  if (type == 4) return 0;
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

/* Argument i of n, a device; -1 where it is left out. */
static int device_of(PyObject *const *args, Py_ssize_t n, Py_ssize_t i) { return i < n ? (int)PyLong_AsLong(args[i]) : -1; }

static PyObject *py_matrix(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 2 && n != 3) return PyErr_Format(PyExc_TypeError, "matrix(tensor, address, device)");
  tp_tensor *to = address(args[1]);
  if (to == NULL) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "a null address");
  const int device = device_of(args, n, 2);
  if (PyErr_Occurred()) return NULL;
  return truth(describe(args[0], 2, device, to));
}

static PyObject *py_row(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "row(tensor, address)");
  tp_tensor *to = address(args[1]);
  if (to == NULL) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "a null address");
  return truth(describe(args[0], 1, -1, to));
}

static PyObject *py_matrices(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 3 && n != 4) return PyErr_Format(PyExc_TypeError, "matrices(sequence, count, address, device)");
  const Py_ssize_t count = PyLong_AsSsize_t(args[1]);
  if (PyErr_Occurred()) return NULL;
  tp_tensor *to = address(args[2]);
  if (PyErr_Occurred()) return NULL;
  const int device = device_of(args, n, 3);
  if (PyErr_Occurred()) return NULL;
  Py_ssize_t done = 0;
  if (to != NULL && (PyList_Check(args[0]) || PyTuple_Check(args[0]))) {
    /* attributes run the tensor's own code, so the sequence's length is read anew each time */
    while (done < count && done < PySequence_Fast_GET_SIZE(args[0])) {
      PyObject *t = PySequence_Fast_GET_ITEM(args[0], done);
      Py_INCREF(t);
      const int ok = describe(t, 2, device, to + done);
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

/* Addresses of contiguous CUDA tensors, or None where the caller has to look for itself. */
static PyObject *py_vector(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 3 && n != 4) return PyErr_Format(PyExc_TypeError, "vector(tensor, type, entries, device)");
  const long type = PyLong_AsLong(args[1]);
  if (PyErr_Occurred()) return NULL;
  const long long entries = PyLong_AsLongLong(args[2]);
  if (PyErr_Occurred()) return NULL;
  const int device = device_of(args, n, 3);
  if (PyErr_Occurred()) return NULL;
  unsigned long long at = 0, bytes = 0;
#ifdef TP_WITH_TORCH
  at = with_torch && type >= 0 ? tp_address_torch(args[0], (int)type, entries, device, &bytes) : 0;
#endif
  (void)type, (void)entries, (void)device, (void)bytes;
  if (at == 0) Py_RETURN_NONE;
  return PyLong_FromUnsignedLongLong(at);
}

static PyObject *py_bytes(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 1 && n != 2) return PyErr_Format(PyExc_TypeError, "bytes(tensor, device)");
  const int device = device_of(args, n, 1);
  if (PyErr_Occurred()) return NULL;
  unsigned long long at = 0, bytes = 0;
#ifdef TP_WITH_TORCH
  at = with_torch ? tp_address_torch(args[0], -1, -1, device, &bytes) : 0;
#endif
  (void)device;
  if (at == 0) Py_RETURN_NONE;
  return Py_BuildValue("KK", at, bytes);
}

/* Calls of the library with many arguments that take a few us: ctypes converts each argument by itself, 1 us a
 * call. The first argument is the entry point's address (this module does not link the library), then
 * come its own: integers, and for a pointer also None or an object with a buffer (a ctypes array). An
 * integer that its parameter does not hold is an error: cut to 32 bits, a window of 2^32 + 7 would be one of 7. */
static int integer(PyObject *arg, Py_ssize_t i, int narrow, unsigned long long *v) {
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(arg, &over);
  if (over == 0 && !(x == -1 && PyErr_Occurred()) && (!narrow || (x >= INT32_MIN && x <= INT32_MAX))) {
    *v = (unsigned long long)x;
    return 1;
  }
  if (over > 0 && !narrow) { /* addresses go up to 2^64 */
    *v = PyLong_AsUnsignedLongLong(arg);
    if (!PyErr_Occurred()) return 1;
    PyErr_Clear();
  }
  if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "argument %zd is out of range: %S", i, arg);
  return 0;
}
static int values(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, unsigned pointers, unsigned narrow, unsigned long long *v) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n), 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (PyLong_Check(args[i])) {
      if (!integer(args[i], i, narrow >> i & 1, v + i)) return 0;
    } else if (PyIndex_Check(args[i])) {
      PyObject *x = PyNumber_Index(args[i]);
      if (x == NULL) return 0;
      const int ok = integer(x, i, narrow >> i & 1, v + i);
      Py_DECREF(x);
      if (!ok) return 0;
    } else if (!(pointers >> i & 1)) {
      return PyErr_Format(PyExc_TypeError, "argument %zd must be an integer", i), 0;
    } else if (args[i] == Py_None) {
      v[i] = 0;
    } else {
      Py_buffer b;
      if (PyObject_GetBuffer(args[i], &b, PyBUF_SIMPLE) != 0) return 0;
      v[i] = (unsigned long long)(uintptr_t)b.buf;
      PyBuffer_Release(&b); /* the caller holds the object */
    }
  }
  if (v[0] == 0) return PyErr_Format(PyExc_ValueError, "a null address"), 0;
  return 1;
}
#define AT(i) ((void *)(uintptr_t)v[i])
#define ENTRY(name, count, pointers, narrow, ...)                                                 \
  static PyObject *py_##name(PyObject *self, PyObject *const *args, Py_ssize_t n) { \
    (void)self;                                                                   \
    unsigned long long v[count + 1];                                              \
    if (!values(args, n, count + 1, pointers, narrow, v)) return NULL;            \
    tp_status st;                                                                 \
    Py_BEGIN_ALLOW_THREADS                                                        \
    st = ((__typeof__(&tp_##name))AT(0))(__VA_ARGS__);                            \
    Py_END_ALLOW_THREADS                                                          \
    return PyLong_FromLong((long)st);                                             \
  }
/* after the count: which arguments are pointers, and which are 32 bits wide, a bit each */
ENTRY(rotary, 14, 0x7caa, 0x350, AT(1), (int64_t)v[2], AT(3), (int32_t)v[4], AT(5), (int32_t)v[6], AT(7), (int32_t)v[8], (int32_t)v[9], AT(10), AT(11),
      AT(12), AT(13), AT(14))
ENTRY(window_attn, 10, 0x59e, 0x60, AT(1), AT(2), AT(3), AT(4), (int32_t)v[5], (int32_t)v[6], AT(7), AT(8), (size_t)v[9], AT(10))
ENTRY(cache4_store, 11, 0xffa, 0, AT(1), (int64_t)v[2], AT(3), AT(4), AT(5), AT(6), AT(7), AT(8), AT(9), AT(10), AT(11))
ENTRY(cache4_load, 10, 0x7fa, 0, AT(1), (int64_t)v[2], AT(3), AT(4), AT(5), AT(6), AT(7), AT(8), AT(9), AT(10))
ENTRY(cache4_attn, 14, 0x59fa, 0x600, AT(1), (int64_t)v[2], AT(3), AT(4), AT(5), AT(6), AT(7), AT(8), (int32_t)v[9], (int32_t)v[10], AT(11), AT(12),
      (size_t)v[13], AT(14))

static PyObject *py_dtypes(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 4) return PyErr_Format(PyExc_TypeError, "dtypes(f32, bf16, e4m3, u8)");
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(args[i]);
    Py_XSETREF(known[i], args[i]);
  }
  Py_RETURN_NONE;
}

/* The torch that runs, as its "version revision". */
static PyObject *py_reads_torch(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  const char *version = n == 1 ? PyUnicode_AsUTF8(args[0]) : NULL;
  if (version == NULL) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_TypeError, "reads_torch(version)");
#ifdef TP_WITH_TORCH
  with_torch = strcmp(version, TP_TORCH_VERSION) == 0;
#endif
  return PyBool_FromLong(with_torch);
}

static PyMethodDef methods[] = {
    {"dtypes", (PyCFunction)(void (*)(void))py_dtypes, METH_FASTCALL, "dtypes(f32, bf16, e4m3, u8): the type objects of TP_F32, TP_BF16, TP_E4M3, TP_U8"},
    {"reads_torch", (PyCFunction)(void (*)(void))py_reads_torch, METH_FASTCALL, "reads_torch(version and revision of the torch that runs) -> whether tensors are read without their attributes"},
    {"matrix", (PyCFunction)(void (*)(void))py_matrix, METH_FASTCALL, "matrix(tensor, address[, device]) -> whether it was described there (device: the GPU on which it must lie, -1: any)"},
    {"row", (PyCFunction)(void (*)(void))py_row, METH_FASTCALL, "row(tensor, address): a 1-D tensor as a matrix of one row"},
    {"matrices", (PyCFunction)(void (*)(void))py_matrices, METH_FASTCALL, "matrices(sequence, count, address[, device]) -> how many of the first were described"},
    {"vector", (PyCFunction)(void (*)(void))py_vector, METH_FASTCALL, "vector(tensor, type, entries[, device]) -> address of a contiguous CUDA tensor of the type (tp_dtype, 4 for int32) with that many entries (-1: any), or None"},
    {"bytes", (PyCFunction)(void (*)(void))py_bytes, METH_FASTCALL, "bytes(tensor[, device]) -> (address, size) of a contiguous CUDA tensor, or None"},
#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, #name "(address of tp_" #name ", its arguments) -> status"}
    METHOD(rotary), METHOD(window_attn), METHOD(cache4_store), METHOD(cache4_load), METHOD(cache4_attn),
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
