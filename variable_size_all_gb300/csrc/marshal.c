/* marshal.c -- the checks that a call of the Python binding makes of each
 * tensor, in C: a call on W ranks looks at some dozens of small tensors, and
 * their attributes cost more host time in Python than the kernel takes.
 *
 * pointers(tensors, dtype, shapes, address) -> bool: true when every tensor is
 * a contiguous CUDA tensor of `dtype` and of its shape in the list `shapes`
 * (None: any); their data pointers are then at `address`, 8 bytes each.  False
 * otherwise (the binding then finds out which, and says so).
 *
 * rows(tensors) -> (rows of each, their common width), or None when they are
 * not all 2-D tensors of one width.
 *
 * sizes(tensors) -> the number of elements of each, or None.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

static PyObject *s_is_cuda, *s_is_contiguous, *s_dtype, *s_shape, *s_data_ptr, *s_numel;

/* 1: the attribute is `want`; 0: it is not, or there is none. */
static int is_attr(PyObject *t, PyObject *name, PyObject *want) {
  PyObject *v = PyObject_GetAttr(t, name);
  if (v == NULL) {
    PyErr_Clear();
    return 0;
  }
  Py_DECREF(v);
  return v == want;
}

static PyObject *pointers(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "pointers(tensors, dtype, shapes, address)");
    return NULL;
  }
  void **out = (void **)PyLong_AsVoidPtr(args[3]);
  if (out == NULL && PyErr_Occurred()) return NULL;
  PyObject *list = PySequence_Fast(args[0], "a sequence of tensors");
  if (list == NULL) return NULL;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(list);
  int good = args[2] == Py_None || (PyList_Check(args[2]) && PyList_GET_SIZE(args[2]) == count);
  for (Py_ssize_t i = 0; i < count && good; ++i) {
    PyObject *t = PySequence_Fast_GET_ITEM(list, i);
    good = is_attr(t, s_is_cuda, Py_True) && is_attr(t, s_dtype, args[1]);
    if (good && args[2] != Py_None) {
      PyObject *shape = PyObject_GetAttr(t, s_shape);
      const int same =
          shape == NULL ? 0 : PyObject_RichCompareBool(shape, PyList_GET_ITEM(args[2], i), Py_EQ);
      Py_XDECREF(shape);
      if (same < 0) PyErr_Clear();
      good = same == 1;
    }
    if (good) {
      PyObject *v = PyObject_CallMethodNoArgs(t, s_is_contiguous);
      good = v == Py_True;
      Py_XDECREF(v);
    }
    if (good) {
      PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
      good = p != NULL;
      if (p != NULL) out[i] = PyLong_AsVoidPtr(p);
      Py_XDECREF(p);
    }
    if (PyErr_Occurred()) {
      PyErr_Clear();
      good = 0;
    }
  }
  Py_DECREF(list);
  return PyBool_FromLong(good);
}

static PyObject *rows(PyObject *self, PyObject *tensors) {
  (void)self;
  PyObject *list = PySequence_Fast(tensors, "a sequence of tensors");
  if (list == NULL) return NULL;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(list);
  PyObject *out = PyList_New(count), *width = NULL;
  int good = out != NULL && count > 0;
  for (Py_ssize_t i = 0; i < count && good; ++i) {
    PyObject *shape = PyObject_GetAttr(PySequence_Fast_GET_ITEM(list, i), s_shape);
    good = shape != NULL && PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2;
    if (good) {
      PyObject *w = PyTuple_GET_ITEM(shape, 1), *n = PyTuple_GET_ITEM(shape, 0);
      if (width == NULL) {
        width = w;
        Py_INCREF(width);
      } else {
        good = PyObject_RichCompareBool(width, w, Py_EQ) == 1;
      }
      Py_INCREF(n);
      PyList_SET_ITEM(out, i, n);
    }
    Py_XDECREF(shape);
  }
  Py_DECREF(list);
  PyErr_Clear();
  PyObject *result = good ? PyTuple_Pack(2, out, width) : Py_NewRef(Py_None);
  Py_XDECREF(out);
  Py_XDECREF(width);
  return result;
}

static PyObject *sizes(PyObject *self, PyObject *tensors) {
  (void)self;
  PyObject *list = PySequence_Fast(tensors, "a sequence of tensors");
  if (list == NULL) return NULL;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(list);
  PyObject *out = PyList_New(count);
  int good = out != NULL;
  for (Py_ssize_t i = 0; i < count && good; ++i) {
    PyObject *n = PyObject_CallMethodNoArgs(PySequence_Fast_GET_ITEM(list, i), s_numel);
    good = n != NULL;
    if (good) PyList_SET_ITEM(out, i, n);
  }
  Py_DECREF(list);
  PyErr_Clear();
  if (good) return out;
  Py_XDECREF(out);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"pointers", (PyCFunction)(void (*)(void))pointers, METH_FASTCALL,
     "Checks a list of tensors and stores their data pointers."},
    {"rows", rows, METH_O, "Rows and common width of a list of 2-D tensors."},
    {"sizes", sizes, METH_O, "The number of elements of each tensor."},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_numel = PyUnicode_InternFromString("numel");
  if (s_is_cuda == NULL || s_is_contiguous == NULL || s_dtype == NULL || s_shape == NULL ||
      s_data_ptr == NULL || s_numel == NULL)
    return NULL;
  return PyModule_Create(&module);
}
