/* marshal.c -- the checks that a call of the Python binding makes of each
 * tensor, in C: a call on W ranks looks at some dozens of small tensors, and
 * their attributes cost more host time in Python than the kernel takes.
 *
 * pointers(tensors, dtype, shapes, address) -> bool: true when every tensor is
 * a contiguous CUDA tensor of `dtype` and of its shape in the list `shapes`
 * (None: any); their data pointers are then at `address`, 8 bytes each.  False
 * otherwise (the binding then finds out which, and says so).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

static PyObject *s_is_cuda, *s_is_contiguous, *s_dtype, *s_shape, *s_data_ptr;

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

static PyMethodDef methods[] = {
    {"pointers", (PyCFunction)(void (*)(void))pointers, METH_FASTCALL,
     "Checks a list of tensors and stores their data pointers."},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (s_is_cuda == NULL || s_is_contiguous == NULL || s_dtype == NULL || s_shape == NULL ||
      s_data_ptr == NULL)
    return NULL;
  return PyModule_Create(&module);
}
