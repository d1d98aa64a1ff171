// marshal.cpp -- the checks that a call of the Python binding makes of each
// tensor, against torch's own tensors: a call on W ranks looks at some dozens of
// small tensors, and reading five attributes of each through Python took longer
// (12 us of a combine's 27 on 8 ranks) than the kernel does.
//
// pointers(address, count, (tensors, dtype, shapes), ...) -> bool: true when
// every list has `count` tensors, all of them contiguous CUDA tensors of the
// list's `dtype` and of their shapes in its list `shapes` of tuples (None: any);
// their data pointers are then at `address`, 8 bytes each, list after list.  A
// list that is None itself takes no place.  False otherwise (the binding then
// finds out which, and says so).
//
// rows(tensors) -> (rows of each, their common width), or None when they are
// not all 2-D tensors of one width.
//
// sizes(tensors) -> the number of elements of each, or None.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Dtype.h>

#include <cstdint>

namespace {

// A list's or tuple's items; false for anything else.
bool items_of(PyObject* o, PyObject*** items, Py_ssize_t* count) {
  if (PyList_Check(o)) {
    *items = reinterpret_cast<PyListObject*>(o)->ob_item;
    *count = PyList_GET_SIZE(o);
    return true;
  }
  if (PyTuple_Check(o)) {
    *items = reinterpret_cast<PyTupleObject*>(o)->ob_item;
    *count = PyTuple_GET_SIZE(o);
    return true;
  }
  return false;
}

const at::Tensor* tensor_of(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool has_shape(const at::Tensor& t, PyObject* shape) {
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
  for (Py_ssize_t d = 0; d < t.dim(); ++d)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d)) != t.size(d)) return false;
  return true;
}

bool list_pointers(PyObject* tensors, PyObject* dtype, PyObject* shapes, Py_ssize_t count,
                   void** out) {
  PyObject** items = nullptr;
  Py_ssize_t n = 0;
  if (!items_of(tensors, &items, &n) || n != count || !THPDtype_Check(dtype)) return false;
  if (shapes != Py_None && (!PyList_Check(shapes) || PyList_GET_SIZE(shapes) != count)) return false;
  const at::ScalarType type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor* t = tensor_of(items[i]);
    if (t == nullptr || !t->is_cuda() || t->scalar_type() != type || !t->is_contiguous()) return false;
    if (shapes != Py_None && !has_shape(*t, PyList_GET_ITEM(shapes, i))) return false;
    out[i] = t->data_ptr();
  }
  return true;
}

// Runs f, turning a C++ exception into false.
template <typename F>
bool quietly(F f) {
  try {
    return f();
  } catch (...) {
    return false;
  }
}

PyObject* pointers(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 2) {
    PyErr_SetString(PyExc_TypeError, "pointers(address, count, (tensors, dtype, shapes), ...)");
    return nullptr;
  }
  void** out = static_cast<void**>(PyLong_AsVoidPtr(args[0]));
  const Py_ssize_t count = PyLong_AsSsize_t(args[1]);
  if (PyErr_Occurred()) return nullptr;
  const bool good = quietly([&] {
    for (Py_ssize_t i = 2; i < n; ++i) {
      if (!PyTuple_Check(args[i]) || PyTuple_GET_SIZE(args[i]) != 3) return false;
      if (PyTuple_GET_ITEM(args[i], 0) == Py_None) continue;
      if (!list_pointers(PyTuple_GET_ITEM(args[i], 0), PyTuple_GET_ITEM(args[i], 1),
                         PyTuple_GET_ITEM(args[i], 2), count, out))
        return false;
      out += count;
    }
    return true;
  });
  PyErr_Clear();
  return PyBool_FromLong(good);
}

PyObject* rows(PyObject*, PyObject* tensors) {
  PyObject** items = nullptr;
  Py_ssize_t n = 0;
  if (!items_of(tensors, &items, &n) || n == 0) Py_RETURN_NONE;
  PyObject* out = PyList_New(n);
  if (out == nullptr) return nullptr;
  int64_t width = -1;
  const bool good = quietly([&] {
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t = tensor_of(items[i]);
      if (t == nullptr || t->dim() != 2 || (i > 0 && t->size(1) != width)) return false;
      width = t->size(1);
      PyObject* v = PyLong_FromLongLong(t->size(0));
      if (v == nullptr) return false;
      PyList_SET_ITEM(out, i, v);
    }
    return true;
  });
  PyErr_Clear();
  PyObject* result = good ? Py_BuildValue("(OL)", out, static_cast<long long>(width)) : Py_NewRef(Py_None);
  Py_DECREF(out);
  return result;
}

PyObject* sizes(PyObject*, PyObject* tensors) {
  PyObject** items = nullptr;
  Py_ssize_t n = 0;
  if (!items_of(tensors, &items, &n)) Py_RETURN_NONE;
  PyObject* out = PyList_New(n);
  if (out == nullptr) return nullptr;
  const bool good = quietly([&] {
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t = tensor_of(items[i]);
      PyObject* v = t == nullptr ? nullptr : PyLong_FromLongLong(t->numel());
      if (v == nullptr) return false;
      PyList_SET_ITEM(out, i, v);
    }
    return true;
  });
  PyErr_Clear();
  if (good) return out;
  Py_DECREF(out);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pointers)), METH_FASTCALL,
     "Checks lists of tensors and stores their data pointers."},
    {"rows", rows, METH_O, "Rows and common width of a list of 2-D tensors."},
    {"sizes", sizes, METH_O, "The number of elements of each tensor."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
