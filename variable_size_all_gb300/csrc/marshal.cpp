// marshal.cpp -- the checks that a call of the Python binding makes of each
// tensor, against torch's own tensors: a call on W ranks looks at some dozens of
// small tensors, and reading five attributes of each through Python took longer
// (12 us of a combine's 27 on 8 ranks) than the kernel does.
//
// route, route_backward, expert_matmul, expert_matmul_backward, combine_weighted,
// combine_weighted_backward, norm, norm_backward, quantise, dequantise and
// expert_matmul_mx(function, handle, stream, W, the method's arguments)
// -> the library's return value: the whole call, where every list has W good
// tensors and every number is in its range.  None where one is not, or is
// missing: nothing has been called, and the binding goes through its arguments
// one by one.  (8 ranks, host time: routing 3.6 us against 9.4, a weighted
// combine 3.7 against 14.4, launches included.)
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

#include <climits>
#include <cstdint>

#include "a2av_mx.h"

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

// ----------------------------------------------------- whole calls --
constexpr int kRanks = A2AV_MAX_RANKS;

// What every whole call begins with.
struct Call {
  void *function, *handle, *stream;
  int W;
};

bool int_of(PyObject* o, int* v) {
  if (!PyLong_Check(o)) return false;
  const long long x = PyLong_AsLongLong(o);
  *v = (int)x;
  return x >= INT_MIN && x <= INT_MAX && !PyErr_Occurred();
}

bool call_of(PyObject* const* args, Call* c) {
  c->function = PyLong_Check(args[0]) ? PyLong_AsVoidPtr(args[0]) : nullptr;
  c->handle = PyLong_Check(args[1]) ? PyLong_AsVoidPtr(args[1]) : nullptr;
  if (c->function == nullptr || c->handle == nullptr || !PyLong_Check(args[2])) return false;
  c->stream = PyLong_AsVoidPtr(args[2]);
  return int_of(args[3], &c->W) && c->W >= 1 && c->W <= kRanks && !PyErr_Occurred();
}

bool is_good(const at::Tensor* t, at::ScalarType type) {
  return t != nullptr && t->is_cuda() && t->scalar_type() == type && t->is_contiguous();
}

// The data pointers of W good tensors that `fits`(tensor, index) accepts.
template <typename F>
bool take(PyObject* list, int W, at::ScalarType type, void** out, F fits) {
  PyObject** items = nullptr;
  Py_ssize_t n = 0;
  if (!items_of(list, &items, &n) || n != W) return false;
  for (int i = 0; i < W; ++i) {
    const at::Tensor* t = tensor_of(items[i]);
    if (!is_good(t, type) || !fits(*t, i)) return false;
    out[i] = t->data_ptr();
  }
  return true;
}

// The same for tensors of [rows[i], width].
bool take_rows(PyObject* list, int W, at::ScalarType type, void** out, const int64_t* rows,
               int64_t width) {
  return take(list, W, type, out, [&](const at::Tensor& t, int i) {
    return t.dim() == 2 && t.size(0) == rows[i] && t.size(1) == width;
  });
}

// And where the rows are what is asked for: `width` is the first one's, that all have.
bool take_any_rows(PyObject* list, int W, at::ScalarType type, void** out, int64_t* rows,
                   int64_t* width) {
  return take(list, W, type, out, [&](const at::Tensor& t, int i) {
    if (t.dim() != 2 || (i > 0 && t.size(1) != *width)) return false;
    *width = t.size(1);
    rows[i] = t.size(0);
    return true;
  });
}

// A list's first tensor's type, and its code.
bool type_of(PyObject* list, bool f32, at::ScalarType* type, int* code) {
  PyObject** items = nullptr;
  Py_ssize_t n = 0;
  const at::Tensor* t = items_of(list, &items, &n) && n > 0 ? tensor_of(items[0]) : nullptr;
  if (t == nullptr) return false;
  *type = t->scalar_type();
  *code = *type == at::kBFloat16 ? A2AV_BF16 : *type == at::kHalf ? A2AV_F16 : A2AV_F32;
  return *code != A2AV_F32 || (f32 && *type == at::kFloat);
}

// The second dimension of a list's first tensor; 0 where it has none.
int64_t width_of(PyObject* list) {
  PyObject** items = nullptr;
  Py_ssize_t n = 0;
  const at::Tensor* t = items_of(list, &items, &n) && n > 0 ? tensor_of(items[0]) : nullptr;
  return t != nullptr && t->dim() == 2 ? t->size(1) : 0;
}

bool has_sizes(const at::Tensor& t, int64_t a, int64_t b) {
  return t.dim() == 2 && t.size(0) == a && t.size(1) == b;
}

// A tensor of int64 [a, b].
bool matrix_of(PyObject* o, int64_t a, int64_t b, const int64_t** out) {
  const at::Tensor* t = tensor_of(o);
  if (!is_good(t, at::kLong) || !has_sizes(*t, a, b)) return false;
  *out = static_cast<const int64_t*>(t->data_ptr());
  return true;
}

// Checks with `prepare`, then calls with `enqueue`, without the interpreter's lock.
template <typename P, typename E>
PyObject* whole(Py_ssize_t n, Py_ssize_t want, P prepare, E enqueue) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  const bool good = quietly(prepare) && !PyErr_Occurred();
  PyErr_Clear();
  if (!good) Py_RETURN_NONE;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = enqueue();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// The lists a router's call has in either direction.
struct Routing {
  Call c;
  a2av_route_t shape;
  at::ScalarType type;
  int64_t tokens[kRanks];
  void *logits[kRanks], *keys[kRanks], *weights[kRanks];

  bool take_all(PyObject* x, PyObject* k, PyObject* w, PyObject* topk, PyObject* score,
                PyObject* renormalise, PyObject* scale) {
    int64_t E = 0;
    if (!type_of(x, true, &type, &shape.dtype) ||
        !take_any_rows(x, c.W, type, logits, tokens, &E) || !int_of(topk, &shape.topk) ||
        shape.topk < 1 || shape.topk > E || E > INT_MAX || !int_of(score, &shape.score))
      return false;
    shape.experts = (int)E;
    shape.renormalise = PyObject_IsTrue(renormalise) == 1;
    shape.scale = (float)PyFloat_AsDouble(scale);
    return take_rows(k, c.W, at::kInt, keys, tokens, shape.topk) &&
           take_rows(w, c.W, at::kFloat, weights, tokens, shape.topk);
  }
};

// (..., logits, keys, weights, topk, counts, bias, score, groups, top_groups, group_top,
// renormalise, scale)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Routing r;
  const int64_t* counts = nullptr;
  const float* bias = nullptr;
  return whole(
      n, 16,
      [&] {
        if (!call_of(args, &r.c) ||
            !r.take_all(args[4], args[5], args[6], args[7], args[10], args[14], args[15]) ||
            !int_of(args[11], &r.shape.groups) || !int_of(args[12], &r.shape.top_groups) ||
            !int_of(args[13], &r.shape.group_top))
          return false;
        if (args[8] != Py_None && !matrix_of(args[8], r.c.W, r.shape.experts, &counts)) return false;
        if (args[9] != Py_None) {
          const at::Tensor* t = tensor_of(args[9]);
          if (!is_good(t, at::kFloat) || t->dim() != 1 || t->size(0) != r.shape.experts) return false;
          bias = static_cast<const float*>(t->data_ptr());
        }
        return true;
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_route)>(r.c.function)(
            static_cast<a2av_handle*>(r.c.handle), &r.shape, r.logits, r.tokens, bias,
            reinterpret_cast<int32_t* const*>(r.keys), reinterpret_cast<float* const*>(r.weights),
            const_cast<int64_t*>(counts), r.c.stream);
      });
}

// (..., logits, keys, d_weights, d_logits, topk, score, renormalise, scale)
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Routing r;
  void* d_logits[kRanks];
  return whole(
      n, 12,
      [&] {
        r.shape.groups = r.shape.top_groups = r.shape.group_top = 1;
        return call_of(args, &r.c) &&
               r.take_all(args[4], args[5], args[6], args[8], args[9], args[10], args[11]) &&
               take_rows(args[7], r.c.W, r.type, d_logits, r.tokens, r.shape.experts);
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_route_backward)>(r.c.function)(
            static_cast<a2av_handle*>(r.c.handle), &r.shape, r.logits, r.tokens,
            reinterpret_cast<const int32_t* const*>(r.keys),
            reinterpret_cast<const float* const*>(r.weights), d_logits, r.c.stream);
      });
}

// The lists an expert's product has in either direction; `out` are its results
// or their gradients.
struct Product {
  Call c;
  a2av_expert_t shape;
  at::ScalarType type;
  int64_t held[kRanks], K, Z, D, N;
  const int64_t* counts;
  void *rows[kRanks], *weights[kRanks], *out[kRanks];

  bool take_all(PyObject* x, PyObject* s, PyObject* w, PyObject* y, PyObject* activation,
                PyObject* gated) {
    int64_t n[kRanks];
    if (!type_of(w, false, &type, &shape.dtype) || !take_any_rows(x, c.W, type, rows, held, &D) ||
        !take_any_rows(y, c.W, type, out, n, &N) || !int_of(activation, &shape.activation))
      return false;
    for (int p = 0; p < c.W; ++p)
      if (n[p] != held[p]) return false;
    shape.gated = PyObject_IsTrue(gated) == 1;
    Z = shape.gated ? 2 * N : N;
    if (!take(w, c.W, type, weights, [&](const at::Tensor& t, int i) {
          if (t.dim() != 3 || (i > 0 && t.size(0) != K)) return false;
          K = t.size(0);
          return t.size(1) == Z && t.size(2) == D;
        }))
      return false;
    shape.experts_per_peer = (int)K;
    shape.in_features = D;
    shape.out_features = N;
    return K <= INT_MAX && matrix_of(s, c.W, c.W * K, &counts);
  }

  // Optional lists of [rows, width], [K, Z] and [K, Z, D].
  bool take_by_row(PyObject* list, int64_t width, void** to) const {
    return list == Py_None || take_rows(list, c.W, type, to, held, width);
  }
  bool take_bias(PyObject* list, void** to) const {
    return list == Py_None || take(list, c.W, type, to, [&](const at::Tensor& t, int) {
             return has_sizes(t, K, Z);
           });
  }
  bool take_weights(PyObject* list, void** to) const {
    return list == Py_None || take(list, c.W, type, to, [&](const at::Tensor& t, int) {
             return t.dim() == 3 && t.size(0) == K && t.size(1) == Z && t.size(2) == D;
           });
  }
};

// (..., rows, counts, weights, outputs, activation, gated, bias, residual, pre)
PyObject* expert_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Product m;
  void *bias[kRanks], *residual[kRanks], *pre[kRanks];
  return whole(
      n, 13,
      [&] {
        return call_of(args, &m.c) &&
               m.take_all(args[4], args[5], args[6], args[7], args[8], args[9]) &&
               m.take_bias(args[10], bias) && m.take_by_row(args[11], m.N, residual) &&
               m.take_by_row(args[12], m.Z, pre);
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_expert_matmul)>(m.c.function)(
            static_cast<a2av_handle*>(m.c.handle), &m.shape, m.rows, m.held, m.counts, m.weights,
            args[10] == Py_None ? nullptr : bias, args[11] == Py_None ? nullptr : residual, m.out,
            args[12] == Py_None ? nullptr : pre, m.c.stream);
      });
}

// (..., rows, counts, weights, d_outputs, d_rows, d_weights, d_bias, pre, activation, gated,
// workspace, a2av_expert_matmul_workspace_bytes); None as well where the workspace is too small.
PyObject* expert_matmul_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Product m;
  void *d_rows[kRanks], *d_weights[kRanks], *d_bias[kRanks], *pre[kRanks], *workspace = nullptr;
  int64_t bytes = 0;
  bool activated = false;
  return whole(
      n, 16,
      [&] {
        if (!call_of(args, &m.c) ||
            !m.take_all(args[4], args[5], args[6], args[7], args[12], args[13]) ||
            !m.take_by_row(args[8], m.D, d_rows) || !m.take_weights(args[9], d_weights) ||
            !m.take_bias(args[10], d_bias))
          return false;
        activated = m.shape.activation != A2AV_ACT_NONE || m.shape.gated;
        if (activated && (args[11] == Py_None || !m.take_by_row(args[11], m.Z, pre))) return false;
        const at::Tensor* t = tensor_of(args[14]);
        void* size_of = PyLong_Check(args[15]) ? PyLong_AsVoidPtr(args[15]) : nullptr;
        if (!is_good(t, at::kByte) || size_of == nullptr) return false;
        int64_t total = 0;
        for (int p = 0; p < m.c.W; ++p) total += m.held[p];
        const int64_t need = reinterpret_cast<decltype(&a2av_expert_matmul_workspace_bytes)>(size_of)(
            m.c.W, &m.shape, total);
        workspace = t->data_ptr();
        bytes = t->numel();
        return need > 0 && bytes >= need;
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_expert_matmul_backward)>(m.c.function)(
            static_cast<a2av_handle*>(m.c.handle), &m.shape, m.rows, m.held, m.counts, m.weights,
            activated ? pre : nullptr, m.out, args[8] == Py_None ? nullptr : d_rows,
            args[9] == Py_None ? nullptr : d_weights, args[10] == Py_None ? nullptr : d_bias, workspace,
            bytes, m.c.stream);
      });
}

// The lists a weighted combine has in either direction.
struct Weighted {
  Call c;
  at::ScalarType type;
  int K, k, dtype;
  int64_t H, tokens[kRanks], held[kRanks];
  const int64_t* splits;
  void *token_rows[kRanks], *keys[kRanks], *pos[kRanks], *weights[kRanks], *peers[kRanks],
      *d_peers[kRanks];
  bool has_weights, has_peers, has_d_peers;

  bool take_all(PyObject* p, PyObject* s, PyObject* ks, PyObject* ps, PyObject* per, PyObject* ws,
                PyObject* rows, PyObject* dp, PyObject* dw) {
    H = 0;
    if (!type_of(rows, true, &type, &dtype) ||
        !take_any_rows(rows, c.W, type, token_rows, tokens, &H) ||
        !matrix_of(s, c.W, c.W, &splits) || !int_of(per, &K))
      return false;
    int64_t items = -1;  // of the first rank that has tokens, for each of them
    const auto fits = [&](const at::Tensor& t, int i) {
      if (items < 0 && tokens[i] > 0) items = t.numel() / tokens[i];
      return t.numel() == tokens[i] * (items < 0 ? 0 : items);
    };
    if (!take(ks, c.W, at::kInt, keys, fits)) return false;
    // (no token on any rank: the width that the keys or the weights have)
    for (PyObject* list : {ks, ws, dw})
      if (items < 0 && width_of(list) > 0) items = width_of(list);
    if (items == 0 || items > INT_MAX) return false;
    k = items < 0 ? 1 : (int)items;
    if (!take(ps, c.W, at::kLong, pos, fits)) return false;
    has_weights = ws != Py_None;
    if (has_weights && !take_rows(ws, c.W, at::kFloat, weights, tokens, k)) return false;
    has_peers = p != Py_None;
    has_d_peers = dp != Py_None;
    int64_t width = H;
    if (has_peers && (!take_any_rows(p, c.W, type, peers, held, &width) || width != H)) return false;
    if (!has_d_peers) return has_peers;
    if (has_peers) return take_rows(dp, c.W, type, d_peers, held, H);
    return take_any_rows(dp, c.W, type, d_peers, held, &width) && width == H;
  }
};

// (..., peers, in_splits, keys, sorted_pos, keys_per_peer, weights, outputs, residual)
PyObject* combine_weighted(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Weighted m;
  void* residual[kRanks];
  return whole(
      n, 12,
      [&] {
        return call_of(args, &m.c) && args[4] != Py_None &&
               m.take_all(args[4], args[5], args[6], args[7], args[8], args[9], args[10], Py_None,
                          Py_None) &&
               (args[11] == Py_None ||
                take_rows(args[11], m.c.W, m.type, residual, m.tokens, m.H));
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_combine_weighted)>(m.c.function)(
            static_cast<a2av_handle*>(m.c.handle), m.K, m.k, m.H, m.dtype, m.peers, m.held, m.splits,
            reinterpret_cast<const int32_t* const*>(m.keys),
            reinterpret_cast<const int64_t* const*>(m.pos),
            m.has_weights ? reinterpret_cast<const float* const*>(m.weights) : nullptr, m.tokens,
            args[11] == Py_None ? nullptr : residual, m.token_rows, m.c.stream);
      });
}

// (..., peers, in_splits, keys, sorted_pos, keys_per_peer, weights, d_outputs, d_peers, d_weights)
PyObject* combine_weighted_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Weighted m;
  void* d_weights[kRanks];
  return whole(
      n, 13,
      [&] {
        return call_of(args, &m.c) &&
               m.take_all(args[4], args[5], args[6], args[7], args[8], args[9], args[10], args[11],
                          args[12]) &&
               (args[12] == Py_None ||
                take_rows(args[12], m.c.W, at::kFloat, d_weights, m.tokens, m.k));
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_combine_weighted_backward)>(m.c.function)(
            static_cast<a2av_handle*>(m.c.handle), m.K, m.k, m.H, m.dtype,
            m.has_peers ? m.peers : nullptr, m.held, m.splits,
            reinterpret_cast<const int32_t* const*>(m.keys),
            reinterpret_cast<const int64_t* const*>(m.pos),
            m.has_weights ? reinterpret_cast<const float* const*>(m.weights) : nullptr, m.tokens,
            m.token_rows, m.has_d_peers ? m.d_peers : nullptr,
            args[12] == Py_None ? nullptr : reinterpret_cast<float* const*>(d_weights), m.c.stream);
      });
}

// A packed row's bytes by the library's own function, or -1.
int64_t packed_bytes(PyObject* entry, int64_t features, int format) {
  void* f = PyLong_Check(entry) ? PyLong_AsVoidPtr(entry) : nullptr;
  return f == nullptr ? -1 : reinterpret_cast<decltype(&a2av_mx_row_bytes)>(f)(features, format);
}

// A float [n].
bool vector_of(PyObject* o, int64_t n, float** out) {
  const at::Tensor* t = tensor_of(o);
  if (!is_good(t, at::kFloat) || t->dim() != 1 || t->size(0) != n) return false;
  *out = static_cast<float*>(t->data_ptr());
  return true;
}

// An optional list of [rows[i], width].
bool take_optional(PyObject* list, int W, at::ScalarType type, void** out, const int64_t* rows,
                   int64_t width) {
  return list == Py_None || take_rows(list, W, type, out, rows, width);
}

// The lists that a norm's calls begin with.
struct Normed {
  Call c;
  at::ScalarType type;
  int dtype;
  int64_t rows[kRanks], H;
  void* x[kRanks];
  float *weight, eps;

  bool take_all(PyObject* list, PyObject* w, PyObject* e) {
    H = 0;
    eps = (float)PyFloat_AsDouble(e);
    return type_of(list, true, &type, &dtype) && take_any_rows(list, c.W, type, x, rows, &H) &&
           vector_of(w, H, &weight);
  }
};

// (..., x, weight, outputs, residual, sums, eps, format, plain, a2av_mx_row_bytes)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Normed m;
  int format = A2AV_PLAIN;
  void *out[kRanks], *residual[kRanks], *sums[kRanks], *plain[kRanks];
  return whole(
      n, 13,
      [&] {
        if (!call_of(args, &m.c) || !m.take_all(args[4], args[5], args[9]) || !int_of(args[10], &format) ||
            !take_optional(args[7], m.c.W, m.type, residual, m.rows, m.H) ||
            !take_optional(args[8], m.c.W, m.type, sums, m.rows, m.H))
          return false;
        if (format == A2AV_PLAIN)
          return args[11] == Py_None && take_rows(args[6], m.c.W, m.type, out, m.rows, m.H);
        return take_rows(args[6], m.c.W, at::kByte, out, m.rows, packed_bytes(args[12], m.H, format)) &&
               take_optional(args[11], m.c.W, m.type, plain, m.rows, m.H);
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_norm)>(m.c.function)(
            static_cast<a2av_handle*>(m.c.handle), m.H, m.dtype, format, m.eps, m.x, m.rows, m.weight,
            args[7] == Py_None ? nullptr : residual, args[8] == Py_None ? nullptr : sums, out,
            args[11] == Py_None ? nullptr : plain, m.c.stream);
      });
}

// (..., sums, weight, d_outputs, d_x, d_weight, d_sums, eps, workspace,
// a2av_norm_workspace_bytes); None as well where the workspace is too small.
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Normed m;
  void *dy[kRanks], *dx[kRanks], *ds[kRanks], *workspace = nullptr;
  float* d_weight = nullptr;
  int64_t bytes = 0;
  return whole(
      n, 13,
      [&] {
        if (!call_of(args, &m.c) || !m.take_all(args[4], args[5], args[10]) ||
            !take_rows(args[6], m.c.W, m.type, dy, m.rows, m.H) ||
            !take_rows(args[7], m.c.W, m.type, dx, m.rows, m.H) ||
            !take_optional(args[9], m.c.W, m.type, ds, m.rows, m.H))
          return false;
        if (args[8] == Py_None) return true;
        const at::Tensor* t = tensor_of(args[11]);
        void* size_of = PyLong_Check(args[12]) ? PyLong_AsVoidPtr(args[12]) : nullptr;
        if (!vector_of(args[8], m.H, &d_weight) || !is_good(t, at::kByte) || size_of == nullptr)
          return false;
        int64_t total = 0;
        for (int p = 0; p < m.c.W; ++p) total += m.rows[p];
        workspace = t->data_ptr();
        bytes = t->numel();
        const int64_t need =
            reinterpret_cast<decltype(&a2av_norm_workspace_bytes)>(size_of)(m.H, total);
        return need > 0 && bytes >= need;
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_norm_backward)>(m.c.function)(
            static_cast<a2av_handle*>(m.c.handle), m.H, m.dtype, m.eps, m.x, m.rows, m.weight, dy,
            args[9] == Py_None ? nullptr : ds, dx, d_weight, workspace, bytes, m.c.stream);
      });
}

// (..., rows to read, rows to write, format, in_splits, a2av_mx_row_bytes); `back`: from packed ones.
PyObject* packing(PyObject* const* args, Py_ssize_t n, bool back) {
  Call c;
  at::ScalarType type;
  int dtype, format;
  int64_t rows[kRanks], D = 0;
  void *plain[kRanks], *packed[kRanks];
  const int64_t* splits = nullptr;
  return whole(
      n, 9,
      [&] {
        return call_of(args, &c) && type_of(args[back ? 5 : 4], true, &type, &dtype) &&
               take_any_rows(args[back ? 5 : 4], c.W, type, plain, rows, &D) &&
               int_of(args[6], &format) && (args[7] == Py_None || matrix_of(args[7], c.W, c.W, &splits)) &&
               take_rows(args[back ? 4 : 5], c.W, at::kByte, packed, rows,
                         packed_bytes(args[8], D, format));
      },
      [&] {
        // (the two have one signature)
        return reinterpret_cast<decltype(&a2av_quantise)>(c.function)(
            static_cast<a2av_handle*>(c.handle), D, dtype, format, back ? packed : plain, rows, splits,
            back ? plain : packed, c.stream);
      });
}
PyObject* quantise(PyObject*, PyObject* const* args, Py_ssize_t n) { return packing(args, n, false); }
PyObject* dequantise(PyObject*, PyObject* const* args, Py_ssize_t n) { return packing(args, n, true); }

// (..., rows, counts, weights, outputs, in_features, format, activation, gated, bias,
// residual, a2av_mx_row_bytes)
PyObject* expert_matmul_mx(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Call c;
  a2av_expert_t shape;
  at::ScalarType type;
  int format, D;
  int64_t held[kRanks], K = 0, Z, N = 0, bytes;
  const int64_t* counts;
  void *rows[kRanks], *weights[kRanks], *out[kRanks], *bias[kRanks], *residual[kRanks];
  return whole(
      n, 15,
      [&] {
        if (!call_of(args, &c) || !type_of(args[7], false, &type, &shape.dtype) ||
            !take_any_rows(args[7], c.W, type, out, held, &N) || !int_of(args[8], &D) ||
            !int_of(args[9], &format) || !int_of(args[10], &shape.activation))
          return false;
        bytes = packed_bytes(args[14], D, format);
        shape.gated = PyObject_IsTrue(args[11]) == 1;
        Z = shape.gated ? 2 * N : N;
        if (!take_rows(args[4], c.W, at::kByte, rows, held, bytes) ||
            !take(args[6], c.W, at::kByte, weights, [&](const at::Tensor& t, int i) {
              if (t.dim() != 3 || (i > 0 && t.size(0) != K)) return false;
              K = t.size(0);
              return t.size(1) == Z && t.size(2) == bytes;
            }) ||
            K > INT_MAX || !matrix_of(args[5], c.W, c.W * K, &counts) ||
            !take_optional(args[13], c.W, type, residual, held, N))
          return false;
        shape.experts_per_peer = (int)K;
        shape.in_features = D;
        shape.out_features = N;
        return args[12] == Py_None || take(args[12], c.W, type, bias, [&](const at::Tensor& t, int) {
                 return has_sizes(t, K, Z);
               });
      },
      [&] {
        return reinterpret_cast<decltype(&a2av_expert_matmul_mx)>(c.function)(
            static_cast<a2av_handle*>(c.handle), &shape, format, rows, held, counts, weights,
            args[12] == Py_None ? nullptr : bias, args[13] == Py_None ? nullptr : residual, out,
            c.stream);
      });
}

#define A2AV_WHOLE(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, "A whole call."}

PyMethodDef methods[] = {
    {"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pointers)), METH_FASTCALL,
     "Checks lists of tensors and stores their data pointers."},
    {"rows", rows, METH_O, "Rows and common width of a list of 2-D tensors."},
    {"sizes", sizes, METH_O, "The number of elements of each tensor."},
    A2AV_WHOLE(route),
    A2AV_WHOLE(route_backward),
    A2AV_WHOLE(expert_matmul),
    A2AV_WHOLE(expert_matmul_backward),
    A2AV_WHOLE(combine_weighted),
    A2AV_WHOLE(combine_weighted_backward),
    A2AV_WHOLE(norm),
    A2AV_WHOLE(norm_backward),
    A2AV_WHOLE(quantise),
    A2AV_WHOLE(dequantise),
    A2AV_WHOLE(expert_matmul_mx),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  // (the torch whose headers these are: the binding compares)
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", A2AV_TORCH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
