// Python binding of the training-step operators: the calls of training.py on
// torch tensors, as a CPython extension module. At the sizes of a decoding
// step the host's part is most of a call: reading the tensors here takes 1 us
// where attribute reads and ctypes conversions in Python took 3.5 to 7.
//
// A tensor has to be on the current GPU, of a type that the C function takes, with its
// last dimension contiguous, and may require gradients only where none are
// recorded: ValueError otherwise, naming the argument. The library checks the
// rest: NsError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <exception>
#include <initializer_list>
#include <sstream>
#include <string>

#include "nsgb300.h"

namespace {

PyObject* g_check = nullptr;  // _lib.check

struct Refused {};  // the Python error is set

constexpr int kMaxArgs = 16;

// Names of a call's arguments, the first `required` of them without a default.
struct Signature {
  const char* function;
  int required, count;
  const char* names[kMaxArgs];
  PyObject* keys[kMaxArgs];
};

// The arguments of one call by position, nullptr where the default stands.
struct Args {
  const Signature& sig;
  PyObject* at[kMaxArgs] = {};

  Args(const Signature& s, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) : sig(s) {
    if (n > s.count) {
      PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", s.function, s.count, n);
      throw Refused();
    }
    for (Py_ssize_t i = 0; i < n; ++i) at[i] = args[i];
    const Py_ssize_t k = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t i = 0; i < k; ++i) {
      PyObject* key = PyTuple_GET_ITEM(kwnames, i);
      int j = 0;
      while (j < s.count && s.keys[j] != key) ++j;
      if (j == s.count)
        for (j = 0; j < s.count && PyUnicode_Compare(s.keys[j], key) != 0;) ++j;
      if (j == s.count || at[j]) {
        PyErr_Format(PyExc_TypeError, j == s.count ? "%s() got an unexpected keyword argument %R"
                                                   : "%s() got multiple values for argument %R",
                     s.function, key);
        throw Refused();
      }
      at[j] = args[n + i];
    }
    for (int i = 0; i < s.required; ++i)
      if (!at[i]) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", s.function, s.names[i]);
        throw Refused();
      }
  }

  bool given(int i) const { return at[i] && at[i] != Py_None; }

  [[noreturn]] void bad(int i, const std::string& want) const {
    std::ostringstream m;
    m << sig.names[i] << ": " << want << ", got ";
    if (THPVariable_Check(at[i])) {
      const at::Tensor& t = THPVariable_Unpack(at[i]);
      m << t.dtype().name() << " " << t.sizes() << " with strides " << t.strides() << " on " << t.device();
    } else {
      m << Py_TYPE(at[i])->tp_name;
    }
    PyErr_SetString(PyExc_ValueError, m.str().c_str());
    throw Refused();
  }

  const at::Tensor& tensor(int i) const {
    if (!THPVariable_Check(at[i])) bad(i, "a tensor");
    return THPVariable_Unpack(at[i]);
  }
  // On the GPU that the call runs on.
  bool here(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == c10::cuda::current_device(); }
  // A GPU tensor of `dims` dimensions.
  const at::Tensor& gpu(int i, int dims) const {
    const at::Tensor& t = tensor(i);
    if (!here(t) || t.dim() != dims) bad(i, "a GPU tensor of " + std::to_string(dims) + " dimensions");
    return t;
  }
  // The address of a tensor's values. The calls record nothing: a graph would end here without a word.
  void* address(int i, const at::Tensor& t) const {
    if (t.requires_grad() && c10::GradMode::is_enabled())
      bad(i, "a tensor without gradients to record (detached, under no_grad or in an autograd.Function)");
    return t.data_ptr();
  }
  // The address of `numel` contiguous values; null for None.
  void* whole(int i, at::ScalarType type, int64_t numel) const {
    if (!given(i)) return nullptr;
    const at::Tensor& t = tensor(i);
    if (!here(t) || t.scalar_type() != type || t.numel() != numel || !t.is_contiguous())
      bad(i, std::to_string(numel) + " contiguous GPU values of " + c10::toString(type));
    return address(i, t);
  }
  const void* indices(int i, int64_t numel, int* bytes) const {
    const at::Tensor& t = tensor(i);
    const at::ScalarType type = t.scalar_type();
    if (!here(t) || (type != at::kInt && type != at::kLong) || t.numel() != numel || !t.is_contiguous())
      bad(i, std::to_string(numel) + " contiguous GPU indices (int32 or int64)");
    *bytes = type == at::kLong ? 8 : 4;
    return t.data_ptr();
  }
  void* scratch(int i, uint64_t* bytes) const {
    *bytes = 0;
    if (!given(i)) return nullptr;
    const at::Tensor& t = tensor(i);
    if (!here(t) || !t.is_contiguous()) bad(i, "a contiguous GPU tensor");
    *bytes = t.nbytes();
    return t.data_ptr();
  }
  int dtype(int i) const {
    switch (tensor(i).scalar_type()) {
      case at::kBFloat16: return NS_DT_BF16;
      case at::kHalf: return NS_DT_FP16;
      case at::kFloat: return NS_DT_FP32;
      default: bad(i, "bfloat16, float16 or float32");
    }
  }
  // Address and row stride of a matrix [rows, cols] (negative: any) with
  // contiguous rows.
  void* matrix(int i, at::ScalarType type, int64_t rows, int64_t cols, int64_t* stride) const {
    const at::Tensor& t = gpu(i, 2);
    const int64_t n = t.size(0), d = t.size(1);
    if (t.scalar_type() != type || (rows >= 0 && n != rows) || (cols >= 0 && d != cols)) {
      std::string want = std::string("a matrix of ") + c10::toString(type);
      if (rows >= 0) want += ", " + std::to_string(rows) + " rows";
      if (cols >= 0) want += ", " + std::to_string(cols) + " columns";
      bad(i, want);
    }
    if (t.stride(1) != 1 && d > 1) bad(i, "contiguous rows");
    *stride = n > 1 ? t.stride(0) : std::max(t.stride(0), d);
    return address(i, t);
  }
  int64_t number(int i, int64_t otherwise) const {
    if (!at[i]) return otherwise;
    const long long v = PyLong_AsLongLong(at[i]);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
  }
  // Clamped to int, so that a value out of range reaches the library's checks as one.
  int small(int i, int otherwise) const {
    return static_cast<int>(std::clamp<int64_t>(number(i, otherwise), INT_MIN, INT_MAX));
  }
  float real(int i, float otherwise) const {
    if (!at[i]) return otherwise;
    const double v = PyFloat_AsDouble(at[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return static_cast<float>(v);
  }
  bool flag(int i) const {
    const int v = at[i] ? PyObject_IsTrue(at[i]) : 0;
    if (v < 0) throw Refused();
    return v != 0;
  }
  // The last argument: a torch stream, a handle, or None for torch's current one.
  void* stream() const {
    PyObject* s = at[sig.count - 1];
    if (!s || s == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* handle = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
    if (!handle) throw Refused();
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }
  // What the call returns; the arguments that it wrote count one write more for autograd.
  PyObject* result(int rc, std::initializer_list<int> written) const {
    if (rc == NS_OK) {
      for (int i : written)
        if (given(i)) {
          const at::Tensor& t = THPVariable_Unpack(at[i]);
          if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
        }
      Py_RETURN_NONE;
    }
    return PyObject_CallFunction(g_check, "is", rc, sig.function);
  }
};

// [tokens, k] of row_of_slot at argument i.
int* slots(const Args& a, int i, int64_t* tokens, int64_t* k) {
  const at::Tensor& t = a.gpu(i, 2);
  *tokens = t.size(0);
  *k = t.size(1);
  return static_cast<int*>(a.whole(i, at::kInt, *tokens * *k));
}

// A count for a C int: what does not fit is out of every range.
int as_int(int64_t v) { return static_cast<int>(std::min<int64_t>(v, INT_MAX)); }

PyObject* moe_sort(const Args& a) {
  const at::Tensor& t = a.gpu(0, 2);
  const int64_t tokens = t.size(0), k = t.size(1), rows = a.tensor(3).numel();
  int id_bytes;
  uint64_t ws_bytes;
  const void* ids = a.indices(0, tokens * k, &id_bytes);
  const int experts = a.small(1, 0);
  void* ws = a.scratch(6, &ws_bytes);
  return a.result(ns_moe_sort(ids, id_bytes, tokens, as_int(k), experts, a.small(7, 1), a.number(8, 0), rows,
                              static_cast<int*>(a.whole(2, at::kInt, tokens * k)),
                              static_cast<int*>(a.whole(3, at::kInt, rows)),
                              static_cast<int*>(a.whole(4, at::kInt, experts)),
                              static_cast<int*>(a.whole(5, at::kInt, static_cast<int64_t>(experts) + 1)), ws, ws_bytes,
                              a.stream()),
                  {2, 3, 4, 5});
}

PyObject* moe_dispatch(const Args& a) {
  int64_t tokens, k, x_ld, out_ld;
  const int* row_of_slot = slots(a, 1, &tokens, &k);
  const at::ScalarType type = a.tensor(0).scalar_type();
  const void* x = a.matrix(0, type, tokens, -1, &x_ld);
  const int64_t dim = a.tensor(0).size(1), rows = a.tensor(2).numel();
  const int* slot_of_row = static_cast<int*>(a.whole(2, at::kInt, rows));
  void* out = a.matrix(3, type, rows, dim, &out_ld);
  return a.result(ns_moe_dispatch(x, x_ld, a.dtype(0), tokens, as_int(k), dim, row_of_slot, slot_of_row, rows, out,
                                  out_ld, a.stream()),
                  {3});
}

PyObject* moe_dispatch_grad(const Args& a) {
  int64_t tokens, k, rows_ld, x_ld;
  const int* row_of_slot = slots(a, 1, &tokens, &k);
  const at::ScalarType type = a.tensor(0).scalar_type();
  const void* grad_rows = a.matrix(0, type, -1, -1, &rows_ld);
  const int64_t rows = a.tensor(0).size(0), dim = a.tensor(0).size(1);
  void* grad_x = a.matrix(2, type, tokens, dim, &x_ld);
  return a.result(ns_moe_dispatch_grad(grad_rows, rows_ld, a.dtype(0), tokens, as_int(k), dim, row_of_slot, rows,
                                       grad_x, x_ld, a.stream()),
                  {2});
}

PyObject* moe_combine(const Args& a) {
  int64_t tokens, k, rows_ld, y_ld;
  const int* row_of_slot = slots(a, 2, &tokens, &k);
  const at::ScalarType type = a.tensor(0).scalar_type();
  const void* expert_rows = a.matrix(0, type, -1, -1, &rows_ld);
  const int64_t rows = a.tensor(0).size(0), dim = a.tensor(0).size(1);
  const float* weights = static_cast<float*>(a.whole(1, at::kFloat, tokens * k));
  void* y = a.matrix(3, type, tokens, dim, &y_ld);
  return a.result(ns_moe_combine(expert_rows, rows_ld, a.dtype(0), tokens, as_int(k), dim, row_of_slot, weights, rows,
                                 y, y_ld, a.stream()),
                  {3});
}

PyObject* moe_combine_grad(const Args& a) {
  int64_t tokens, k, y_ld, rows_ld, grad_ld;
  const int* row_of_slot = slots(a, 3, &tokens, &k);
  const at::ScalarType type = a.tensor(1).scalar_type();
  const int64_t rows = a.tensor(4).numel();
  const void* expert_rows = a.matrix(1, type, rows, -1, &rows_ld);
  const int64_t dim = a.tensor(1).size(1);
  const void* grad_y = a.matrix(0, type, tokens, dim, &y_ld);
  const float* weights = static_cast<float*>(a.whole(2, at::kFloat, tokens * k));
  const int* slot_of_row = static_cast<int*>(a.whole(4, at::kInt, rows));
  void* grad_rows = a.matrix(5, type, rows, dim, &grad_ld);
  float* grad_weights = static_cast<float*>(a.whole(6, at::kFloat, tokens * k));
  return a.result(ns_moe_combine_grad(grad_y, y_ld, expert_rows, rows_ld, a.dtype(1), tokens, as_int(k), dim,
                                      row_of_slot, slot_of_row, weights, rows, grad_rows, grad_ld, grad_weights,
                                      a.stream()),
                  {5, 6});
}

// Queries, keys and what has their shapes: addresses, and (token, head) strides.
struct Heads {
  int64_t tokens, dim, heads[2];
  at::ScalarType type;
  void* at[6];
  int64_t strides[12];
  int n = 0;

  void add(const Args& a, int i, int side) {
    const at::Tensor& t = a.gpu(i, 3);
    if (n == 0) {
      tokens = t.size(0);
      dim = t.size(2);
      type = t.scalar_type();
    }
    if (n < 2) heads[side] = t.size(1);
    if (t.scalar_type() != type || t.size(0) != tokens || t.size(1) != heads[side] || t.size(2) != dim)
      a.bad(i, std::string(c10::toString(type)) + " [" + std::to_string(tokens) + ", " + std::to_string(heads[side]) +
                   ", " + std::to_string(dim) + "]");
    if (t.stride(2) != 1 && dim > 1) a.bad(i, "contiguous heads");
    at[n] = a.address(i, t);
    strides[2 * n] = t.stride(0);
    strides[2 * n + 1] = t.stride(1);
    ++n;
  }
};

// Weights, table and positions, from argument `w` (q_weight) and `r` (table) on.
struct Rotation {
  const void *q_weight, *k_weight, *positions = nullptr;
  const float* table = nullptr;
  int weight_dtype, position_bytes = 4;
  int64_t rot_dim = 0, table_rows = 0;

  Rotation(const Args& a, const Heads& h, int w, int r) {
    const int first = a.given(w) ? w : w + 1;
    const at::ScalarType type = a.given(first) ? a.tensor(first).scalar_type() : h.type;
    if (type != h.type && type != at::kFloat) a.bad(first, std::string(c10::toString(h.type)) + " or Float");
    weight_dtype = type == at::kFloat ? NS_DT_FP32 : type == at::kHalf ? NS_DT_FP16 : NS_DT_BF16;
    q_weight = a.whole(w, type, h.dim);
    k_weight = a.whole(w + 1, type, h.dim);
    if (a.given(r)) {
      const at::Tensor& t = a.gpu(r, 2);
      table_rows = t.size(0);
      rot_dim = t.size(1);
      table = static_cast<float*>(a.whole(r, at::kFloat, table_rows * rot_dim));
    }
    if (a.given(r + 1)) positions = a.indices(r + 1, h.tokens, &position_bytes);
  }
};

PyObject* qk_norm_rope(const Args& a) {
  Heads h;
  for (int i = 0; i < 4; ++i) h.add(a, i, i & 1);
  const Rotation r(a, h, 4, 6);
  return a.result(ns_qk_norm_rope(h.at[0], h.at[1], h.at[2], h.at[3], h.strides, a.dtype(0), h.tokens,
                                  as_int(h.heads[0]), as_int(h.heads[1]), as_int(h.dim), as_int(r.rot_dim), a.flag(9),
                                  r.q_weight, r.k_weight, r.weight_dtype, a.real(8, 1e-6f), r.table, r.table_rows,
                                  r.positions, r.position_bytes, a.stream()),
                  {2, 3});
}

PyObject* qk_norm_rope_grad(const Args& a) {
  Heads h;
  for (int i : {2, 3, 4, 5, 0, 1}) h.add(a, i, i & 1);
  const Rotation r(a, h, 6, 10);
  uint64_t ws_bytes;
  void* ws = a.scratch(12, &ws_bytes);
  return a.result(ns_qk_norm_rope_grad(
      h.at[4], h.at[5], h.at[0], h.at[1], h.at[2], h.at[3], h.strides, a.dtype(2), h.tokens, as_int(h.heads[0]),
      as_int(h.heads[1]), as_int(h.dim), as_int(r.rot_dim), a.flag(14), r.q_weight, r.k_weight, r.weight_dtype,
      static_cast<float*>(a.whole(8, at::kFloat, h.dim)), static_cast<float*>(a.whole(9, at::kFloat, h.dim)),
      a.real(13, 1e-6f), r.table, r.table_rows, r.positions, r.position_bytes, ws, ws_bytes, a.stream()),
                  {4, 5, 8, 9});
}

// The student's and the teacher's logits, from arguments 0, 1 and 2.
struct Logits {
  const void *logits, *values, *ids;
  int64_t stride, tokens, vocab, top;
  int dtype, values_dtype, id_bytes;
  at::ScalarType type;

  explicit Logits(const Args& a) {
    type = a.tensor(0).scalar_type();
    logits = a.matrix(0, type, -1, -1, &stride);
    tokens = a.tensor(0).size(0);
    vocab = a.tensor(0).size(1);
    const at::Tensor& v = a.gpu(1, 2);
    top = v.size(1);
    dtype = a.dtype(0);
    values_dtype = a.dtype(1);
    values = a.whole(1, v.scalar_type(), tokens * top);
    if (a.tensor(2).sizes() != v.sizes()) a.bad(2, "the shape of teacher_values");
    ids = a.indices(2, tokens * top, &id_bytes);
  }
};

PyObject* distill_loss(const Args& a) {
  const Logits l(a);
  int64_t grad_ld = 0;
  void* grad = a.given(5) ? a.matrix(5, l.type, l.tokens, l.vocab, &grad_ld) : nullptr;
  return a.result(ns_distill_loss(l.logits, l.stride, l.dtype, l.tokens, l.vocab, l.values, l.values_dtype, l.ids,
                                  l.id_bytes, as_int(l.top), static_cast<float*>(a.whole(6, at::kFloat, l.tokens)),
                                  static_cast<float*>(a.whole(7, at::kFloat, l.tokens)), a.real(8, 1.0f),
                                  static_cast<float*>(a.whole(3, at::kFloat, l.tokens)),
                                  static_cast<float*>(a.whole(4, at::kFloat, l.tokens)), grad, grad_ld, a.stream()),
                  {3, 4, 5});
}

PyObject* distill_grad(const Args& a) {
  const Logits l(a);
  int64_t grad_ld = 0;
  void* grad = a.matrix(4, l.type, l.tokens, l.vocab, &grad_ld);
  return a.result(ns_distill_grad(l.logits, l.stride, l.dtype, l.tokens, l.vocab, l.values, l.values_dtype, l.ids,
                                  l.id_bytes, as_int(l.top), static_cast<float*>(a.whole(5, at::kFloat, l.tokens)),
                                  static_cast<float*>(a.whole(6, at::kFloat, l.tokens)), a.real(7, 1.0f),
                                  static_cast<float*>(a.whole(3, at::kFloat, l.tokens)), grad, grad_ld, a.stream()),
                  {4});
}

Signature g_signatures[] = {
    {"ns_moe_sort", 7, 10,
     {"expert_ids", "experts", "row_of_slot", "slot_of_row", "counts", "offsets", "workspace", "align", "capacity", "stream"}},
    {"ns_moe_dispatch", 4, 5, {"x", "row_of_slot", "slot_of_row", "out", "stream"}},
    {"ns_moe_dispatch_grad", 3, 4, {"grad_rows", "row_of_slot", "grad_x", "stream"}},
    {"ns_moe_combine", 4, 5, {"expert_rows", "weights", "row_of_slot", "y", "stream"}},
    {"ns_moe_combine_grad", 7, 8,
     {"grad_y", "expert_rows", "weights", "row_of_slot", "slot_of_row", "grad_rows", "grad_weights", "stream"}},
    {"ns_qk_norm_rope", 4, 11,
     {"q", "k", "q_out", "k_out", "q_weight", "k_weight", "table", "positions", "eps", "interleaved", "stream"}},
    {"ns_qk_norm_rope_grad", 6, 16,
     {"grad_q_out", "grad_k_out", "q", "k", "grad_q", "grad_k", "q_weight", "k_weight", "grad_q_weight", "grad_k_weight",
      "table", "positions", "workspace", "eps", "interleaved", "stream"}},
    {"ns_distill_loss", 5, 10,
     {"logits", "teacher_values", "teacher_ids", "loss", "lse", "grad_logits", "weights", "teacher_lse", "temperature", "stream"}},
    {"ns_distill_grad", 5, 9,
     {"logits", "teacher_values", "teacher_ids", "lse", "grad_logits", "weights", "teacher_lse", "temperature", "stream"}},
};

using Body = PyObject* (*)(const Args&);

// One Python call: no C++ exception leaves it.
template <int I, Body B>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  try {
    return B(Args(g_signatures[I], args, n, kwnames));
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define NS_METHOD(I, BODY, DOC) \
  {g_signatures[I].function, reinterpret_cast<PyCFunction>(call<I, BODY>), METH_FASTCALL | METH_KEYWORDS, DOC}

PyMethodDef g_methods[] = {
    NS_METHOD(0, moe_sort,
              "ns_moe_sort(expert_ids, experts, row_of_slot, slot_of_row, counts, offsets, workspace, align=1, "
              "capacity=0, stream=None)\n--\n\n"
              "Stable sort of the slots of expert_ids [tokens, k] by expert: writes row_of_slot [tokens, k],\n"
              "slot_of_row [rows], counts [experts] and offsets [experts + 1], all int32 (-1: no row, no slot).\n"
              "Negative ids go nowhere."),
    NS_METHOD(1, moe_dispatch,
              "ns_moe_dispatch(x, row_of_slot, slot_of_row, out, stream=None)\n--\n\n"
              "out [rows, dim]: the token of each row's slot, zero in rows without one."),
    NS_METHOD(2, moe_dispatch_grad,
              "ns_moe_dispatch_grad(grad_rows, row_of_slot, grad_x, stream=None)\n--\n\n"
              "grad_x [tokens, dim]: the sum of each token's kept rows of grad_rows."),
    NS_METHOD(3, moe_combine,
              "ns_moe_combine(expert_rows, weights, row_of_slot, y, stream=None)\n--\n\n"
              "y [tokens, dim]: the sum of each token's kept rows times their fp32 weights [tokens, k] (None: 1)."),
    NS_METHOD(4, moe_combine_grad,
              "ns_moe_combine_grad(grad_y, expert_rows, weights, row_of_slot, slot_of_row, grad_rows, grad_weights, "
              "stream=None)\n--\n\n"
              "grad_rows [rows, dim] = weight * grad_y of each row's token (zero in rows without a slot) and\n"
              "grad_weights [tokens, k] fp32. grad_rows may be expert_rows itself."),
    NS_METHOD(5, qk_norm_rope,
              "ns_qk_norm_rope(q, k, q_out, k_out, q_weight=None, k_weight=None, table=None, positions=None, "
              "eps=1e-6, interleaved=False, stream=None)\n--\n\n"
              "Root-mean-square norm of every head of q and k [tokens, heads, dim], then the rotation by table\n"
              "[positions, rot_dim] (cosines, then sines) at positions [tokens] (None: 0, 1, ...). Tokens and\n"
              "heads may be strided; the outputs may be the inputs."),
    NS_METHOD(6, qk_norm_rope_grad,
              "ns_qk_norm_rope_grad(grad_q_out, grad_k_out, q, k, grad_q, grad_k, q_weight=None, k_weight=None, "
              "grad_q_weight=None, grad_k_weight=None, table=None, positions=None, workspace=None, eps=1e-6, "
              "interleaved=False, stream=None)\n--\n\n"
              "Gradient of ns_qk_norm_rope: grad_q, grad_k and, where given, the fp32 weight gradients [dim]\n"
              "(these need the workspace)."),
    NS_METHOD(7, distill_loss,
              "ns_distill_loss(logits, teacher_values, teacher_ids, loss, lse, grad_logits=None, weights=None, "
              "teacher_lse=None, temperature=1.0, stream=None)\n--\n\n"
              "Divergence of the student's softmax from the teacher's top entries: loss and lse fp32 [tokens]\n"
              "and, if grad_logits is given, the gradient in the logits [tokens, vocab] in the same pass.\n"
              "grad_logits may be logits itself."),
    NS_METHOD(8, distill_grad,
              "ns_distill_grad(logits, teacher_values, teacher_ids, lse, grad_logits, weights=None, "
              "teacher_lse=None, temperature=1.0, stream=None)\n--\n\n"
              "The gradient alone, from the lse that ns_distill_loss wrote; other weights are fine, but the gradient of a\n"
              "token that the loss left out (weight 0 or no entry) is NaN once it counts."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_training", "Calls of the training-step operators on torch tensors.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__training() {
  for (Signature& s : g_signatures)
    for (int i = 0; i < s.count; ++i)
      if (!(s.keys[i] = PyUnicode_InternFromString(s.names[i]))) return nullptr;
  PyObject* lib = PyImport_ImportModule("newton_schulz_shape_gb300._lib");
  if (!lib) return nullptr;
  g_check = PyObject_GetAttrString(lib, "check");
  Py_DECREF(lib);
  return g_check ? PyModule_Create(&g_module) : nullptr;
}
