// Python binding of the products, the quantiser and the route grouping
// (include/moe.h) for torch tensors: checks of the operands, outputs and scratch
// from torch's allocator, the current stream, and the call.  A few rows' product
// runs in a few microseconds, which the same steps in Python took longer than
// (10.1 us a call, 3.9 us here).  It calls the library through the addresses
// that bind() receives, so it works with whichever build was loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/torch.h>

#include <optional>
#include <string>

#include "moe.h"

namespace {

// Set by bind().
decltype(&moe_grouped_mm) f_mm;
decltype(&moe_grouped_mm_dx) f_dx;
decltype(&moe_grouped_mm_dw) f_dw;
decltype(&moe_mm_scratch_bytes) f_mm_scratch;
decltype(&moe_quant_int8) f_quant;
decltype(&moe_int8_mm) f_int8;
decltype(&moe_grouped_int8_mm) f_grouped_int8;
decltype(&moe_group_routes) f_group;
decltype(&moe_group_routes_scratch_bytes) f_group_scratch;
decltype(&moe_last_error) f_last_error;
PyObject *g_moe_error, *g_raw_stream;   // the package's exception; torch's stream handle of a device

struct Refused {
  PyObject *type;
  std::string text;
};
struct PythonError {};   // already set

[[noreturn]] void refuse(PyObject *type, const std::string &text) { throw Refused{type, text}; }

using at::Tensor;
using at::ScalarType;

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); i++) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
std::string type_text(ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return std::string("torch.") + c10::toString(t);
  }
}

bool none(PyObject *o) { return !o || o == Py_None; }

const Tensor &tensor(PyObject *o, const char *name) {
  if (none(o)) refuse(PyExc_ValueError, std::string(name) + " is required");
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

const Tensor &tensor_of(PyObject *o, const char *name, int64_t dim) {
  if (!none(o)) {
    const Tensor &t = tensor(o, name);
    if (t.dim() == dim) return t;
  }
  refuse(PyExc_ValueError, std::string(name) + " must be a tensor of " + std::to_string(dim) + " dimensions");
}

typedef std::initializer_list<ScalarType> Types;

void has_type(const Tensor &t, const char *name, Types types) {
  for (ScalarType s : types)
    if (t.scalar_type() == s) return;
  std::string text = std::string(name) + ": expected ";
  for (const ScalarType *s = types.begin(); s != types.end(); s++) text += (s != types.begin() ? " or " : "") + type_text(*s);
  refuse(PyExc_TypeError, text + ", got " + type_text(t.scalar_type()));
}

// The operands of one call: types and shapes as they are added, then that all
// are contiguous on one GPU and that autograd expects nothing of the call, which
// it does not see: a result without a history would lose gradients silently.
struct Operands {
  struct { const Tensor *t; const char *name; } list[8];
  int n = 0;
  const Tensor &add(const Tensor &t, const char *name, Types types, at::IntArrayRef shape) {
    has_type(t, name, types);
    if (t.sizes() != shape)
      refuse(PyExc_ValueError, std::string(name) + ": expected shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    list[n].t = &t;
    list[n++].name = name;
    return t;
  }
  void check() const {
    if (at::GradMode::is_enabled())
      for (int i = 0; i < n; i++)
        if (list[i].t->requires_grad())
          refuse(PyExc_ValueError, std::string(list[i].name) + " requires grad, and autograd does not record this call: make it " +
                                       "under torch.no_grad() or in an autograd.Function, and the gradients' calls yourself");
    for (int i = 0; i < n; i++) {
      const Tensor &t = *list[i].t;
      if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(list[i].name) + " must be contiguous");
      if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(list[i].name) + " must be a device tensor");
      if (t.device() != list[0].t->device())
        refuse(PyExc_ValueError, std::string(list[i].name) + " is on " + t.device().str() + ", " + list[0].name + " on " +
                                     list[0].t->device().str());
    }
  }
};

int code(ScalarType t) { return t == at::kBFloat16 ? MOE_T_BF16 : t == at::kHalf ? MOE_T_FP16 : MOE_T_FP32; }

// The output's type, and the given output among the operands.
ScalarType out_type(Operands &ops, PyObject *out, PyObject *dtype, ScalarType fallback, Types allowed, at::IntArrayRef shape) {
  std::optional<ScalarType> want;
  if (!none(dtype)) {
    if (!THPDtype_Check(dtype)) refuse(PyExc_TypeError, "out_dtype: expected a torch.dtype");
    want = reinterpret_cast<THPDtype *>(dtype)->scalar_type;
  }
  if (!none(out)) {
    const Tensor &t = tensor(out, "out");
    if (want && t.scalar_type() != *want)
      refuse(PyExc_TypeError, "out: expected " + type_text(*want) + ", got " + type_text(t.scalar_type()));
    ops.add(t, "out", allowed, shape);
    return t.scalar_type();
  }
  const ScalarType r = want ? *want : fallback;
  for (ScalarType s : allowed)
    if (r == s) return r;
  std::string text = "out_dtype: expected ";
  for (const ScalarType *s = allowed.begin(); s != allowed.end(); s++)
    text += (s != allowed.begin() ? " or " : "") + type_text(*s);
  refuse(PyExc_TypeError, text + ", got " + type_text(r));
}

Tensor make(at::IntArrayRef shape, ScalarType type, const Tensor &like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

struct Scratch {
  Tensor keep;
  void *p = nullptr;
  size_t bytes = 0;
  Scratch(PyObject *given, size_t need, const Tensor &like) {
    if (!none(given)) {
      keep = tensor(given, "scratch");
      has_type(keep, "scratch", {at::kByte});
      if (!keep.is_contiguous()) refuse(PyExc_ValueError, "scratch must be contiguous");
      if (!keep.is_cuda()) refuse(PyExc_ValueError, "scratch must be a device tensor");
      if (keep.device() != like.device())
        refuse(PyExc_ValueError, "scratch is on " + keep.device().str() + ", the operands on " + like.device().str());
    } else if (need) {
      keep = make({(int64_t)need}, at::kByte, like);
    } else {
      return;
    }
    p = keep.data_ptr();
    bytes = keep.numel();
  }
};

int size32(int64_t v, const char *name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is above 2^31 - 1");
  return (int)v;
}

// The current stream of t's device, with that device current in `guard`'s scope.
void *stream_of(const Tensor &t) {
  PyObject *index = PyLong_FromLong(t.get_device());
  PyObject *s = index ? PyObject_CallOneArg(g_raw_stream, index) : nullptr;
  Py_XDECREF(index);
  if (!s) throw PythonError();
  void *p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw PythonError();
  return p;
}

void done(int rc) {
  if (rc == MOE_OK) return;
  PyObject *e = PyObject_CallFunction(g_moe_error, "is", rc, f_last_error());
  if (e) {
    PyErr_SetObject(g_moe_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

// The output of a call that succeeded.  A given one has been written through its
// pointer: its version moves on, so that autograd reports a saved tensor that was
// overwritten (inference tensors have no version).
PyObject *result(PyObject *given, const Tensor &made) {
  if (none(given)) return THPVariable_Wrap(made);
  if (!made.is_inference()) made.unsafeGetTensorImpl()->bump_version();
  Py_INCREF(given);
  return given;
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const PythonError &) {
  } catch (...) {                        // torch's own, with their types: an allocation that fails, among others
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

const void *ptr(const Tensor *t) { return t ? t->const_data_ptr() : nullptr; }

// (x, w, first, rows, out, out_dtype, scratch)
PyObject *grouped_mm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2), &w = tensor_of(a[1], "w", 3), &first = tensor(a[2], "first");
    const int64_t T = x.size(0), K = x.size(1), E = w.size(0), N = w.size(1);
    const ScalarType type = x.scalar_type();
    ops.add(x, "x", {at::kBFloat16, at::kHalf}, x.sizes());
    ops.add(w, "w", {type}, {E, N, K});
    ops.add(first, "first", {at::kInt}, {E + 1});
    const Tensor *rows = nullptr;
    int64_t R = T;
    if (!none(a[3])) {
      rows = &tensor_of(a[3], "rows", 1);
      R = rows->size(0);
      ops.add(*rows, "rows", {at::kInt}, {R});
    }
    const ScalarType ot = out_type(ops, a[4], a[5], type, {type, at::kFloat}, {R, N});
    ops.check();
    const int e = size32(E, "E"), r = size32(R, "R"), nn = size32(N, "N"), k = size32(K, "K");
    c10::DeviceGuard guard(x.device());
    const Tensor out = none(a[4]) ? make({R, N}, ot, x) : tensor(a[4], "out");
    const Scratch s(a[6], f_mm_scratch(MOE_MM_FORWARD, e, r, nn, k), x);
    done(f_mm(code(type), ptr(&x), T, (const int32_t *)ptr(rows), ptr(&w), (const int32_t *)ptr(&first), e, r, nn, k,
              code(ot), out.data_ptr(), s.p, s.bytes, stream_of(x)));
    return result(a[4], out);
  });
}

// (dy, w, first, out, out_dtype, scratch)
PyObject *grouped_mm_dx(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    Operands ops;
    const Tensor &dy = tensor_of(a[0], "dy", 2), &w = tensor_of(a[1], "w", 3), &first = tensor(a[2], "first");
    const int64_t R = dy.size(0), N = dy.size(1), E = w.size(0), K = w.size(2);
    const ScalarType type = dy.scalar_type();
    ops.add(dy, "dy", {at::kBFloat16, at::kHalf}, dy.sizes());
    ops.add(w, "w", {type}, {E, N, K});
    ops.add(first, "first", {at::kInt}, {E + 1});
    const ScalarType ot = out_type(ops, a[3], a[4], type, {type, at::kFloat}, {R, K});
    ops.check();
    const int e = size32(E, "E"), r = size32(R, "R"), nn = size32(N, "N"), k = size32(K, "K");
    c10::DeviceGuard guard(dy.device());
    const Tensor out = none(a[3]) ? make({R, K}, ot, dy) : tensor(a[3], "out");
    const Scratch s(a[5], f_mm_scratch(MOE_MM_DX, e, r, nn, k), dy);
    done(f_dx(code(type), ptr(&dy), ptr(&w), (const int32_t *)ptr(&first), e, r, nn, k, code(ot), out.data_ptr(), s.p,
              s.bytes, stream_of(dy)));
    return result(a[3], out);
  });
}

// (dy, x, first, rows, out, out_dtype, accumulate, scratch)
PyObject *grouped_mm_dw(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    Operands ops;
    const Tensor &dy = tensor_of(a[0], "dy", 2), &x = tensor_of(a[1], "x", 2), &first = tensor_of(a[2], "first", 1);
    const int64_t R = dy.size(0), N = dy.size(1), T = x.size(0), K = x.size(1), E = first.size(0) - 1;
    const ScalarType type = dy.scalar_type();
    if (none(a[3]) && T != R)
      refuse(PyExc_ValueError, "x: expected " + std::to_string(R) + " rows as dy, got " + std::to_string(T));
    const int accumulate = PyObject_IsTrue(a[6]);
    if (accumulate < 0) throw PythonError();
    if (accumulate && none(a[4])) refuse(PyExc_ValueError, "accumulate needs out");
    ops.add(dy, "dy", {at::kBFloat16, at::kHalf}, dy.sizes());
    ops.add(x, "x", {type}, x.sizes());
    if (E < 1) refuse(PyExc_ValueError, "first: expected at least 2 offsets, got " + std::to_string(E + 1));
    ops.add(first, "first", {at::kInt}, {E + 1});
    const Tensor *rows = nullptr;
    if (!none(a[3])) {
      rows = &tensor(a[3], "rows");
      ops.add(*rows, "rows", {at::kInt}, {R});
    }
    const ScalarType ot = out_type(ops, a[4], a[5], type, {type, at::kFloat}, {E, N, K});
    ops.check();
    const int e = size32(E, "E"), r = size32(R, "R"), nn = size32(N, "N"), k = size32(K, "K");
    c10::DeviceGuard guard(dy.device());
    const Tensor out = none(a[4]) ? make({E, N, K}, ot, dy) : tensor(a[4], "out");
    const Scratch s(a[7], f_mm_scratch(MOE_MM_DW, e, r, nn, k), dy);
    done(f_dw(code(type), ptr(&dy), ptr(&x), T, (const int32_t *)ptr(rows), (const int32_t *)ptr(&first), e, r, nn, k,
              code(ot), accumulate, out.data_ptr(), s.p, s.bytes, stream_of(dy)));
    return result(a[4], out);
  });
}

// (x, out, scales) -> (codes, scales)
PyObject *quant_int8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject * {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2);
    ops.add(x, "x", {at::kBFloat16, at::kHalf}, x.sizes());
    if (!none(a[1])) ops.add(tensor(a[1], "out"), "out", {at::kChar}, x.sizes());
    if (!none(a[2])) ops.add(tensor(a[2], "scales"), "scales", {at::kFloat}, {x.size(0)});
    ops.check();
    const int rows = size32(x.size(0), "rows"), cols = size32(x.size(1), "cols");
    c10::DeviceGuard guard(x.device());
    const Tensor q = none(a[1]) ? make(x.sizes(), at::kChar, x) : tensor(a[1], "out");
    const Tensor s = none(a[2]) ? make({x.size(0)}, at::kFloat, x) : tensor(a[2], "scales");
    done(f_quant(code(x.scalar_type()), ptr(&x), rows, cols, (int8_t *)q.data_ptr(), (float *)s.data_ptr(), stream_of(x)));
    PyObject *pq = result(a[1], q), *ps = result(a[2], s), *r = pq && ps ? PyTuple_Pack(2, pq, ps) : nullptr;
    Py_XDECREF(pq);
    Py_XDECREF(ps);
    return r;
  });
}

// (x, x_scales, w, w_scales, out, out_dtype, scratch)
PyObject *int8_mm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2), &w = tensor_of(a[2], "w", 2);
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    ops.add(x, "x", {at::kChar}, x.sizes());
    const Tensor &xs = ops.add(tensor(a[1], "x_scales"), "x_scales", {at::kFloat}, {M});
    ops.add(w, "w", {at::kChar}, {N, K});
    const Tensor &ws = ops.add(tensor(a[3], "w_scales"), "w_scales", {at::kFloat}, {N});
    const ScalarType ot = out_type(ops, a[4], a[5], at::kBFloat16, {at::kBFloat16, at::kHalf, at::kFloat}, {M, N});
    ops.check();
    const int m = size32(M, "M"), nn = size32(N, "N"), k = size32(K, "K");
    c10::DeviceGuard guard(x.device());
    const Tensor out = none(a[4]) ? make({M, N}, ot, x) : tensor(a[4], "out");
    const Scratch s(a[6], f_mm_scratch(MOE_MM_INT8, 1, m, nn, k), x);
    done(f_int8((const int8_t *)ptr(&x), (const float *)ptr(&xs), (const int8_t *)ptr(&w), (const float *)ptr(&ws), m, nn,
                k, code(ot), out.data_ptr(), s.p, s.bytes, stream_of(x)));
    return result(a[4], out);
  });
}

// (x, x_scales, w, w_scales, first, rows, out, out_dtype, scratch)
PyObject *grouped_int8_mm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2), &w = tensor_of(a[2], "w", 3);
    const int64_t T = x.size(0), K = x.size(1), E = w.size(0), N = w.size(1);
    ops.add(x, "x", {at::kChar}, x.sizes());
    const Tensor &xs = ops.add(tensor(a[1], "x_scales"), "x_scales", {at::kFloat}, {T});
    ops.add(w, "w", {at::kChar}, {E, N, K});
    const Tensor &ws = ops.add(tensor(a[3], "w_scales"), "w_scales", {at::kFloat}, {E, N});
    const Tensor &first = ops.add(tensor(a[4], "first"), "first", {at::kInt}, {E + 1});
    const Tensor *rows = nullptr;
    int64_t R = T;
    if (!none(a[5])) {
      rows = &tensor_of(a[5], "rows", 1);
      R = rows->size(0);
      ops.add(*rows, "rows", {at::kInt}, {R});
    }
    const ScalarType ot = out_type(ops, a[6], a[7], at::kBFloat16, {at::kBFloat16, at::kHalf, at::kFloat}, {R, N});
    ops.check();
    const int e = size32(E, "E"), r = size32(R, "R"), nn = size32(N, "N"), k = size32(K, "K");
    c10::DeviceGuard guard(x.device());
    const Tensor out = none(a[6]) ? make({R, N}, ot, x) : tensor(a[6], "out");
    const Scratch s(a[8], f_mm_scratch(MOE_MM_INT8, e, r, nn, k), x);
    done(f_grouped_int8((const int8_t *)ptr(&x), (const float *)ptr(&xs), T, (const int32_t *)ptr(rows),
                        (const int8_t *)ptr(&w), (const float *)ptr(&ws), (const int32_t *)ptr(&first), e, r, nn, k,
                        code(ot), out.data_ptr(), s.p, s.bytes, stream_of(x)));
    return result(a[6], out);
  });
}

// (topk_ids, num_experts, scratch) -> (first, order, token, inverse)
PyObject *group_routes(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject * {
    Operands ops;
    const Tensor &ids = tensor_of(a[0], "topk_ids", 2);
    ops.add(ids, "topk_ids", {at::kInt}, ids.sizes());
    ops.check();
    const long E = PyLong_AsLong(a[1]);
    if (E == -1 && PyErr_Occurred()) throw PythonError();
    if (E < 1) refuse(PyExc_ValueError, "num_experts must be positive, got " + std::to_string(E));
    const int64_t T = ids.size(0), k = ids.size(1), R = T * k;
    const int t = size32(T, "T"), kk = size32(k, "top_k"), e = size32(E, "num_experts");
    c10::DeviceGuard guard(ids.device());
    // one allocation for the four
    const Tensor all = make({E + 1 + 3 * R}, at::kInt, ids);
    int32_t *p = (int32_t *)all.data_ptr();
    const Scratch s(a[2], f_group_scratch(t, kk, e), ids);
    done(f_group((const int32_t *)ptr(&ids), t, kk, e, p, p + E + 1, p + E + 1 + R, p + E + 1 + 2 * R, s.p, s.bytes,
                 stream_of(ids)));
    PyObject *r = PyTuple_New(4);
    if (!r) throw PythonError();
    for (int i = 0; i < 4; i++) {
      const int64_t at0 = i ? E + 1 + (i - 1) * R : 0;
      PyObject *o = THPVariable_Wrap(i == 3 ? all.as_strided({T, k}, {k, 1}, at0) : all.as_strided({i ? R : E + 1}, {1}, at0));
      if (!o) {
        Py_DECREF(r);
        throw PythonError();
      }
      PyTuple_SET_ITEM(r, i, o);
    }
    return r;
  });
}

// (addresses by name, exception class, stream handle function)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject * {
    auto get = [&](const char *name) {
      PyObject *v = PyDict_GetItemString(a[0], name);   // borrowed
      void *p = v ? PyLong_AsVoidPtr(v) : nullptr;
      if (!p) refuse(PyExc_ValueError, std::string("no address of ") + name);
      return p;
    };
    f_mm = (decltype(f_mm))get("moe_grouped_mm");
    f_dx = (decltype(f_dx))get("moe_grouped_mm_dx");
    f_dw = (decltype(f_dw))get("moe_grouped_mm_dw");
    f_mm_scratch = (decltype(f_mm_scratch))get("moe_mm_scratch_bytes");
    f_quant = (decltype(f_quant))get("moe_quant_int8");
    f_int8 = (decltype(f_int8))get("moe_int8_mm");
    f_grouped_int8 = (decltype(f_grouped_int8))get("moe_grouped_int8_mm");
    f_group = (decltype(f_group))get("moe_group_routes");
    f_group_scratch = (decltype(f_group_scratch))get("moe_group_routes_scratch_bytes");
    f_last_error = (decltype(f_last_error))get("moe_last_error");
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    g_moe_error = a[1];
    g_raw_stream = a[2];
    Py_RETURN_NONE;
  });
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(bind),       FAST(grouped_mm), FAST(grouped_mm_dx),   FAST(grouped_mm_dw), FAST(quant_int8),
                           FAST(int8_mm),    FAST(grouped_int8_mm), FAST(group_routes), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_products", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__products() { return PyModule_Create(&g_module); }
