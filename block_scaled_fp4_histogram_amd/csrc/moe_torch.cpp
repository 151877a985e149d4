// Python binding of the products, the gated block, the quantisers and the route grouping
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
decltype(&moe_grouped_glu) f_glu;
decltype(&moe_grouped_glu_dx) f_glu_dx;
decltype(&moe_glu_grad) f_glu_grad;
decltype(&moe_quant_fp8) f_quant_fp8;
decltype(&moe_grouped_fp8_mm) f_fp8;
decltype(&moe_grouped_fp8_glu) f_fp8_glu;
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
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
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

// An argument that a gated block's form takes, and the form of five in a row:
// activation, limit (None: no clamp), alpha, beta, layout.
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
int whole(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v < INT32_MIN || v > INT32_MAX ? -1 : (int)v;
}
moe_glu_form form(PyObject *const *a) {
  return {whole(a[0]), whole(a[4]), none(a[1]) ? 0.f : (float)number(a[1]), (float)number(a[2]), (float)number(a[3])};
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v;
}
// A given output among the operands (undefined: not given).
Tensor optional_out(Operands &ops, PyObject *given, const char *name, at::IntArrayRef shape, ScalarType type) {
  if (none(given)) return Tensor();
  return ops.add(tensor(given, name), name, {type}, shape);
}
PyObject *pair(PyObject *given0, const Tensor &t0, PyObject *given1, const Tensor &t1) {
  PyObject *p0 = result(given0, t0), *p1 = result(given1, t1), *r = p0 && p1 ? PyTuple_Pack(2, p0, p1) : nullptr;
  Py_XDECREF(p0);
  Py_XDECREF(p1);
  return r;
}
int64_t half(int64_t n, const char *name) {
  if (n % 2) refuse(PyExc_ValueError, std::string(name) + ": expected two branches, got " + std::to_string(n) + " rows");
  return n / 2;
}

// The groups of a product's rows, or one of all of them; the arguments are first and rows.
template <bool GROUPED>
struct Groups {
  const Tensor *first = nullptr, *rows = nullptr;
  int64_t R;
  Groups(Operands &ops, PyObject *const *a, int64_t E, int64_t T) : R(T) {
    if (!GROUPED) return;
    first = &tensor(a[0], "first");
    ops.add(*first, "first", {at::kInt}, {E + 1});
    if (none(a[1])) return;
    rows = &tensor_of(a[1], "rows", 1);
    R = rows->size(0);
    ops.add(*rows, "rows", {at::kInt}, {R});
  }
};

// (x, w[, first, rows], the form's five, keep_pre, out, out_dtype, pre, scratch) -> h or (h, pre)
template <bool GROUPED>
PyObject *glu(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, GROUPED ? 14 : 12, [&]() -> PyObject * {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2), &w = tensor_of(a[1], "w", GROUPED ? 3 : 2);
    const int64_t T = x.size(0), K = x.size(1), E = GROUPED ? w.size(0) : 1, I = half(w.size(w.dim() - 2), "w");
    const ScalarType type = x.scalar_type();
    ops.add(x, "x", {at::kBFloat16, at::kHalf}, x.sizes());
    if (GROUPED) ops.add(w, "w", {type}, {E, 2 * I, K});
    else ops.add(w, "w", {type}, {2 * I, K});
    const Groups<GROUPED> g(ops, a + 2, E, T);
    PyObject *const *o = a + (GROUPED ? 4 : 2);
    const moe_glu_form f = form(o);
    const bool keep = truth(o[5]) || !none(o[8]);
    const ScalarType ot = out_type(ops, o[6], o[7], type, {type, at::kFloat}, {g.R, I});
    Tensor pre = optional_out(ops, o[8], "pre", {g.R, 2 * I}, type);
    ops.check();
    const int e = size32(E, "E"), r = size32(g.R, "R"), i = size32(I, "I"), k = size32(K, "K");
    c10::DeviceGuard guard(x.device());
    const Tensor out = none(o[6]) ? make({g.R, I}, ot, x) : tensor(o[6], "out");
    if (keep && !pre.defined()) pre = make({g.R, 2 * I}, type, x);
    const Scratch s(o[9], f_mm_scratch(MOE_MM_GLU, e, r, i, k), x);
    done(f_glu(code(type), ptr(&x), T, (const int32_t *)ptr(g.rows), ptr(&w), (const int32_t *)ptr(g.first), e, r, i, k,
               &f, code(ot), out.data_ptr(), keep ? pre.data_ptr() : nullptr, s.p, s.bytes, stream_of(x)));
    return keep ? pair(o[6], out, o[8], pre) : result(o[6], out);
  });
}

// (dy, w, pre[, first], the form's five, keep_h, out, h, scratch) -> d_pre or (d_pre, h)
template <bool GROUPED>
PyObject *glu_dx(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, GROUPED ? 13 : 12, [&]() -> PyObject * {
    Operands ops;
    const Tensor &dy = tensor_of(a[0], "dy", 2), &w = tensor_of(a[1], "w", GROUPED ? 3 : 2), &pre = tensor_of(a[2], "pre", 2);
    const int64_t R = dy.size(0), N = dy.size(1), E = GROUPED ? w.size(0) : 1, I = w.size(w.dim() - 1);
    const ScalarType type = dy.scalar_type();
    ops.add(dy, "dy", {at::kBFloat16, at::kHalf}, dy.sizes());
    if (GROUPED) ops.add(w, "w", {type}, {E, N, I});
    else ops.add(w, "w", {type}, {N, I});
    ops.add(pre, "pre", {type}, {R, 2 * I});
    const Tensor *first = nullptr;
    if (GROUPED) first = &ops.add(tensor(a[3], "first"), "first", {at::kInt}, {E + 1});
    PyObject *const *o = a + (GROUPED ? 4 : 3);
    const moe_glu_form f = form(o);
    const bool keep = truth(o[5]) || !none(o[7]);
    Tensor out = optional_out(ops, o[6], "out", {R, 2 * I}, type), h = optional_out(ops, o[7], "h", {R, I}, type);
    ops.check();
    const int e = size32(E, "E"), r = size32(R, "R"), nn = size32(N, "N"), i = size32(I, "I");
    c10::DeviceGuard guard(dy.device());
    if (!out.defined()) out = make({R, 2 * I}, type, dy);
    if (keep && !h.defined()) h = make({R, I}, type, dy);
    const Scratch s(o[8], f_mm_scratch(MOE_MM_GLU_DX, e, r, nn, i), dy);
    done(f_glu_dx(code(type), ptr(&dy), ptr(&w), ptr(&pre), (const int32_t *)ptr(first), e, r, nn, i, &f, out.data_ptr(),
                  keep ? h.data_ptr() : nullptr, s.p, s.bytes, stream_of(dy)));
    return keep ? pair(o[6], out, o[7], h) : result(o[6], out);
  });
}

// (dh, pre, the form's five, keep_h, out, h) -> d_pre or (d_pre, h)
PyObject *glu_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    Operands ops;
    const Tensor &dh = tensor_of(a[0], "dh", 2), &pre = tensor_of(a[1], "pre", 2);
    const int64_t R = dh.size(0), I = dh.size(1);
    const ScalarType type = dh.scalar_type();
    ops.add(dh, "dh", {at::kBFloat16, at::kHalf}, dh.sizes());
    ops.add(pre, "pre", {type}, {R, 2 * I});
    const moe_glu_form f = form(a + 2);
    const bool keep = truth(a[7]) || !none(a[9]);
    Tensor out = optional_out(ops, a[8], "out", {R, 2 * I}, type), h = optional_out(ops, a[9], "h", {R, I}, type);
    ops.check();
    const int r = size32(R, "R"), i = size32(I, "I");
    c10::DeviceGuard guard(dh.device());
    if (!out.defined()) out = make({R, 2 * I}, type, dh);
    if (keep && !h.defined()) h = make({R, I}, type, dh);
    done(f_glu_grad(code(type), ptr(&dh), ptr(&pre), r, i, &f, out.data_ptr(), keep ? h.data_ptr() : nullptr, stream_of(dh)));
    return keep ? pair(a[8], out, a[9], h) : result(a[8], out);
  });
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// (x, out, scales) -> (codes, scales)
PyObject *quant_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject * {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2);
    const int64_t R = x.size(0), b = blocks(x.size(1));
    ops.add(x, "x", {at::kBFloat16, at::kHalf}, x.sizes());
    Tensor q = optional_out(ops, a[1], "out", x.sizes(), at::kFloat8_e4m3fn);
    Tensor s = optional_out(ops, a[2], "scales", {R, b}, at::kFloat);
    ops.check();
    const int rows = size32(R, "rows"), cols = size32(x.size(1), "cols");
    c10::DeviceGuard guard(x.device());
    if (!q.defined()) q = make(x.sizes(), at::kFloat8_e4m3fn, x);
    if (!s.defined()) s = make({R, b}, at::kFloat, x);
    done(f_quant_fp8(code(x.scalar_type()), ptr(&x), rows, cols, (uint8_t *)q.data_ptr(), (float *)s.data_ptr(), stream_of(x)));
    return pair(a[1], q, a[2], s);
  });
}

// (x, x_scales, w, w_scales[, first, rows][, the form's five], out, out_dtype, scratch, fast_sums)
template <bool GROUPED, bool GLU>
PyObject *fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8 + (GROUPED ? 2 : 0) + (GLU ? 5 : 0), [&] {
    Operands ops;
    const Tensor &x = tensor_of(a[0], "x", 2), &w = tensor_of(a[2], "w", GROUPED ? 3 : 2);
    const int64_t T = x.size(0), K = x.size(1), E = GROUPED ? w.size(0) : 1, W = w.size(w.dim() - 2);
    const int64_t N = GLU ? half(W, "w") : W;
    ops.add(x, "x", {at::kFloat8_e4m3fn}, x.sizes());
    const Tensor &xs = ops.add(tensor(a[1], "x_scales"), "x_scales", {at::kFloat}, {T, blocks(K)});
    if (GROUPED) ops.add(w, "w", {at::kFloat8_e4m3fn}, {E, W, K});
    else ops.add(w, "w", {at::kFloat8_e4m3fn}, {W, K});
    const Tensor &ws = tensor(a[3], "w_scales");
    const int64_t shape[4] = {E, 2, blocks(N), blocks(K)}, plain[3] = {E, blocks(N), blocks(K)};
    const at::IntArrayRef want = GLU ? at::IntArrayRef(shape, 4) : at::IntArrayRef(plain, 3);
    ops.add(ws, "w_scales", {at::kFloat}, GROUPED ? want : want.slice(1));
    const Groups<GROUPED> g(ops, a + 4, E, T);
    PyObject *const *o = a + (GROUPED ? 6 : 4);
    moe_glu_form f = {};
    if (GLU) f = form(o), o += 5;
    const ScalarType ot = out_type(ops, o[0], o[1], at::kBFloat16, {at::kBFloat16, at::kHalf, at::kFloat}, {g.R, N});
    const bool fast = truth(o[3]);
    if (fast && ot == at::kFloat) refuse(PyExc_TypeError, "fast_sums: fp32 results are summed in fp32");
    ops.check();
    const int e = size32(E, "E"), r = size32(g.R, "R"), nn = size32(N, "N"), k = size32(K, "K");
    const int sums = fast ? MOE_FP8_FAST_SUMS : 0, oc = code(ot) | sums;
    c10::DeviceGuard guard(x.device());
    const Tensor out = none(o[0]) ? make({g.R, N}, ot, x) : tensor(o[0], "out");
    const Scratch s(o[2], f_mm_scratch((GLU ? MOE_MM_FP8_GLU : MOE_MM_FP8) | sums, e, r, nn, k), x);
    const uint8_t *px = (const uint8_t *)ptr(&x), *pw = (const uint8_t *)ptr(&w);
    const float *pxs = (const float *)ptr(&xs), *pws = (const float *)ptr(&ws);
    const int32_t *first = (const int32_t *)ptr(g.first), *rows = (const int32_t *)ptr(g.rows);
    if (GLU) done(f_fp8_glu(px, pxs, T, rows, pw, pws, first, e, r, nn, k, &f, oc, out.data_ptr(), s.p, s.bytes, stream_of(x)));
    else done(f_fp8(px, pxs, T, rows, pw, pws, first, e, r, nn, k, oc, out.data_ptr(), s.p, s.bytes, stream_of(x)));
    return result(o[0], out);
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
    f_glu = (decltype(f_glu))get("moe_grouped_glu");
    f_glu_dx = (decltype(f_glu_dx))get("moe_grouped_glu_dx");
    f_glu_grad = (decltype(f_glu_grad))get("moe_glu_grad");
    f_quant_fp8 = (decltype(f_quant_fp8))get("moe_quant_fp8");
    f_fp8 = (decltype(f_fp8))get("moe_grouped_fp8_mm");
    f_fp8_glu = (decltype(f_fp8_glu))get("moe_grouped_fp8_glu");
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

#define NAMED(name, ...) {name, (PyCFunction)(void (*)(void))__VA_ARGS__, METH_FASTCALL, nullptr}
#define FAST(name) NAMED(#name, name)
PyMethodDef g_methods[] = {FAST(bind),       FAST(grouped_mm), FAST(grouped_mm_dx),   FAST(grouped_mm_dw), FAST(quant_int8),
                           FAST(int8_mm),    FAST(grouped_int8_mm), FAST(group_routes), FAST(glu_grad), FAST(quant_fp8),
                           NAMED("glu", glu<false>),       NAMED("grouped_glu", glu<true>),
                           NAMED("glu_dx", glu_dx<false>), NAMED("grouped_glu_dx", glu_dx<true>),
                           NAMED("fp8_mm", fp8<false, false>), NAMED("grouped_fp8_mm", fp8<true, false>),
                           NAMED("fp8_glu", fp8<false, true>), NAMED("grouped_fp8_glu", fp8<true, true>),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_products", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__products() { return PyModule_Create(&g_module); }
