// torch_calls.cpp -- the torch-facing calls of the low-rank adapters and of
// gradient clipping: checks of the tensors, outputs, workspace and the call
// into the HIP library, with no Python between them.  One token through an
// adapter costs the GPU 6 us and 48 gradients of a small model 10 us; the same
// checks written in Python took 13 us and 58 us, 590 us for 600 gradients.
//
// The library's functions are handed over by the ctypes binding (bind), so
// that both use the one library that was loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "snack.h"

namespace {

using at::Tensor;

struct library_t {
  decltype(&snack_lora_workspace) lora_workspace;
  decltype(&snack_lora_fwd) lora_fwd;
  decltype(&snack_lora_bwd) lora_bwd;
  decltype(&snack_grad_workspace) grad_workspace;
  decltype(&snack_grad_norm) grad_norm;
  decltype(&snack_grad_clip) grad_clip;
  PyObject* check;  // check(status, what) raises
} lib;

// Thrown after a Python error has been set.
struct refused {};

template <typename... Args>
[[noreturn]] void refuse(PyObject* kind, const char* format, Args... args) {
  PyErr_Format(kind, format, args...);
  throw refused();
}

void check(snack_status st, const char* what) {
  if (st == SNACK_OK) return;
  PyObject* r = PyObject_CallFunction(lib.check, "is", (int)st, what);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "%s: status %d", what, (int)st);
  throw refused();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: expected a tensor", name);
  return THPVariable_Unpack(o);
}
// None is an undefined tensor.
Tensor maybe(PyObject* o, const char* name) {
  return o == Py_None ? Tensor() : tensor(o, name);
}
void* ptr(const Tensor& t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; }
void* stream() { return c10::hip::getCurrentHIPStream().stream(); }

PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

Tensor bytes_on(const Tensor& like, size_t n) {
  return at::empty({(int64_t)n}, like.options().dtype(at::kByte));
}

// t has been written past torch: autograd has to know (inference tensors have
// no version).
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Calls f without the interpreter's lock.
template <typename F> snack_status unlocked(F f) {
  snack_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

template <typename F> PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ adapters
struct rows_t { Tensor t; int64_t ld; };

// x as a T x n matrix with contiguous rows, and its row stride.  must: x
// itself (an output); otherwise rows that do not lie so are copied.
rows_t rows(const Tensor& x, const char* name, int64_t T, int64_t n, const Tensor& like, bool must) {
  if (x.scalar_type() != like.scalar_type() || x.device() != like.device())
    refuse(PyExc_TypeError, "%s: expected the dtype and device of the activations", name);
  if (x.dim() != 2 || x.size(0) != T || x.size(1) != n)
    refuse(PyExc_ValueError, "%s: expected shape (%lld, %lld)", name, (long long)T, (long long)n);
  const int64_t ld = x.stride(0);
  if ((x.stride(1) != 1 && n > 1) || (ld < n && T > 1)) {
    if (must) refuse(PyExc_ValueError, "%s: rows must be contiguous and must not overlap", name);
    return {x.contiguous(), n};
  }
  return {x, T > 1 ? ld : n};
}

struct bank_t {
  snack_lora lora;
  snack_dtype dtype;
  int64_t T;
};

void check_list(const Tensor& v, const char* name, at::ScalarType type, int64_t n, const Tensor& x) {
  if (v.defined() && (v.scalar_type() != type || v.numel() != n || v.device() != x.device() ||
                      !v.is_contiguous()))
    refuse(PyExc_ValueError, "%s: expected %lld contiguous %s on the activations' device", name,
           (long long)n, c10::toString(type));
}

bank_t bank_of(const Tensor& x, const Tensor& ids, const Tensor& A, const Tensor& B,
               const Tensor& scale, const Tensor& ranks) {
  if (x.dim() != 2) refuse(PyExc_ValueError, "x: expected a matrix, got %d axes", (int)x.dim());
  if (A.dim() != 3 || B.dim() != 3 || A.size(0) != B.size(0) || A.size(1) != B.size(1))
    refuse(PyExc_ValueError, "A (L, R, K) and B (L, R, M) expected");
  const at::ScalarType type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16)
    refuse(PyExc_TypeError, "unsupported dtype %s", c10::toString(type));
  if (!x.is_cuda()) refuse(PyExc_TypeError, "the adapters run on the GPU only");
  if (A.scalar_type() != type || B.scalar_type() != type || A.device() != x.device() ||
      B.device() != x.device())
    refuse(PyExc_TypeError, "A and B must have the activations' dtype and device");
  if (!A.is_contiguous() || !B.is_contiguous())
    refuse(PyExc_ValueError, "A and B must be contiguous");
  const int64_t T = x.size(0), L = A.size(0), R = A.size(1), K = A.size(2), M = B.size(2);
  if (ids.dim() != 1) refuse(PyExc_ValueError, "ids: expected a vector");
  check_list(ids, "ids", at::kInt, T, x);
  check_list(scale, "scale", at::kFloat, L, x);
  check_list(ranks, "ranks", at::kInt, L, x);
  if (T > INT32_MAX || K > INT32_MAX || M > INT32_MAX || L > INT32_MAX || R > INT32_MAX)
    refuse(PyExc_ValueError, "a size does not fit 32 bits");
  return {{(int32_t)M, (int32_t)K, (int32_t)L, (int32_t)R, ptr(A), ptr(B), (const float*)ptr(scale),
           (const int32_t*)ptr(ranks)},
          type == at::kBFloat16 ? SNACK_BF16 : SNACK_F32, T};
}

void check_t(const Tensor& t, const bank_t& b, const Tensor& x) {
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != b.T || t.size(1) != b.lora.R ||
      !t.is_contiguous() || t.device() != x.device())
    refuse(PyExc_ValueError, "t: expected a contiguous float32 (%lld, %d) tensor on x's device",
           (long long)b.T, (int)b.lora.R);
}

// lora_fwd(x, ids, A, B, scale, ranks, base, out, t) -> out
PyObject* lora_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) refuse(PyExc_TypeError, "9 arguments expected");
    const Tensor &x0 = tensor(a[0], "x"), &ids = tensor(a[1], "ids"), &A = tensor(a[2], "A"),
                 &B = tensor(a[3], "B");
    const Tensor scale = maybe(a[4], "scale"), ranks = maybe(a[5], "ranks"),
                 base0 = maybe(a[6], "base"), t = maybe(a[8], "t");
    Tensor out = maybe(a[7], "out");
    const bank_t b = bank_of(x0, ids, A, B, scale, ranks);
    const int64_t M = b.lora.M;
    const c10::DeviceGuard guard(x0.device());
    const rows_t x = rows(x0, "x", b.T, b.lora.K, x0, false);
    int64_t ldy = M;
    if (out.defined()) ldy = rows(out, "out", b.T, M, x0, true).ld;
    else out = at::empty({b.T, M}, x0.options());
    rows_t base{Tensor(), M};
    if (base0.defined()) base = rows(base0, "base", b.T, M, x0, false);
    if (t.defined()) check_t(t, b, x0);
    size_t need = 0;
    check(lib.lora_workspace(&b.lora, b.dtype, (int32_t)b.T, 0, &need), "snack_lora_workspace");
    const Tensor ws = bytes_on(x0, need);
    void* s = stream();
    check(unlocked([&] {
            return lib.lora_fwd(&b.lora, b.dtype, (const int32_t*)ptr(ids), (int32_t)b.T, ptr(x.t),
                                x.ld, ptr(base.t), base.ld, ptr(out), ldy, (float*)ptr(t), ptr(ws),
                                need, s);
          }),
          "snack_lora_fwd");
    if (a[7] != Py_None) written(out);
    if (t.defined()) written(t);
    return wrap(out);
  });
}

// lora_bwd(dy, x, ids, A, B, scale, ranks, t, base, out, dx?, dA?, dB?) -> (dx, dA, dB)
PyObject* lora_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) refuse(PyExc_TypeError, "13 arguments expected");
    const Tensor &dy0 = tensor(a[0], "dy"), &x0 = tensor(a[1], "x"), &ids = tensor(a[2], "ids"),
                 &A = tensor(a[3], "A"), &B = tensor(a[4], "B");
    const Tensor scale = maybe(a[5], "scale"), ranks = maybe(a[6], "ranks"), t = maybe(a[7], "t"),
                 base0 = maybe(a[8], "base");
    const int want_dx = PyObject_IsTrue(a[10]), want_dA = PyObject_IsTrue(a[11]),
              want_dB = PyObject_IsTrue(a[12]);
    if (want_dx < 0 || want_dA < 0 || want_dB < 0) throw refused();
    const bank_t b = bank_of(x0, ids, A, B, scale, ranks);
    const int64_t M = b.lora.M, K = b.lora.K;
    const c10::DeviceGuard guard(x0.device());
    const rows_t x = rows(x0, "x", b.T, K, x0, false), dy = rows(dy0, "dy", b.T, M, x0, false);
    if (t.defined()) check_t(t, b, x0);
    Tensor dx, dA, dB;
    rows_t base{Tensor(), K};
    int64_t lddx = K;
    if (want_dx) {
      dx = maybe(a[9], "out");
      if (dx.defined()) lddx = rows(dx, "out", b.T, K, x0, true).ld;
      else dx = at::empty({b.T, K}, x0.options());
      if (base0.defined()) base = rows(base0, "base", b.T, K, x0, false);
    }
    if (want_dA) dA = at::empty(A.sizes(), A.options());
    if (want_dB) dB = at::empty(B.sizes(), B.options());
    size_t need = 0;
    check(lib.lora_workspace(&b.lora, b.dtype, (int32_t)b.T, 1, &need), "snack_lora_workspace");
    const Tensor ws = bytes_on(x0, need);
    void* s = stream();
    check(unlocked([&] {
            return lib.lora_bwd(&b.lora, b.dtype, (const int32_t*)ptr(ids), (const float*)ptr(t),
                                (int32_t)b.T, ptr(x.t), x.ld, ptr(dy.t), dy.ld, ptr(base.t),
                                base.ld, ptr(dx), lddx, ptr(dA), ptr(dB), ptr(ws), need, s);
          }),
          "snack_lora_bwd");
    if (want_dx && a[9] != Py_None) written(dx);
    PyObject* r = PyTuple_New(3);
    if (!r) throw refused();
    PyTuple_SET_ITEM(r, 0, wrap(dx));
    PyTuple_SET_ITEM(r, 1, wrap(dA));
    PyTuple_SET_ITEM(r, 2, wrap(dB));
    return r;
  });
}

// ------------------------------------------------------------------ clipping
struct list_t {
  PyObject* seq;
  explicit list_t(PyObject* o) : seq(PySequence_Fast(o, "a list of tensors expected")) {
    if (!seq) throw refused();
  }
  ~list_t() { Py_DECREF(seq); }
  list_t(const list_t&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  const Tensor& operator[](Py_ssize_t i) const {
    return tensor(PySequence_Fast_GET_ITEM(seq, i), "a gradient or its output");
  }
};

// The table of the list; outs NULL: in place.
std::vector<snack_grad> table_of(const list_t& grads, const list_t* outs) {
  const Py_ssize_t n = grads.size();
  if (outs && outs->size() != n)
    refuse(PyExc_ValueError, "%zd gradients but %zd outputs", n, outs->size());
  if (n > INT32_MAX) refuse(PyExc_ValueError, "too many gradients");
  std::vector<snack_grad> tab((size_t)n);
  const c10::Device dev = grads[0].device();
  if (!dev.is_cuda()) refuse(PyExc_TypeError, "gradients must be on the GPU");
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor& g = grads[i];
    const at::ScalarType type = g.scalar_type();
    if (type != at::kFloat && type != at::kBFloat16)
      refuse(PyExc_TypeError, "unsupported dtype %s", c10::toString(type));
    if (g.device() != dev) refuse(PyExc_TypeError, "gradients must be on one device");
    const bool dense = g.is_contiguous();
    if (!dense && !g.unsafeGetTensorImpl()->is_non_overlapping_and_dense())
      refuse(PyExc_ValueError, "a gradient must fill its memory without gaps or overlaps");
    void* out = nullptr;
    if (outs) {
      const Tensor& o = (*outs)[i];
      if (o.sizes() != g.sizes() || o.scalar_type() != type || o.device() != dev)
        refuse(PyExc_ValueError, "an output must have its gradient's shape, dtype and device");
      if (!(dense && o.is_contiguous()) && o.strides() != g.strides())
        refuse(PyExc_ValueError, "an output must have its gradient's strides");
      out = ptr(o);
    }
    tab[(size_t)i] = {ptr(g), out, g.numel(),
                      type == at::kBFloat16 ? SNACK_BF16 : SNACK_F32, 0};
  }
  return tab;
}

// clip(grads, outs or None, max_norm or None, eps) -> norm; max_norm None: the
// norm alone.
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) refuse(PyExc_TypeError, "4 arguments expected");
    const bool scale = a[2] != Py_None;
    const double max_norm = scale ? PyFloat_AsDouble(a[2]) : 0.0, eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw refused();
    const list_t grads(a[0]);
    if (grads.size() == 0) refuse(PyExc_ValueError, "no gradients");
    std::unique_ptr<list_t> outs;
    if (a[1] != Py_None) outs.reset(new list_t(a[1]));
    const std::vector<snack_grad> tab = table_of(grads, outs.get());
    const int32_t count = (int32_t)tab.size();
    const Tensor& first = grads[0];
    const c10::DeviceGuard guard(first.device());
    const Tensor norm = at::empty({}, first.options().dtype(at::kFloat));
    size_t need = 0;
    check(lib.grad_workspace(count, &need), "snack_grad_workspace");
    const Tensor ws = bytes_on(first, need);
    void* s = stream();
    check(unlocked([&] {
            return scale ? lib.grad_clip(tab.data(), count, (float)max_norm, (float)eps,
                                         (float*)ptr(norm), ptr(ws), need, s)
                         : lib.grad_norm(tab.data(), count, (float*)ptr(norm), ptr(ws), need, s);
          }),
          scale ? "snack_grad_clip" : "snack_grad_norm");
    if (scale) {
      const list_t& to = outs ? *outs : grads;
      for (Py_ssize_t i = 0; i < to.size(); ++i) written(to[i]);
    }
    return wrap(norm);
  });
}

// bind(check, addresses of the library's functions in library_t's order)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[6];
  PyObject* check;
  if (!PyArg_ParseTuple(args, "OKKKKKK", &check, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5]))
    return nullptr;
  lib.lora_workspace = (decltype(lib.lora_workspace))p[0];
  lib.lora_fwd = (decltype(lib.lora_fwd))p[1];
  lib.lora_bwd = (decltype(lib.lora_bwd))p[2];
  lib.grad_workspace = (decltype(lib.grad_workspace))p[3];
  lib.grad_norm = (decltype(lib.grad_norm))p[4];
  lib.grad_clip = (decltype(lib.grad_clip))p[5];
  Py_INCREF(check);
  lib.check = check;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"lora_fwd", (PyCFunction)(void (*)(void))lora_fwd, METH_FASTCALL, nullptr},
    {"lora_bwd", (PyCFunction)(void (*)(void))lora_bwd, METH_FASTCALL, nullptr},
    {"clip", (PyCFunction)(void (*)(void))clip, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module_def); }
