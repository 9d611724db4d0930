// torch_calls.cpp -- the torch-facing calls of the low-rank adapters, of
// gradient clipping, and of dropout, embedding, token log-probabilities and the
// losses: checks of the tensors, outputs, workspace and the call
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

#include <cstddef>
#include <cstring>
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
  decltype(&snack_dropout) dropout;
  decltype(&snack_embed_fwd) embed_fwd;
  decltype(&snack_embed_workspace) embed_workspace;
  decltype(&snack_embed_bwd) embed_bwd;
  decltype(&snack_logp_workspace) logp_workspace;
  decltype(&snack_logp_fwd) logp_fwd;
  decltype(&snack_logp_bwd) logp_bwd;
  decltype(&snack_seqs_workspace) seqs_workspace;
  decltype(&snack_preference) preference;
  decltype(&snack_policy_loss) policy_loss;
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

// ------------------------------------------------- dropout, tokens and losses
struct matrix_t { Tensor t; int64_t rows, cols, ld; };

// x of any shape as rows of its last axis, `ld` elements apart.  must: x itself
// (an output); otherwise what does not lie so is copied.
matrix_t matrix(const Tensor& x, const char* name, bool must) {
  const int64_t n = x.dim(), cols = n ? x.size(n - 1) : 1;
  if (x.is_contiguous()) return {x, cols ? x.numel() / cols : 0, cols, cols};
  bool fits = x.numel() == 0 || cols == 1 || x.stride(n - 1) == 1;
  int64_t rows = 1, ld = cols, next = 0;  // next: the stride that one more axis has to have
  for (int64_t d = n - 2; d >= 0; --d) {
    if (x.size(d) == 1) continue;
    if (rows == 1) ld = x.stride(d);
    else if (x.stride(d) != next) fits = false;
    rows *= x.size(d);
    next = x.stride(d) * x.size(d);
  }
  if (fits && (ld >= cols || rows <= 1)) return {x, rows, cols, rows > 1 ? ld : cols};
  if (must) refuse(PyExc_ValueError, "%s: rows must be contiguous, evenly apart and must not overlap", name);
  return {x.contiguous(), cols ? x.numel() / cols : 0, cols, cols};
}

snack_dtype dtype_of(const Tensor& x, const char* name) {
  const at::ScalarType type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16)
    refuse(PyExc_TypeError, "%s: unsupported dtype %s", name, c10::toString(type));
  if (!x.is_cuda()) refuse(PyExc_TypeError, "%s: expected a tensor on the GPU", name);
  return type == at::kBFloat16 ? SNACK_BF16 : SNACK_F32;
}

void same(const Tensor& t, const char* name, const Tensor& like, at::IntArrayRef sizes) {
  if (t.scalar_type() != like.scalar_type() || t.device() != like.device())
    refuse(PyExc_TypeError, "%s: expected dtype %s on the other tensors' device", name,
           c10::toString(like.scalar_type()));
  if (t.sizes() != sizes) refuse(PyExc_ValueError, "%s: unexpected shape", name);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw refused();
  return v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw refused();
  return v;
}

// Token numbers: int32 or int64, any shape.
struct tokens_t { Tensor t; int32_t bytes; };
tokens_t tokens(const Tensor& ids, const char* name, const Tensor& like) {
  if (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong)
    refuse(PyExc_TypeError, "%s: expected int32 or int64", name);
  if (ids.device() != like.device())
    refuse(PyExc_TypeError, "%s: expected on the other tensors' device", name);
  return {ids.contiguous(), ids.scalar_type() == at::kLong ? 8 : 4};
}

std::vector<int64_t> with_axis(at::IntArrayRef sizes, int64_t n) {
  std::vector<int64_t> v(sizes.begin(), sizes.end());
  v.push_back(n);
  return v;
}

PyObject* tuple(std::initializer_list<Tensor> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  if (!r) throw refused();
  Py_ssize_t i = 0;
  for (const Tensor& t : items) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

Tensor scratch(const Tensor& like, size_t n) { return n ? bytes_on(like, n) : Tensor(); }

// dropout(x, p, seed, step, step tensor or None, residual, out) -> out
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7) refuse(PyExc_TypeError, "7 arguments expected");
    const Tensor& x0 = tensor(a[0], "x");
    const double p = number(a[1]);
    const uint64_t seed = PyLong_AsUnsignedLongLongMask(a[2]);
    const uint64_t step = PyLong_AsUnsignedLongLongMask(a[3]);
    if (PyErr_Occurred()) throw refused();
    const Tensor more = maybe(a[4], "step"), res0 = maybe(a[5], "residual");
    Tensor out = maybe(a[6], "out");
    const snack_dtype dt = dtype_of(x0, "x");
    if (more.defined() && (more.scalar_type() != at::kLong || more.numel() != 1 ||
                           more.device() != x0.device()))
      refuse(PyExc_TypeError, "step: expected a number or one int64 on x's device");
    if (res0.defined()) same(res0, "residual", x0, x0.sizes());
    if (out.defined()) same(out, "out", x0, x0.sizes());
    const c10::DeviceGuard guard(x0.device());
    if (!out.defined()) out = at::empty(x0.sizes(), x0.options());
    matrix_t x = matrix(x0, "x", false), y = matrix(out, "out", true), r = x;
    if (res0.defined()) r = matrix(res0, "residual", false);
    const int64_t rows = x.rows, cols = x.cols;
    void* s = stream();
    check(unlocked([&] {
            return lib.dropout(dt, ptr(x.t), x.ld, res0.defined() ? ptr(r.t) : nullptr, r.ld,
                               ptr(out), y.ld, rows, cols, p, seed, step,
                               (const uint64_t*)ptr(more), s);
          }),
          "snack_dropout");
    if (a[6] != Py_None) written(out);
    return wrap(out);
  });
}

// embed_fwd(ids, weight, scale, out) -> out
PyObject* embed_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) refuse(PyExc_TypeError, "4 arguments expected");
    const Tensor &ids0 = tensor(a[0], "ids"), &w0 = tensor(a[1], "weight");
    const double scale = number(a[2]);
    Tensor out = maybe(a[3], "out");
    const snack_dtype dt = dtype_of(w0, "weight");
    if (w0.dim() != 2) refuse(PyExc_ValueError, "weight: expected a matrix");
    if (w0.size(0) > INT32_MAX || w0.size(1) > INT32_MAX)
      refuse(PyExc_ValueError, "a size does not fit 32 bits");
    const c10::DeviceGuard guard(w0.device());
    const tokens_t ids = tokens(ids0, "ids", w0);
    const std::vector<int64_t> sizes = with_axis(ids0.sizes(), w0.size(1));
    if (out.defined()) same(out, "out", w0, sizes);
    else out = at::empty(sizes, w0.options());
    const matrix_t w = matrix(w0, "weight", false), y = matrix(out, "out", true);
    void* s = stream();
    check(unlocked([&] {
            return lib.embed_fwd(dt, ptr(ids.t), ids.bytes, ids.t.numel(), ptr(w.t), w.ld,
                                 (int32_t)w0.size(0), (int32_t)w0.size(1), (float)scale, ptr(out),
                                 y.ld, s);
          }),
          "snack_embed_fwd");
    if (a[3] != Py_None) written(out);
    return wrap(out);
  });
}

// embed_bwd(dy, ids, rows, scale, base, out) -> out
PyObject* embed_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) refuse(PyExc_TypeError, "6 arguments expected");
    const Tensor &dy0 = tensor(a[0], "dy"), &ids0 = tensor(a[1], "ids");
    const long long V = PyLong_AsLongLong(a[2]);
    if (PyErr_Occurred()) throw refused();
    const double scale = number(a[3]);
    const Tensor base0 = maybe(a[4], "base");
    Tensor out = maybe(a[5], "out");
    const snack_dtype dt = dtype_of(dy0, "dy");
    if (dy0.dim() < 1) refuse(PyExc_ValueError, "dy: expected rows");
    const int64_t D = dy0.size(dy0.dim() - 1);
    if (V < 0 || V > INT32_MAX || D > INT32_MAX)
      refuse(PyExc_ValueError, "a size does not fit 31 bits");
    same(dy0, "dy", dy0, with_axis(ids0.sizes(), D));
    const c10::DeviceGuard guard(dy0.device());
    const tokens_t ids = tokens(ids0, "ids", dy0);
    if (base0.defined()) same(base0, "base", dy0, {V, D});
    if (out.defined()) same(out, "out", dy0, {V, D});
    else out = at::empty({V, D}, dy0.options());
    const matrix_t dy = matrix(dy0, "dy", false), w = matrix(out, "out", true);
    matrix_t base = w;
    if (base0.defined()) base = matrix(base0, "base", false);
    size_t need = 0;
    check(lib.embed_workspace(dt, ids.t.numel(), (int32_t)V, (int32_t)D, &need),
          "snack_embed_workspace");
    const Tensor ws = scratch(dy0, need);
    void* s = stream();
    check(unlocked([&] {
            return lib.embed_bwd(dt, ptr(ids.t), ids.bytes, ids.t.numel(), ptr(dy.t), dy.ld,
                                 (int32_t)V, (int32_t)D, (float)scale,
                                 base0.defined() ? ptr(base.t) : nullptr, base.ld, ptr(out), w.ld,
                                 ptr(ws), need, s);
          }),
          "snack_embed_bwd");
    if (a[5] != Py_None) written(out);
    return wrap(out);
  });
}

struct logits_t { matrix_t x; tokens_t t; int32_t V; int64_t T; snack_dtype dt; };

logits_t logits_of(const Tensor& x0, const Tensor& t0) {
  const snack_dtype dt = dtype_of(x0, "logits");
  if (x0.dim() < 1) refuse(PyExc_ValueError, "logits: expected rows");
  const int64_t V = x0.size(x0.dim() - 1);
  if (V < 1 || V > INT32_MAX) refuse(PyExc_ValueError, "logits: rows must have 1 to 2^31 - 1");
  same(x0, "targets and logits", x0, with_axis(t0.sizes(), V));
  return {matrix(x0, "logits", false), tokens(t0, "targets", x0), (int32_t)V, t0.numel(), dt};
}

// logp_fwd(logits, targets) -> (logp, norm)
PyObject* logp_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 2) refuse(PyExc_TypeError, "2 arguments expected");
    const Tensor &x0 = tensor(a[0], "logits"), &t0 = tensor(a[1], "targets");
    const c10::DeviceGuard guard(x0.device());
    const logits_t l = logits_of(x0, t0);
    const auto f32 = x0.options().dtype(at::kFloat);
    const Tensor logp = at::empty(t0.sizes(), f32), norm = at::empty(with_axis(t0.sizes(), 2), f32);
    size_t need = 0;
    check(lib.logp_workspace(l.dt, l.T, l.V, &need), "snack_logp_workspace");
    const Tensor ws = scratch(x0, need);
    void* s = stream();
    check(unlocked([&] {
            return lib.logp_fwd(l.dt, ptr(l.x.t), l.x.ld, l.T, l.V, ptr(l.t.t), l.t.bytes,
                                (float*)ptr(logp), (float*)ptr(norm), ptr(ws), need, s);
          }),
          "snack_logp_fwd");
    return tuple({logp, norm});
  });
}

// logp_bwd(dlogp, logits, targets, norm, out) -> out
PyObject* logp_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) refuse(PyExc_TypeError, "5 arguments expected");
    const Tensor &g0 = tensor(a[0], "dlogp"), &x0 = tensor(a[1], "logits"),
                 &t0 = tensor(a[2], "targets"), &n0 = tensor(a[3], "norm");
    Tensor out = maybe(a[4], "out");
    const c10::DeviceGuard guard(x0.device());
    const logits_t l = logits_of(x0, t0);
    for (const Tensor* t : {&g0, &n0})
      if (t->scalar_type() != at::kFloat || t->device() != x0.device())
        refuse(PyExc_TypeError, "dlogp and norm: expected float32 on the logits' device");
    if (g0.sizes() != t0.sizes() || n0.sizes() != at::IntArrayRef(with_axis(t0.sizes(), 2)))
      refuse(PyExc_ValueError, "dlogp: expected the targets' shape, norm: one axis of 2 more");
    const Tensor g = g0.contiguous(), norm = n0.contiguous();
    if (out.defined()) same(out, "out", x0, x0.sizes());
    else out = at::empty(x0.sizes(), x0.options());
    const matrix_t y = matrix(out, "out", true);
    void* s = stream();
    check(unlocked([&] {
            return lib.logp_bwd(l.dt, (const float*)ptr(g), ptr(l.x.t), l.x.ld, l.T, l.V,
                                ptr(l.t.t), l.t.bytes, (const float*)ptr(norm), ptr(out), y.ld, s);
          }),
          "snack_logp_bwd");
    if (a[4] != Py_None) written(out);
    return wrap(out);
  });
}

// The sequences of per-token tensors, and the tensors made contiguous.
struct answers_t {
  snack_seqs q;
  Tensor logps, starts, mask;
  size_t need;
};

Tensor per_token(PyObject* o, const char* name, const Tensor& logps) {
  Tensor t = maybe(o, name);
  if (!t.defined()) return t;
  same(t, name, logps, logps.sizes());
  return t.contiguous();
}

answers_t answers_of(PyObject* logps0, PyObject* starts0, PyObject* mask0) {
  answers_t r{};
  const Tensor& lp = tensor(logps0, "logps");
  if (lp.scalar_type() != at::kFloat || !lp.is_cuda())
    refuse(PyExc_TypeError, "logps: expected float32 on the GPU");
  if (lp.numel() > INT32_MAX) refuse(PyExc_ValueError, "too many tokens");
  r.logps = lp.contiguous();
  r.starts = maybe(starts0, "starts");
  int64_t S;
  if (r.starts.defined()) {
    if (r.starts.scalar_type() != at::kInt || r.starts.dim() != 1 || r.starts.numel() < 1 ||
        r.starts.device() != lp.device())
      refuse(PyExc_ValueError, "starts: expected a vector of int32 on the device of logps, one "
             "more than sequences");
    r.starts = r.starts.contiguous();
    S = r.starts.numel() - 1;
  } else {
    if (lp.dim() != 2 && lp.dim() != 1)
      refuse(PyExc_ValueError, "logps: without starts, a row for each sequence expected");
    S = lp.dim() == 2 ? lp.size(0) : 1;
  }
  if (S > INT32_MAX) refuse(PyExc_ValueError, "too many sequences");
  r.mask = maybe(mask0, "mask");
  if (r.mask.defined()) {
    if ((r.mask.scalar_type() != at::kBool && r.mask.scalar_type() != at::kByte) ||
        r.mask.device() != lp.device() || r.mask.sizes() != lp.sizes())
      refuse(PyExc_ValueError, "mask: expected bool or uint8 of the shape and device of logps");
    r.mask = r.mask.contiguous();
  }
  r.q = {(int32_t)S, (int32_t)lp.numel(), (const int32_t*)ptr(r.starts),
         r.mask.defined() && lp.numel() ? (const uint8_t*)ptr(r.mask) : nullptr};
  check(lib.seqs_workspace(r.q.S, r.q.T, &r.need), "snack_seqs_workspace");
  return r;
}

const float* dloss_of(PyObject* o, const Tensor& logps, Tensor& keep) {
  keep = maybe(o, "dloss");
  if (keep.defined() && (keep.scalar_type() != at::kFloat || keep.numel() != 1 ||
                         keep.device() != logps.device()))
    refuse(PyExc_TypeError, "dloss: expected one float32 on the device of logps");
  return (const float*)ptr(keep);
}

// preference(logps, starts, ref, mask, beta, smoothing, form, average, dloss, loss?, grad?)
//   -> (loss, rewards, grad)
PyObject* preference(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) refuse(PyExc_TypeError, "11 arguments expected");
    const answers_t b = answers_of(a[0], a[1], a[3]);
    const Tensor& lp0 = tensor(a[0], "logps");
    const Tensor ref = per_token(a[2], "ref", lp0);
    const long form = PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) throw refused();
    const snack_pref pref{number(a[4]), number(a[5]), (int32_t)form, truth(a[7])};
    const bool want_loss = truth(a[9]), want = truth(a[10]);
    Tensor dl;
    const float* dloss = dloss_of(a[8], lp0, dl);
    const c10::DeviceGuard guard(lp0.device());
    Tensor loss, rewards, grad;
    if (want_loss) {
      loss = at::empty({}, b.logps.options());
      rewards = at::empty({b.q.S / 2, 2}, b.logps.options());
    }
    if (want) grad = at::empty(lp0.sizes(), b.logps.options());
    const Tensor ws = scratch(b.logps, b.need);
    void* s = stream();
    check(unlocked([&] {
            return lib.preference(&b.q, &pref, (const float*)ptr(b.logps), (const float*)ptr(ref),
                                  dloss, (float*)ptr(loss), (float*)ptr(rewards),
                                  (float*)ptr(grad), ptr(ws), b.need, s);
          }),
          "snack_preference");
    return tuple({loss, rewards, grad});
  });
}

// policy(logps, old, advantages, starts, ref, mask, low, high, kl, by tokens?, sequence means?,
//        dloss, loss?, grad?) -> (loss, stats, grad)
PyObject* policy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 14) refuse(PyExc_TypeError, "14 arguments expected");
    const answers_t b = answers_of(a[0], a[3], a[5]);
    const Tensor& lp0 = tensor(a[0], "logps");
    const Tensor old = per_token(a[1], "old", lp0), ref = per_token(a[4], "ref", lp0);
    const snack_policy policy{number(a[6]), number(a[7]), number(a[8]), truth(a[9]), truth(a[10])};
    const Tensor& adv0 = tensor(a[2], "advantages");
    if (adv0.scalar_type() != at::kFloat || adv0.device() != lp0.device())
      refuse(PyExc_TypeError, "advantages: expected float32 on the device of logps");
    if (policy.by_token ? adv0.sizes() != lp0.sizes() : adv0.dim() != 1 || adv0.size(0) != b.q.S)
      refuse(PyExc_ValueError, "advantages: expected one for each %s",
             policy.by_token ? "token" : "sequence");
    const Tensor adv = adv0.contiguous();
    const bool want_loss = truth(a[12]), want = truth(a[13]);
    Tensor dl;
    const float* dloss = dloss_of(a[11], lp0, dl);
    const c10::DeviceGuard guard(lp0.device());
    Tensor loss, stats, grad;
    if (want_loss) {
      loss = at::empty({}, b.logps.options());
      stats = at::empty({2}, b.logps.options());
    }
    if (want) grad = at::empty(lp0.sizes(), b.logps.options());
    const Tensor ws = scratch(b.logps, b.need);
    void* s = stream();
    check(unlocked([&] {
            return lib.policy_loss(&b.q, &policy, (const float*)ptr(b.logps),
                                   (const float*)ptr(old), (const float*)ptr(ref),
                                   (const float*)ptr(adv), dloss, (float*)ptr(loss),
                                   (float*)ptr(stats), (float*)ptr(grad), ptr(ws), b.need, s);
          }),
          "snack_policy_loss");
    return tuple({loss, stats, grad});
  });
}

// bind(check, addresses of the library's functions in library_t's order)
PyObject* bind(PyObject*, PyObject* args) {
  constexpr Py_ssize_t N = offsetof(library_t, check) / sizeof(void*);
  if (PyTuple_GET_SIZE(args) != N + 1) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected", N + 1);
    return nullptr;
  }
  void* p[N];
  for (Py_ssize_t i = 0; i < N; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, i + 1));
    if (PyErr_Occurred()) return nullptr;
  }
  std::memcpy(&lib, p, sizeof(p));
  PyObject* check = PyTuple_GET_ITEM(args, 0);
  Py_INCREF(check);
  lib.check = check;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"lora_fwd", (PyCFunction)(void (*)(void))lora_fwd, METH_FASTCALL, nullptr},
    {"lora_bwd", (PyCFunction)(void (*)(void))lora_bwd, METH_FASTCALL, nullptr},
    {"clip", (PyCFunction)(void (*)(void))clip, METH_FASTCALL, nullptr},
    {"dropout", (PyCFunction)(void (*)(void))dropout, METH_FASTCALL, nullptr},
    {"embed_fwd", (PyCFunction)(void (*)(void))embed_fwd, METH_FASTCALL, nullptr},
    {"embed_bwd", (PyCFunction)(void (*)(void))embed_bwd, METH_FASTCALL, nullptr},
    {"logp_fwd", (PyCFunction)(void (*)(void))logp_fwd, METH_FASTCALL, nullptr},
    {"logp_bwd", (PyCFunction)(void (*)(void))logp_bwd, METH_FASTCALL, nullptr},
    {"preference", (PyCFunction)(void (*)(void))preference, METH_FASTCALL, nullptr},
    {"policy", (PyCFunction)(void (*)(void))policy, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module_def); }
