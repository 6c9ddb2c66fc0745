// Compiled marshalling of the Python calls of the FP8 expert operators and of the
// linear, gated and integer products: the same look at the tensors as in flint_moe.py (type, shape, layout, device), then the C
// ABI.  Those calls last a few microseconds, and a look of interpreted code as
// long again.  A call that does not fit returns LOOK and has done nothing: the
// interpreted path then names what is wrong, or takes the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "flint_moe.h"

namespace {

constexpr long LOOK = 1;  // no status of the library is positive

struct Entry {
  decltype(&flint_moe_route) route = nullptr;
  decltype(&flint_moe_group_pairs) group_pairs = nullptr;
  decltype(&flint_moe_quantize_rows) quantize_rows = nullptr;
  decltype(&flint_moe_block_gemm) block_gemm = nullptr;
  decltype(&flint_moe_combine) combine = nullptr;
} g_entry;

struct LinearEntry {
  decltype(&flint_moe_linear) linear = nullptr;
  decltype(&flint_moe_linear_backward) linear_backward = nullptr;
  decltype(&flint_moe_gated_linear) gated_linear = nullptr;
  decltype(&flint_moe_gated_linear_backward) gated_linear_backward = nullptr;
  decltype(&flint_moe_integer_quantize_rows) integer_quantize_rows = nullptr;
  decltype(&flint_moe_integer_gemm) integer_gemm = nullptr;
} g_linear;

PyObject* status(long v) { return PyLong_FromLong(v); }

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The current device if the tensor is on it, -1 otherwise.
int device_of(const at::Tensor& t) {
  if (!t.is_cuda()) return -1;
  const int d = t.get_device();
  return d == c10::cuda::current_device() ? d : -1;
}

bool plain(const at::Tensor* t, at::ScalarType type, int device) {
  return t != nullptr && t->is_cuda() && t->get_device() == device && t->scalar_type() == type && t->is_contiguous();
}
bool plain1(const at::Tensor* t, at::ScalarType type, int device, int64_t n) {
  return plain(t, type, device) && t->dim() == 1 && t->size(0) == n;
}
bool plain2(const at::Tensor* t, at::ScalarType type, int device, int64_t rows, int64_t cols) {
  return plain(t, type, device) && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols;
}
// FLINT_MOE_T_* of an activation type, -1 for another.
int act_type(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? FLINT_MOE_T_BF16 : t.scalar_type() == at::kFloat ? FLINT_MOE_T_F32 : -1;
}
bool fits_int(int64_t v) { return v >= 0 && v <= INT_MAX; }

bool to_int(PyObject* o, int* v) {
  const long x = PyLong_AsLong(o);
  if ((x == -1 && PyErr_Occurred()) || x < INT_MIN || x > INT_MAX) {
    PyErr_Clear();
    return false;
  }
  *v = (int)x;
  return true;
}
// The stream argument: None for torch's current one on `device`, or its handle as a number.
bool to_stream(PyObject* o, int device, flint_moe_stream_t* st) {
  if (o == Py_None) {
    *st = reinterpret_cast<flint_moe_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    return true;
  }
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *st = static_cast<flint_moe_stream_t>(p);
  return true;
}

// Without the interpreter's lock while it lives; an exception (a tensor without
// storage has no data pointer) takes the lock again on its way out.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F>
PyObject* call(F&& f) {
  int rc;
  {
    Unlocked unlocked;
    rc = f();
  }
  return status(rc);
}

// route(logits, ids, w, bias | None, score, n_groups, top_groups, group_score, renormalise, scale, stream)
PyObject* py_route(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 11 || g_entry.route == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *ids = tensor(a[1]), *w = tensor(a[2]);
  const at::Tensor* bias = a[3] == Py_None ? nullptr : tensor(a[3]);
  if (x == nullptr || ids == nullptr || x->dim() != 2 || ids->dim() != 2) return status(LOOK);
  const int dev = device_of(*x), type = act_type(*x);
  const int64_t T = x->size(0), E = x->size(1), k = ids->size(1);
  if (dev < 0 || type < 0 || !fits_int(T) || !fits_int(E) || !fits_int(k)) return status(LOOK);
  if (x->stride(1) != 1 && E != 1) return status(LOOK);
  if (!plain2(ids, at::kInt, dev, T, k) || !plain2(w, at::kFloat, dev, T, k)) return status(LOOK);
  if (a[3] != Py_None && !plain1(bias, at::kFloat, dev, E)) return status(LOOK);
  flint_moe_routing r;
  r.n_experts = (int)E;
  r.top_k = (int)k;
  r.renormalise = PyObject_IsTrue(a[8]);
  const double scale = PyFloat_AsDouble(a[9]);
  if (r.renormalise < 0 || (scale == -1.0 && PyErr_Occurred())) {
    PyErr_Clear();
    return status(LOOK);
  }
  r.scale = (float)scale;
  flint_moe_stream_t st;
  if (!to_int(a[4], &r.score) || !to_int(a[5], &r.n_groups) || !to_int(a[6], &r.top_groups) ||
      !to_int(a[7], &r.group_score) || !to_stream(a[10], dev, &st))
    return status(LOOK);
  return call([&] {
    return g_entry.route(&r, x->const_data_ptr(), type, T > 1 ? x->stride(0) : E, (int)T,
                         bias ? static_cast<const float*>(bias->const_data_ptr()) : nullptr,
                         static_cast<int32_t*>(ids->data_ptr()), static_cast<float*>(w->data_ptr()), st);
  });
} catch (...) {
  return status(LOOK);
}

// group_pairs(ids, offsets, order, pos, stream)
PyObject* py_group_pairs(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 5 || g_entry.group_pairs == nullptr) return status(LOOK);
  const at::Tensor *ids = tensor(a[0]), *offsets = tensor(a[1]), *order = tensor(a[2]), *pos = tensor(a[3]);
  if (ids == nullptr || offsets == nullptr || pos == nullptr) return status(LOOK);
  const int dev = device_of(*ids);
  const int64_t pairs = ids->numel(), E = offsets->numel() - 1;
  if (dev < 0 || !fits_int(pairs) || !fits_int(E)) return status(LOOK);
  if (!plain(ids, at::kInt, dev) || !plain1(offsets, at::kInt, dev, E + 1) || !plain1(order, at::kInt, dev, pairs) ||
      !plain(pos, at::kInt, dev) || pos->sizes() != ids->sizes())
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[4], dev, &st)) return status(LOOK);
  return call([&] {
    return g_entry.group_pairs(static_cast<const int32_t*>(ids->const_data_ptr()), (int)pairs, (int)E,
                               static_cast<int32_t*>(offsets->data_ptr()), static_cast<int32_t*>(order->data_ptr()),
                               static_cast<int32_t*>(pos->data_ptr()), st);
  });
} catch (...) {
  return status(LOOK);
}

// quantize_rows(x, q, scales, pos | None, silu_mul, stream)
PyObject* py_quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 6 || g_entry.quantize_rows == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *q = tensor(a[1]), *s = tensor(a[2]);
  const at::Tensor* pos = a[3] == Py_None ? nullptr : tensor(a[3]);
  if (x == nullptr || q == nullptr || x->dim() != 2 || q->dim() != 2) return status(LOOK);
  const int silu = PyObject_IsTrue(a[4]);
  if (silu < 0) {
    PyErr_Clear();
    return status(LOOK);
  }
  const int dev = device_of(*x), type = act_type(*x);
  const int64_t rows = x->size(0), width = x->size(1), places = q->size(0), K = q->size(1);
  if (dev < 0 || type < 0 || !fits_int(rows) || !fits_int(width) || !fits_int(places)) return status(LOOK);
  if (x->stride(1) != 1 || width != (silu ? 2 * K : K)) return status(LOOK);
  if (!plain(q, at::kFloat8_e4m3fn, dev) || !plain2(s, at::kFloat, dev, (K + 127) / 128, places)) return status(LOOK);
  int64_t k = 0;
  if (a[3] != Py_None) {
    if (pos == nullptr || pos->dim() != 2) return status(LOOK);
    k = pos->size(1);
    if (!fits_int(k) || !plain2(pos, at::kInt, dev, rows, k)) return status(LOOK);
  }
  flint_moe_stream_t st;
  if (!to_stream(a[5], dev, &st)) return status(LOOK);
  return call([&] {
    return g_entry.quantize_rows(x->const_data_ptr(), type, rows > 1 ? x->stride(0) : width, (int)rows, (int)K, silu,
                                 pos ? static_cast<const int32_t*>(pos->const_data_ptr()) : nullptr, (int)k,
                                 (int)places, q->data_ptr(), static_cast<float*>(s->data_ptr()), st);
  });
} catch (...) {
  return status(LOOK);
}

// block_gemm(a, a_scales, b, b_scales, y, offsets | None, stream)
PyObject* py_block_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 7 || g_entry.block_gemm == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *xs = tensor(a[1]), *w = tensor(a[2]), *ws = tensor(a[3]), *y = tensor(a[4]);
  const at::Tensor* offsets = a[5] == Py_None ? nullptr : tensor(a[5]);
  if (w == nullptr || ws == nullptr || y == nullptr || w->dim() != 3 || y->dim() != 2) return status(LOOK);
  const int dev = device_of(*y), type = act_type(*y);
  const int64_t E = w->size(0), N = w->size(1), K = w->size(2), M = y->size(0);
  if (dev < 0 || type < 0 || !fits_int(E) || !fits_int(N) || !fits_int(K) || !fits_int(M)) return status(LOOK);
  const int64_t kb = (K + 127) / 128, nb = (N + 127) / 128;
  if (y->size(1) != N || !y->is_contiguous() || !plain2(x, at::kFloat8_e4m3fn, dev, M, K) ||
      !plain2(xs, at::kFloat, dev, kb, M) || !plain(w, at::kFloat8_e4m3fn, dev))
    return status(LOOK);
  if (!plain(ws, at::kFloat, dev) || ws->dim() != 3 || ws->size(0) != E || ws->size(1) != nb || ws->size(2) != kb)
    return status(LOOK);
  if (a[5] != Py_None && !plain1(offsets, at::kInt, dev, E + 1)) return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[6], dev, &st)) return status(LOOK);
  return call([&] {
    return g_entry.block_gemm(x->const_data_ptr(), static_cast<const float*>(xs->const_data_ptr()), (int)M,
                              w->const_data_ptr(), static_cast<const float*>(ws->const_data_ptr()), (int)E,
                              offsets ? static_cast<const int32_t*>(offsets->const_data_ptr()) : nullptr, (int)N,
                              (int)K, y->data_ptr(), type, st);
  });
} catch (...) {
  return status(LOOK);
}

// combine(rows, pos, w, y, shared | None, stream)
PyObject* py_combine(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 6 || g_entry.combine == nullptr) return status(LOOK);
  const at::Tensor *rows = tensor(a[0]), *pos = tensor(a[1]), *w = tensor(a[2]), *y = tensor(a[3]);
  const at::Tensor* shared = a[4] == Py_None ? nullptr : tensor(a[4]);
  if (rows == nullptr || pos == nullptr || y == nullptr || rows->dim() != 2 || pos->dim() != 2 || y->dim() != 2)
    return status(LOOK);
  const int dev = device_of(*y), type = act_type(*rows);
  const int64_t T = y->size(0), N = y->size(1), k = pos->size(1), n_rows = rows->size(0);
  if (dev < 0 || type < 0 || !fits_int(T) || !fits_int(N) || !fits_int(k) || !fits_int(n_rows)) return status(LOOK);
  if (!plain2(y, at::kBFloat16, dev, T, N) || !plain2(rows, rows->scalar_type(), dev, n_rows, N) ||
      !plain2(pos, at::kInt, dev, T, k) || !plain2(w, at::kFloat, dev, T, k))
    return status(LOOK);
  if (a[4] != Py_None && !plain2(shared, at::kBFloat16, dev, T, N)) return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[5], dev, &st)) return status(LOOK);
  return call([&] {
    return g_entry.combine(rows->const_data_ptr(), type, (int)n_rows, static_cast<const int32_t*>(pos->const_data_ptr()),
                           static_cast<const float*>(w->const_data_ptr()), (int)T, (int)k, (int)N,
                           shared ? shared->const_data_ptr() : nullptr, y->data_ptr(), st);
  });
} catch (...) {
  return status(LOOK);
}

// A weight tensor [E][N][K] of this type on the current device (`dev` takes it).
bool weights(const at::Tensor* w, at::ScalarType type, int* dev, int64_t* E, int64_t* N, int64_t* K) {
  if (w == nullptr || w->dim() != 3 || (*dev = device_of(*w)) < 0) return false;
  *E = w->size(0);
  *N = w->size(1);
  *K = w->size(2);
  return fits_int(*E) && fits_int(*N) && fits_int(*K) && plain(w, type, *dev);
}
bool plain3(const at::Tensor* t, at::ScalarType type, int device, int64_t a, int64_t b, int64_t c) {
  return plain(t, type, device) && t->dim() == 3 && t->size(0) == a && t->size(1) == b && t->size(2) == c;
}
// An optional argument: None, or what `fits` takes.
template <typename F>
bool optional(PyObject* o, const at::Tensor** t, F&& fits) {
  *t = o == Py_None ? nullptr : tensor(o);
  return o == Py_None || (*t != nullptr && fits(*t));
}
const void* in(const at::Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
void* out(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
const int32_t* places(const at::Tensor* t) { return static_cast<const int32_t*>(in(t)); }

// linear(x, w, y, offsets | None, stream)
PyObject* py_linear(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 5 || g_linear.linear == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *y = tensor(a[2]), *offsets;
  int dev;
  int64_t E, N, K;
  if (x == nullptr || y == nullptr || x->dim() != 2 || !weights(w, at::kBFloat16, &dev, &E, &N, &K)) return status(LOOK);
  const int64_t M = x->size(0);
  const int type = act_type(*y);
  if (!fits_int(M) || type < 0 || !plain2(x, at::kBFloat16, dev, M, K) || !plain2(y, y->scalar_type(), dev, M, N) ||
      !optional(a[3], &offsets, [&](const at::Tensor* t) { return plain1(t, at::kInt, dev, E + 1); }))
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[4], dev, &st)) return status(LOOK);
  return call([&] {
    return g_linear.linear(in(x), (int)M, in(w), (int)E, places(offsets), (int)N, (int)K, out(y), type, st);
  });
} catch (...) {
  return status(LOOK);
}

// linear_backward(dy, x, w, dx | None, dw | None, offsets | None, stream)
PyObject* py_linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 7 || g_linear.linear_backward == nullptr) return status(LOOK);
  const at::Tensor *dy = tensor(a[0]), *x = tensor(a[1]), *w = tensor(a[2]), *dx, *dw, *offsets;
  int dev;
  int64_t E, N, K;
  if (dy == nullptr || dy->dim() != 2 || !weights(w, at::kBFloat16, &dev, &E, &N, &K)) return status(LOOK);
  const int64_t M = dy->size(0);
  if (!fits_int(M) || !plain2(dy, at::kBFloat16, dev, M, N) || !plain2(x, at::kBFloat16, dev, M, K) ||
      !optional(a[3], &dx, [&](const at::Tensor* t) { return plain2(t, at::kBFloat16, dev, M, K); }) ||
      !optional(a[4], &dw, [&](const at::Tensor* t) { return act_type(*t) >= 0 && plain3(t, t->scalar_type(), dev, E, N, K); }) ||
      !optional(a[5], &offsets, [&](const at::Tensor* t) { return plain1(t, at::kInt, dev, E + 1); }))
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[6], dev, &st)) return status(LOOK);
  const int type = dw ? act_type(*dw) : FLINT_MOE_T_BF16;
  return call([&] {
    return g_linear.linear_backward(in(dy), in(x), (int)M, in(w), (int)E, places(offsets), (int)N, (int)K, out(dx),
                                    out(dw), type, st);
  });
} catch (...) {
  return status(LOOK);
}

// gated_linear(x, w, h, gu | None, offsets | None, act, stream)
PyObject* py_gated_linear(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 7 || g_linear.gated_linear == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *h = tensor(a[2]), *gu, *offsets;
  int dev, act;
  int64_t E, N, K;
  if (x == nullptr || x->dim() != 2 || !weights(w, at::kBFloat16, &dev, &E, &N, &K) || N % 2) return status(LOOK);
  const int64_t M = x->size(0);
  if (!fits_int(M) || !plain2(x, at::kBFloat16, dev, M, K) || !plain2(h, at::kBFloat16, dev, M, N / 2) ||
      !optional(a[3], &gu, [&](const at::Tensor* t) { return plain2(t, at::kBFloat16, dev, M, N); }) ||
      !optional(a[4], &offsets, [&](const at::Tensor* t) { return plain1(t, at::kInt, dev, E + 1); }) ||
      !to_int(a[5], &act))
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[6], dev, &st)) return status(LOOK);
  return call([&] {
    return g_linear.gated_linear(in(x), (int)M, in(w), (int)E, places(offsets), (int)(N / 2), (int)K, act, out(h),
                                 out(gu), st);
  });
} catch (...) {
  return status(LOOK);
}

// gated_linear_backward(dh, gu, x, w, dgu, dx | None, dw | None, offsets | None, act, stream)
PyObject* py_gated_linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 10 || g_linear.gated_linear_backward == nullptr) return status(LOOK);
  const at::Tensor *dh = tensor(a[0]), *gu = tensor(a[1]), *x = tensor(a[2]), *w = tensor(a[3]), *dgu = tensor(a[4]);
  const at::Tensor *dx, *dw, *offsets;
  int dev, act;
  int64_t E, N, K;
  if (dh == nullptr || dh->dim() != 2 || !weights(w, at::kBFloat16, &dev, &E, &N, &K) || N % 2) return status(LOOK);
  const int64_t M = dh->size(0);
  if (!fits_int(M) || !plain2(dh, at::kBFloat16, dev, M, N / 2) || !plain2(gu, at::kBFloat16, dev, M, N) ||
      !plain2(x, at::kBFloat16, dev, M, K) || !plain2(dgu, at::kBFloat16, dev, M, N) ||
      !optional(a[5], &dx, [&](const at::Tensor* t) { return plain2(t, at::kBFloat16, dev, M, K); }) ||
      !optional(a[6], &dw, [&](const at::Tensor* t) { return act_type(*t) >= 0 && plain3(t, t->scalar_type(), dev, E, N, K); }) ||
      !optional(a[7], &offsets, [&](const at::Tensor* t) { return plain1(t, at::kInt, dev, E + 1); }) ||
      !to_int(a[8], &act))
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[9], dev, &st)) return status(LOOK);
  const int type = dw ? act_type(*dw) : FLINT_MOE_T_BF16;
  return call([&] {
    return g_linear.gated_linear_backward(in(dh), in(gu), in(x), (int)M, in(w), (int)E, places(offsets), (int)(N / 2),
                                          (int)K, act, out(dgu), out(dx), out(dw), type, st);
  });
} catch (...) {
  return status(LOOK);
}

// integer_quantize_rows(x, q, scales, pos | None, stream)
PyObject* py_integer_quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 5 || g_linear.integer_quantize_rows == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *q = tensor(a[1]), *s = tensor(a[2]), *pos;
  if (x == nullptr || q == nullptr || x->dim() != 2 || q->dim() != 2) return status(LOOK);
  const int dev = device_of(*x), type = act_type(*x);
  const int64_t rows = x->size(0), K = x->size(1), to = q->size(0);
  if (dev < 0 || type < 0 || !fits_int(rows) || !fits_int(K) || !fits_int(to) || x->stride(1) != 1) return status(LOOK);
  if (!plain2(q, at::kChar, dev, to, K) || !plain1(s, at::kFloat, dev, to)) return status(LOOK);
  if (!optional(a[3], &pos, [&](const at::Tensor* t) {
        return t->dim() == 2 && fits_int(t->size(1)) && plain2(t, at::kInt, dev, rows, t->size(1));
      }))
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[4], dev, &st)) return status(LOOK);
  return call([&] {
    return g_linear.integer_quantize_rows(in(x), type, rows > 1 ? x->stride(0) : K, (int)rows, (int)K, places(pos),
                                          pos ? (int)pos->size(1) : 0, (int)to, static_cast<int8_t*>(out(q)),
                                          static_cast<float*>(out(s)), st);
  });
} catch (...) {
  return status(LOOK);
}

// integer_gemm(a, a_scales, b, b_scales, y, offsets | None, act, stream)
PyObject* py_integer_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 8 || g_linear.integer_gemm == nullptr) return status(LOOK);
  const at::Tensor *x = tensor(a[0]), *xs = tensor(a[1]), *w = tensor(a[2]), *ws = tensor(a[3]), *y = tensor(a[4]);
  const at::Tensor* offsets;
  int dev, act;
  int64_t E, N, K;
  if (x == nullptr || y == nullptr || x->dim() != 2 || !weights(w, at::kChar, &dev, &E, &N, &K) || !to_int(a[6], &act))
    return status(LOOK);
  const int64_t M = x->size(0), width = act == FLINT_MOE_ACT_NONE ? N : N / 2;
  const int type = act_type(*y);
  if (act != FLINT_MOE_ACT_NONE && N % 2) return status(LOOK);
  if (!fits_int(M) || type < 0 || !plain2(x, at::kChar, dev, M, K) || !plain1(xs, at::kFloat, dev, M) ||
      !plain2(ws, at::kFloat, dev, E, N) || !plain2(y, y->scalar_type(), dev, M, width) ||
      !optional(a[5], &offsets, [&](const at::Tensor* t) { return plain1(t, at::kInt, dev, E + 1); }))
    return status(LOOK);
  flint_moe_stream_t st;
  if (!to_stream(a[7], dev, &st)) return status(LOOK);
  return call([&] {
    return g_linear.integer_gemm(static_cast<const int8_t*>(in(x)), static_cast<const float*>(in(xs)), (int)M,
                                 static_cast<const int8_t*>(in(w)), static_cast<const float*>(in(ws)), (int)E,
                                 places(offsets), (int)N, (int)K, act, out(y), type, st);
  });
} catch (...) {
  return status(LOOK);
}

// bind_linear(linear, linear_backward, gated_linear, gated_linear_backward, integer_quantize_rows, integer_gemm)
PyObject* py_bind_linear(PyObject*, PyObject* args) {
  unsigned long long f[6];
  if (!PyArg_ParseTuple(args, "KKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5])) return nullptr;
  g_linear.linear = reinterpret_cast<decltype(g_linear.linear)>(f[0]);
  g_linear.linear_backward = reinterpret_cast<decltype(g_linear.linear_backward)>(f[1]);
  g_linear.gated_linear = reinterpret_cast<decltype(g_linear.gated_linear)>(f[2]);
  g_linear.gated_linear_backward = reinterpret_cast<decltype(g_linear.gated_linear_backward)>(f[3]);
  g_linear.integer_quantize_rows = reinterpret_cast<decltype(g_linear.integer_quantize_rows)>(f[4]);
  g_linear.integer_gemm = reinterpret_cast<decltype(g_linear.integer_gemm)>(f[5]);
  Py_RETURN_NONE;
}

// bind(route, group_pairs, quantize_rows, block_gemm, combine): addresses of the library's entry points
PyObject* py_bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "KKKKK", &f[0], &f[1], &f[2], &f[3], &f[4])) return nullptr;
  g_entry.route = reinterpret_cast<decltype(g_entry.route)>(f[0]);
  g_entry.group_pairs = reinterpret_cast<decltype(g_entry.group_pairs)>(f[1]);
  g_entry.quantize_rows = reinterpret_cast<decltype(g_entry.quantize_rows)>(f[2]);
  g_entry.block_gemm = reinterpret_cast<decltype(g_entry.block_gemm)>(f[3]);
  g_entry.combine = reinterpret_cast<decltype(g_entry.combine)>(f[4]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(route),      FAST(group_pairs), FAST(quantize_rows),
                         FAST(block_gemm), FAST(combine),     {"bind", py_bind, METH_VARARGS, nullptr},
                         FAST(linear),     FAST(linear_backward), FAST(gated_linear), FAST(gated_linear_backward),
                         FAST(integer_quantize_rows), FAST(integer_gemm),
                         {"bind_linear", py_bind_linear, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_flint_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__flint_binding() { return PyModule_Create(&module_def); }
