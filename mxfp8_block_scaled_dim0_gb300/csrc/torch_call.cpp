// torch_call.cpp -- the allocating wrappers of the training operators, and of the 2D
// casts whose outputs they take, as plain CPython functions: they look the arguments
// over, allocate the outputs with torch's allocator and call the C ABI on torch's
// current stream.
//
// An operator on a few tokens takes the GPU two to five microseconds; a wrapper
// in Python takes 9 to 23 (a torch.empty alone 1.5 to 4).  These take 4 to 9, an
// allocation for every output included: outputs in one storage save up to a
// microsecond, but keeping or saving one then keeps or saves all.
//
// The first arguments are addresses of C ABI functions (of whichever build of
// the library the binding has loaded).  Each function returns its outputs, the
// C ABI's error code as an int, or None, before anything was done, where the
// arguments are not exactly what it knows (contiguous CUDA tensors of the right
// types and shapes on the current device) or a dispatch mode is on.  The binding's
// checked path then takes over, which works or raises the error that says what is
// wrong.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int kBF16 = 0, kF32 = 1;           // MX_BF16, MX_F32

template <typename F>
F address(PyObject* o) {
  return reinterpret_cast<F>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o)));
}

// The tensor behind a torch.Tensor or Parameter, or null.
const Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool is_bytes(ScalarType t) {
  return t == at::kByte || t == at::kFloat8_e4m3fn || t == at::kFloat8_e8m0fnu;
}

bool is_bool(PyObject* o) { return o == Py_True || o == Py_False; }

bool plain(const Tensor& t) { return t.layout() == at::kStrided && t.is_contiguous(); }

bool is_2d(const Tensor* t, ScalarType type) {
  return t && t->scalar_type() == type && t->dim() == 2 && plain(*t);
}

bool is_2d(const Tensor* t, ScalarType type, int64_t rows, int64_t cols) {
  return is_2d(t, type) && t->size(0) == rows && t->size(1) == cols;
}

bool is_1d(const Tensor* t, ScalarType type, int64_t n) {
  return t && t->scalar_type() == type && t->dim() == 1 && t->size(0) == n && plain(*t);
}

bool holds_bytes(const Tensor* t, int64_t n) {
  return t && is_bytes(t->scalar_type()) && plain(*t) && t->numel() >= n;
}

int64_t blocked_bytes(int64_t R, int64_t C) { return (R + 127) / 128 * 128 * ((C + 3) / 4 * 4); }

// Index of the current device if all tensors live there, or -1; -1 too where a
// dispatch mode is on: it shall see the allocations, which here go past the dispatcher.
int common_device(std::initializer_list<const Tensor*> ts) {
  if (c10::impl::TorchDispatchModeTLS::any_modes_set()) return -1;
  for (const Tensor* t : ts)
    if (t && !t->is_cuda()) return -1;
  const int dev = c10::cuda::current_device();
  for (const Tensor* t : ts)
    if (t && t->get_device() != dev) return -1;
  return dev;
}

Tensor empty(at::IntArrayRef size, ScalarType type, int dev) {
  return Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, static_cast<int8_t>(dev)),
                                       std::nullopt));
}

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

PyObject* wrapped(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = nullptr;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// The call without the interpreter lock (a full launch queue makes it wait).
template <typename F, typename... A>
int unlocked(F f, A... a) {
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS
  rc = f(a...);
  Py_END_ALLOW_THREADS
  return rc;
}

void* stream(int dev) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// Contiguous bytes (rows x cols), or the transpose of such a matrix.
bool operand(const Tensor* q, bool* by_column) {
  if (!q || !is_bytes(q->scalar_type()) || q->dim() != 2 || q->layout() != at::kStrided) return false;
  *by_column = false;
  if (q->is_contiguous()) return true;
  *by_column = true;
  return q->stride(0) == 1 && q->stride(1) == q->size(0);
}

// matmul(fn, qa, sa, qb, sb, out_type)
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  using Fn = int (*)(const void*, const void*, const void*, const void*, int64_t, int64_t, int64_t,
                     int32_t, void*, int32_t, void*);
  const Tensor *qa = tensor(a[1]), *sa = tensor(a[2]), *qb = tensor(a[3]), *sb = tensor(a[4]);
  const long type = PyLong_AsLong(a[5]);
  bool ca = false, cb = false;
  if (!operand(qa, &ca) || !operand(qb, &cb) || qa->size(1) != qb->size(1)) Py_RETURN_NONE;
  const int64_t M = qa->size(0), N = qb->size(0), K = qa->size(1);
  if (!holds_bytes(sa, blocked_bytes(M, K / 32)) || !holds_bytes(sb, blocked_bytes(N, K / 32)))
    Py_RETURN_NONE;
  const int dev = common_device({qa, sa, qb, sb});
  if (dev < 0) Py_RETURN_NONE;
  Tensor out = empty({M, N}, type == kF32 ? at::kFloat : at::kBFloat16, dev);
  const int rc = unlocked(address<Fn>(a[0]), ptr(qa), ptr(sa), ptr(qb), ptr(sb), M, N, K,
                          (ca ? 1 : 0) | (cb ? 2 : 0), out.data_ptr(), static_cast<int32_t>(type),
                          stream(dev));
  return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// layer_norm(fn, x, w, b or None, eps, save)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  using Fn = int (*)(const void*, const void*, const void*, int32_t, int64_t, int64_t, float, void*,
                     float*, float*, void*, void*, void*);
  const Tensor *x = tensor(a[1]), *w = tensor(a[2]), *b = tensor(a[3]);
  const double eps = PyFloat_CheckExact(a[4]) ? PyFloat_AS_DOUBLE(a[4]) : -1.0;
  const bool save = a[5] == Py_True;
  if (!is_2d(x, at::kBFloat16) || !w || (!b && a[3] != Py_None) || eps < 0 || !is_bool(a[5]))
    Py_RETURN_NONE;
  const int64_t M = x->size(0), D = x->size(1);
  const ScalarType wt = w->scalar_type();
  if ((wt != at::kFloat && wt != at::kBFloat16) || !is_1d(w, wt, D) || (b && !is_1d(b, wt, D)))
    Py_RETURN_NONE;
  const int dev = common_device({x, w, b});
  if (dev < 0) Py_RETURN_NONE;
  Tensor y = empty({M, D}, at::kBFloat16, dev), mean = empty({M}, at::kFloat, dev),
         rstd = empty({M}, at::kFloat, dev), q, s;
  if (save) {
    q = empty({M, D}, at::kByte, dev);
    s = empty({blocked_bytes(M, D / 32)}, at::kByte, dev);
  }
  const int rc = unlocked(address<Fn>(a[0]), ptr(x), ptr(w), ptr(b), wt == at::kFloat ? kF32 : kBF16,
                          M, D, static_cast<float>(eps), y.data_ptr(),
                          static_cast<float*>(mean.data_ptr()),
                          static_cast<float*>(rstd.data_ptr()), save ? q.data_ptr() : nullptr,
                          save ? s.data_ptr() : nullptr, stream(dev));
  if (rc) return PyLong_FromLong(rc);
  return save ? wrapped({y, mean, rstd, q, s}) : wrapped({y, mean, rstd});
  END_HANDLE_TH_ERRORS
}

// layer_norm_backward(fn, work_fn, dy, x or (q0, s0_blk), w, mean, rstd, bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  using Fn = int (*)(const void*, const void*, const void*, const void*, const void*, int32_t,
                     const float*, const float*, int64_t, int64_t, void*, void*, void*, void*, void*);
  const Tensor *dy = tensor(a[2]), *x = tensor(a[3]), *w = tensor(a[4]), *mean = tensor(a[5]),
               *rstd = tensor(a[6]), *q = nullptr, *s = nullptr;
  const bool bias = a[7] == Py_True;
  if (!is_2d(dy, at::kBFloat16) || !w || !is_bool(a[7])) Py_RETURN_NONE;
  const int64_t M = dy->size(0), D = dy->size(1);
  const ScalarType wt = w->scalar_type();
  if ((wt != at::kFloat && wt != at::kBFloat16) || !is_1d(w, wt, D) ||
      !is_1d(mean, at::kFloat, M) || !is_1d(rstd, at::kFloat, M))
    Py_RETURN_NONE;
  if (x) {
    if (!is_2d(x, at::kBFloat16, M, D)) Py_RETURN_NONE;
  } else {
    if (!PyTuple_CheckExact(a[3]) || PyTuple_GET_SIZE(a[3]) != 2) Py_RETURN_NONE;
    q = tensor(PyTuple_GET_ITEM(a[3], 0));
    s = tensor(PyTuple_GET_ITEM(a[3], 1));
    if (!holds_bytes(q, M * D) || !holds_bytes(s, blocked_bytes(M, D / 32))) Py_RETURN_NONE;
  }
  const int dev = common_device({dy, x, q, s, w, mean, rstd});
  if (dev < 0) Py_RETURN_NONE;
  Tensor dx = empty({M, D}, at::kBFloat16, dev), dw = empty({D}, wt, dev), db,
         work = empty({address<int64_t (*)(int64_t, int64_t)>(a[1])(M, D)}, at::kByte, dev);
  if (bias) db = empty({D}, wt, dev);
  const int rc = unlocked(address<Fn>(a[0]), ptr(dy), ptr(x), ptr(q), ptr(s), ptr(w),
                          wt == at::kFloat ? kF32 : kBF16, static_cast<const float*>(ptr(mean)),
                          static_cast<const float*>(ptr(rstd)), M, D, dx.data_ptr(), dw.data_ptr(),
                          bias ? db.data_ptr() : nullptr, work.data_ptr(), stream(dev));
  if (rc) return PyLong_FromLong(rc);
  return wrapped({dx, dw, db});
  END_HANDLE_TH_ERRORS
}

// swiglu(fn, gu, save)
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) Py_RETURN_NONE;
  using Fn = int (*)(const void*, int64_t, int64_t, void*, void*, void*, void*);
  const Tensor* gu = tensor(a[1]);
  const bool save = a[2] == Py_True;
  if (!is_2d(gu, at::kBFloat16) || gu->size(1) % 2 != 0 || !is_bool(a[2])) Py_RETURN_NONE;
  const int64_t M = gu->size(0), F = gu->size(1) / 2;
  const int dev = common_device({gu});
  if (dev < 0) Py_RETURN_NONE;
  Tensor h = empty({M, F}, at::kBFloat16, dev), q, s;
  if (save) {
    q = empty({M, 2 * F}, at::kByte, dev);
    s = empty({blocked_bytes(M, 2 * F / 32)}, at::kByte, dev);
  }
  const int rc = unlocked(address<Fn>(a[0]), ptr(gu), M, F, h.data_ptr(),
                          save ? q.data_ptr() : nullptr, save ? s.data_ptr() : nullptr, stream(dev));
  if (rc) return PyLong_FromLong(rc);
  return save ? wrapped({h, q, s}) : THPVariable_Wrap(h);
  END_HANDLE_TH_ERRORS
}

// swiglu_backward(fn, dh, gu or (q0, s0_blk))
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) Py_RETURN_NONE;
  using Fn = int (*)(const void*, const void*, const void*, const void*, int64_t, int64_t, void*,
                     void*);
  const Tensor *dh = tensor(a[1]), *gu = tensor(a[2]), *q = nullptr, *s = nullptr;
  if (!is_2d(dh, at::kBFloat16)) Py_RETURN_NONE;
  const int64_t M = dh->size(0), F = dh->size(1);
  if (gu) {
    if (!is_2d(gu, at::kBFloat16, M, 2 * F)) Py_RETURN_NONE;
  } else {
    if (!PyTuple_CheckExact(a[2]) || PyTuple_GET_SIZE(a[2]) != 2) Py_RETURN_NONE;
    q = tensor(PyTuple_GET_ITEM(a[2], 0));
    s = tensor(PyTuple_GET_ITEM(a[2], 1));
    if (!holds_bytes(q, 2 * M * F) || !holds_bytes(s, blocked_bytes(M, 2 * F / 32))) Py_RETURN_NONE;
  }
  const int dev = common_device({dh, gu, q, s});
  if (dev < 0) Py_RETURN_NONE;
  Tensor out = empty({M, 2 * F}, at::kBFloat16, dev);
  const int rc = unlocked(address<Fn>(a[0]), ptr(dh), ptr(gu), ptr(q), ptr(s), M, F, out.data_ptr(),
                          stream(dev));
  return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// cast_dim0(fn, x), cast_dim1(fn, x): one direction's bytes and scales.
template <bool DIM1>
PyObject* cast(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) Py_RETURN_NONE;
  using Fn = int (*)(const void*, int64_t, int64_t, void*, void*, void*);
  const Tensor* x = tensor(a[1]);
  if (!is_2d(x, at::kBFloat16)) Py_RETURN_NONE;
  const int64_t M = x->size(0), K = x->size(1), R = DIM1 ? K : M, C = DIM1 ? M : K;
  const int dev = common_device({x});
  if (dev < 0) Py_RETURN_NONE;
  Tensor q = empty({R, C}, at::kByte, dev), s = empty({blocked_bytes(R, C / 32)}, at::kByte, dev);
  const int rc = unlocked(address<Fn>(a[0]), ptr(x), M, K, q.data_ptr(), s.data_ptr(), stream(dev));
  return rc ? PyLong_FromLong(rc) : wrapped({q, s});
  END_HANDLE_TH_ERRORS
}

// cast_dim0_dim1(fn, x)
PyObject* cast_both(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) Py_RETURN_NONE;
  using Fn = int (*)(const void*, int64_t, int64_t, void*, void*, void*, void*, void*);
  const Tensor* x = tensor(a[1]);
  if (!is_2d(x, at::kBFloat16)) Py_RETURN_NONE;
  const int64_t M = x->size(0), K = x->size(1);
  const int dev = common_device({x});
  if (dev < 0) Py_RETURN_NONE;
  Tensor q0 = empty({M, K}, at::kByte, dev), s0 = empty({blocked_bytes(M, K / 32)}, at::kByte, dev),
         q1 = empty({K, M}, at::kByte, dev), s1 = empty({blocked_bytes(K, M / 32)}, at::kByte, dev);
  const int rc = unlocked(address<Fn>(a[0]), ptr(x), M, K, q0.data_ptr(), s0.data_ptr(),
                          q1.data_ptr(), s1.data_ptr(), stream(dev));
  return rc ? PyLong_FromLong(rc) : wrapped({q0, s0, q1, s1});
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"cast_dim0", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cast<false>)), METH_FASTCALL,
     nullptr},
    {"cast_dim1", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cast<true>)), METH_FASTCALL,
     nullptr},
    {"cast_dim0_dim1", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cast_both)),
     METH_FASTCALL, nullptr},
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(matmul)), METH_FASTCALL, nullptr},
    {"layer_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(layer_norm)), METH_FASTCALL,
     nullptr},
    {"layer_norm_backward",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(layer_norm_backward)), METH_FASTCALL,
     nullptr},
    {"swiglu", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(swiglu)), METH_FASTCALL, nullptr},
    {"swiglu_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(swiglu_backward)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_call", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_call(void) { return PyModule_Create(&kModule); }
