// Native side of the Python binding for calls of a few microseconds: reads the
// tensors' addresses, sizes and layouts, checks them and calls the C ABI.  Each
// function returns the call's status, or None where an argument is not exactly what
// the call takes: the caller's checks in Python then name it.
//
// A call takes about 0.4 us here besides the launch, 3.5 in Python.
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <vector>

namespace {

PyObject *g_device, *g_stream;           // torch's queries of the current device and of its stream

// The C ABI's functions, by their addresses in the library that the package loaded
enum Fn { kBalance, kBalanceBackward, kFp4, kInt4, kFp4Topk, kInt4Topk, kGradNorm, kGradClip, kFns };
const char* const kNames[kFns] = {
    "dg_route_balance", "dg_route_balance_backward", "dg_bf16_fp4_gemv_nt", "dg_bf16_int4_gemv_nt",
    "dg_m_grouped_bf16_fp4_gemv_nt_topk", "dg_m_grouped_bf16_int4_gemv_nt_topk", "dg_grad_norm", "dg_grad_clip"};
uintptr_t g_fn[kFns];

// The arguments of a call: tensors by their place, each checked as it is taken.
// Nothing is read any more after the first that does not fit (`ok`).
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args), ok(n == want) {}

  // the tensor at `i` with `dims` dimensions, on the device of all
  const at::Tensor* tensor(int i, int64_t dims) {
    if (!ok || !THPVariable_Check(args_[i])) return lost();
    const at::Tensor& t = THPVariable_Unpack(args_[i]);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.dim() != dims) return lost();
    const int device = (int)t.get_device();
    if (device_ < 0) device_ = device;
    return device == device_ ? &t : lost();
  }
  // a contiguous one of a type and sizes
  void* dense(int i, at::ScalarType type, std::initializer_list<int64_t> sizes, bool optional = false) {
    if (!ok || (optional && args_[i] == Py_None)) return nullptr;
    const at::Tensor* t = tensor(i, (int64_t)sizes.size());
    if (!t || t->scalar_type() != type || !t->sizes().equals(at::IntArrayRef(sizes)) || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  // rows of `cols` bf16 values that may lie apart; *ld: how far
  void* rows(int i, int64_t rows, int64_t cols, int* ld, bool optional = false) {
    *ld = (int)cols;
    if (!ok || (optional && args_[i] == Py_None)) return nullptr;
    const at::Tensor* t = tensor(i, 2);
    if (!t || t->scalar_type() != at::kBFloat16 || t->size(0) != rows || t->size(1) != cols) {
      ok = false;
      return nullptr;
    }
    const int64_t step = rows > 1 ? t->stride(0) : cols;
    if ((cols > 1 && t->stride(1) != 1) || step < cols || step >= (int64_t(1) << 31)) ok = false;
    *ld = (int)step;
    return t->data_ptr();
  }
  int integer(int i) {
    if (!ok) return 0;
    const long v = PyLong_Check(args_[i]) ? PyLong_AsLong(args_[i]) : -1;
    if (!PyLong_Check(args_[i]) || (v == -1 && PyErr_Occurred()) || v != (int)v) {
      PyErr_Clear();
      ok = false;
    }
    return (int)v;
  }
  float real(int i) {
    if (!ok || !(PyFloat_Check(args_[i]) || PyLong_Check(args_[i]))) return (float)(ok = false);
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)v;
  }
  // tensors of a list or tuple: fp32 or bf16, contiguous, on the device of all
  void list(int i, std::vector<void*>* at, std::vector<int>* types, std::vector<long long>* sizes) {
    if (!ok || !(PyList_Check(args_[i]) || PyTuple_Check(args_[i]))) {
      ok = false;
      return;
    }
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(args_[i]);
    PyObject** items = PySequence_Fast_ITEMS(args_[i]);
    at->reserve(n);
    types->reserve(n);
    sizes->reserve(n);
    for (Py_ssize_t k = 0; k < n && ok; ++k) {
      if (!THPVariable_Check(items[k])) {
        ok = false;
        break;
      }
      const at::Tensor& t = THPVariable_Unpack(items[k]);
      const bool f32 = t.scalar_type() == at::kFloat;
      if (t.layout() != at::kStrided || !t.is_cuda() || !(f32 || t.scalar_type() == at::kBFloat16) || !t.is_contiguous()) {
        ok = false;
        break;
      }
      if (device_ < 0) device_ = (int)t.get_device();
      ok = t.get_device() == device_;
      at->push_back(t.data_ptr());
      types->push_back(f32 ? 0 : 1);
      sizes->push_back(t.numel());
    }
  }
  // the stream given at `i`, or the current one; the tensors must be on the current device
  void* stream(int i) {
    if (!ok || device_ < 0) return lost();
    PyObject* here = PyObject_CallNoArgs(g_device);
    const long device = here ? PyLong_AsLong(here) : -1;
    Py_XDECREF(here);
    if (device != device_) return lost();
    if (args_[i] != Py_None) {
      if (!PyLong_Check(args_[i])) return lost();
      void* p = PyLong_AsVoidPtr(args_[i]);
      if (p == nullptr && PyErr_Occurred()) return lost();
      return p;
    }
    PyObject* index = PyLong_FromLong(device_);
    PyObject* raw = index ? PyObject_CallOneArg(g_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!raw) return lost();
    void* p = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (p == nullptr && PyErr_Occurred()) return lost();
    return p;
  }

 private:
  std::nullptr_t lost() {
    PyErr_Clear();
    ok = false;
    return nullptr;
  }
  PyObject* const* args_;
  int device_ = -1;

 public:
  bool ok;
};

// The call with the GIL released, as a status; None where an argument did not fit
template <typename F>
PyObject* finish(const Args& a, F call) {
  if (!a.ok) Py_RETURN_NONE;
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

// What torch throws (a tensor without memory) is for the checks in Python to name; before
// init() no call is made
template <typename F>
PyObject* guarded(F f) {
  if (!g_device) Py_RETURN_NONE;
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

constexpr auto kF = at::kFloat;
constexpr auto kI = at::kInt;
constexpr auto kB = at::kByte;

template <typename... T>
int call(Fn fn, T... args) {
  return reinterpret_cast<int (*)(T...)>(g_fn[fn])(args...);
}

int type_of(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? 0 : t.scalar_type() == at::kBFloat16 ? 1 : -1; }

// logits, topk_ids, seq_starts, loss, counts, score, scale, stream
PyObject* balance(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 8);
    const at::Tensor *x = a.tensor(0, 2), *ids = a.tensor(1, 2), *loss = a.tensor(3, 1);
    if (!a.ok || type_of(*x) < 0) Py_RETURN_NONE;
    const int64_t T = x->size(0), E = x->size(1), k = ids->size(1), S = loss->size(0);
    void* px = a.dense(0, x->scalar_type(), {T, E});
    void* pi = a.dense(1, kI, {T, k});
    void* ps = a.dense(2, kI, {S + 1}, S == 1);
    void* pl = a.dense(3, kF, {S});
    void* pc = a.dense(4, kI, {S, E});
    const int score = a.integer(5);
    const float scale = a.real(6);
    void* st = a.stream(7);
    if (T != (int)T || S != (int)S || E != (int)E || k != (int)k) Py_RETURN_NONE;
    return finish(a, [&] {
      return call(kBalance, px, type_of(*x), pi, ps, pl, pc, (int)T, (int)E, (int)k, (int)S, score, scale, st);
    });
  });
}

// logits, counts, seq_starts, grad_loss, c, grad_logits, top_k, score, scale, stream
PyObject* balance_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 10);
    const at::Tensor *x = a.tensor(0, 2), *counts = a.tensor(1, 2);
    if (!a.ok || type_of(*x) < 0) Py_RETURN_NONE;
    const int64_t T = x->size(0), E = x->size(1), S = counts->size(0);
    void* px = a.dense(0, x->scalar_type(), {T, E});
    void* pc = a.dense(1, kI, {S, E});
    void* ps = a.dense(2, kI, {S + 1}, S == 1);
    void* pg = a.dense(3, kF, {S}, true);
    void* po = a.dense(4, x->scalar_type(), {T, E}, true);
    void* pd = a.dense(5, x->scalar_type(), {T, E});
    const int k = a.integer(6), score = a.integer(7);
    const float scale = a.real(8);
    void* st = a.stream(9);
    if (T != (int)T || S != (int)S || E != (int)E) Py_RETURN_NONE;
    return finish(a, [&] {
      return call(kBalanceBackward, px, type_of(*x), pc, ps, pg, po, pd, (int)T, (int)E, k, (int)S, score, scale, st);
    });
  });
}

// x, b, sfb, c, d, stream
PyObject* fp4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 6);
    const at::Tensor *x = a.tensor(0, 2), *b = a.tensor(1, 2);
    if (!a.ok) Py_RETURN_NONE;
    const int64_t M = x->size(0), K = x->size(1), N = b->size(0);
    if (K % 128 != 0 || M != (int)M || N != (int)N || K != (int)K) Py_RETURN_NONE;
    int ldx, ldc, ldd;
    void* px = a.rows(0, M, K, &ldx);
    void* pb = a.dense(1, kB, {N, K / 2});
    void* ps = a.dense(2, kI, {K / 128, N});
    void* pc = a.rows(3, M, N, &ldc, true);
    void* pd = a.rows(4, M, N, &ldd);
    void* st = a.stream(5);
    return finish(a, [&] { return call(kFp4, px, ldx, pb, ps, pc, ldc, pd, ldd, (int)M, (int)N, (int)K, st); });
  });
}

// x, b, scales, zeros, c, d, stream
PyObject* int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 7);
    const at::Tensor *x = a.tensor(0, 2), *b = a.tensor(1, 2), *s = a.tensor(2, 2);
    if (!a.ok || type_of(*s) < 0) Py_RETURN_NONE;
    const int64_t M = x->size(0), K = x->size(1), N = b->size(0), groups = s->size(0);
    if (groups < 1 || K % groups != 0 || M != (int)M || N != (int)N || K != (int)K) Py_RETURN_NONE;
    int ldx, ldc, ldd;
    void* px = a.rows(0, M, K, &ldx);
    void* pb = a.dense(1, kB, {N, K / 2});
    void* ps = a.dense(2, s->scalar_type(), {groups, N});
    void* pz = a.dense(3, kB, {groups, N}, true);
    void* pc = a.rows(4, M, N, &ldc, true);
    void* pd = a.rows(5, M, N, &ldd);
    void* st = a.stream(6);
    return finish(a, [&] {
      return call(kInt4, px, ldx, pb, ps, type_of(*s), pz, (int)(K / groups), pc, ldc, pd, ldd, (int)M, (int)N, (int)K,
                  st);
    });
  });
}

// x, topk_ids, first_expert, b, sfb, c, d, stream
PyObject* fp4_topk(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 8);
    const at::Tensor *x = a.tensor(0, 2), *ids = a.tensor(1, 2), *b = a.tensor(3, 3);
    if (!a.ok) Py_RETURN_NONE;
    const int64_t R = x->size(0), K = x->size(1), T = ids->size(0), k = ids->size(1), G = b->size(0), N = b->size(1);
    if (K % 128 != 0 || T * k >= int64_t(1) << 31 || R != (int)R || N != (int)N || K != (int)K || G != (int)G)
      Py_RETURN_NONE;
    int ldx, ldc, ldd;
    void* px = a.rows(0, R, K, &ldx);
    void* pi = a.dense(1, kI, {T, k});
    const int first = a.integer(2);
    void* pb = a.dense(3, kB, {G, N, K / 2});
    void* ps = a.dense(4, kI, {G, K / 128, N});
    void* pc = a.rows(5, T * k, N, &ldc, true);
    void* pd = a.rows(6, T * k, N, &ldd);
    void* st = a.stream(7);
    return finish(a, [&] {
      return call(kFp4Topk, px, ldx, (int)R, pi, pb, ps, pc, ldc, pd, ldd, (int)T, (int)k, first, (int)G, (int)N, (int)K,
                  st);
    });
  });
}

// x, topk_ids, first_expert, b, scales, zeros, c, d, stream
PyObject* int4_topk(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 9);
    const at::Tensor *x = a.tensor(0, 2), *ids = a.tensor(1, 2), *b = a.tensor(3, 3), *s = a.tensor(4, 3);
    if (!a.ok || type_of(*s) < 0) Py_RETURN_NONE;
    const int64_t R = x->size(0), K = x->size(1), T = ids->size(0), k = ids->size(1), G = b->size(0), N = b->size(1);
    const int64_t groups = s->size(1);
    if (groups < 1 || K % groups != 0 || T * k >= int64_t(1) << 31 || R != (int)R || N != (int)N || K != (int)K ||
        G != (int)G)
      Py_RETURN_NONE;
    int ldx, ldc, ldd;
    void* px = a.rows(0, R, K, &ldx);
    void* pi = a.dense(1, kI, {T, k});
    const int first = a.integer(2);
    void* pb = a.dense(3, kB, {G, N, K / 2});
    void* ps = a.dense(4, s->scalar_type(), {G, groups, N});
    void* pz = a.dense(5, kB, {G, groups, N}, true);
    void* pc = a.rows(6, T * k, N, &ldc, true);
    void* pd = a.rows(7, T * k, N, &ldd);
    void* st = a.stream(8);
    return finish(a, [&] {
      return call(kInt4Topk, px, ldx, (int)R, pi, pb, ps, type_of(*s), pz, (int)(K / groups), pc, ldc, pd, ldd, (int)T,
                  (int)k, first, (int)G, (int)N, (int)K, st);
    });
  });
}

// grads, norm, stream
PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 3);
    std::vector<void*> at;
    std::vector<int> types;
    std::vector<long long> sizes;
    a.list(0, &at, &types, &sizes);
    void* norm = a.dense(1, kF, {1});
    void* st = a.stream(2);
    if (at.size() > 1u << 30) Py_RETURN_NONE;
    return finish(a, [&] {
      return call(kGradNorm, (const void* const*)at.data(), (const int*)types.data(), (const long long*)sizes.data(),
                  (int)at.size(), norm, st);
    });
  });
}

// grads, out, norm, max_norm, stream
PyObject* grad_clip(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 5);
    std::vector<void*> at, to;
    std::vector<int> types, to_types;
    std::vector<long long> sizes, to_sizes;
    a.list(0, &at, &types, &sizes);
    a.list(1, &to, &to_types, &to_sizes);
    void* norm = a.dense(2, kF, {1});
    const float most = a.real(3);
    void* st = a.stream(4);
    if (at.size() > 1u << 30 || types != to_types || sizes != to_sizes) Py_RETURN_NONE;
    return finish(a, [&] {
      return call(kGradClip, (const void* const*)at.data(), (void* const*)to.data(), (const int*)types.data(),
                  (const long long*)sizes.data(), (int)at.size(), norm, most, st);
    });
  });
}

// init({name: address}, current device, current raw stream): all of it, or nothing where
// an argument does not fit
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3 || !PyDict_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "init(addresses, current_device, current_raw_stream)");
    return nullptr;
  }
  uintptr_t fn[kFns];
  for (int i = 0; i < kFns; ++i) {
    PyObject* v = PyDict_GetItemString(args[0], kNames[i]);
    const unsigned long long at = v ? PyLong_AsUnsignedLongLong(v) : 0;
    if (PyErr_Occurred()) return nullptr;
    if (!at) {
      PyErr_Format(PyExc_ValueError, "no address of %s", kNames[i]);
      return nullptr;
    }
    fn[i] = (uintptr_t)at;
  }
  if (!PyCallable_Check(args[1]) || !PyCallable_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "the queries of the device and of its stream must be callable");
    return nullptr;
  }
  std::copy(fn, fn + kFns, g_fn);
  Py_INCREF(args[1]);
  Py_INCREF(args[2]);
  PyObject *device = g_device, *stream = g_stream;
  g_device = args[1];
  g_stream = args[2];
  Py_XDECREF(device);
  Py_XDECREF(stream);
  Py_RETURN_NONE;
}

#define DG_METHOD(NAME, FN) {NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(FN)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DG_METHOD("init", init),
                           DG_METHOD(kNames[kBalance], balance),
                           DG_METHOD(kNames[kBalanceBackward], balance_backward),
                           DG_METHOD(kNames[kFp4], fp4),
                           DG_METHOD(kNames[kInt4], int4),
                           DG_METHOD(kNames[kFp4Topk], fp4_topk),
                           DG_METHOD(kNames[kInt4Topk], int4_topk),
                           DG_METHOD(kNames[kGradNorm], grad_norm),
                           DG_METHOD(kNames[kGradClip], grad_clip),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
