// The binding's side of the calls that a decode or training step makes most often (cross attention, rotary
// positions), as a CPython module: argument checks, pointers and the stream are taken from the torch tensors here,
// since doing it in Python took longer (5-9 us a call) than the kernels of a small step.
//
// Every function returns the library's status, or -1 when an argument is not what the call takes (nothing has been
// launched then; fattn.py finds out which one and raises).  C++ exceptions (an allocation that fails) become torch's
// Python errors.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "fattn.h"

namespace {

// The library's entry points, as loaded by fattn.py.
struct Api {
  decltype(&fa_cross_fwd) cross_fwd;
  decltype(&fa_cross_workspace_bytes) cross_bytes;
  decltype(&fa_cross_bwd) cross_bwd;
  decltype(&fa_cross_bwd_workspace_bytes) cross_bwd_bytes;
  decltype(&fa_rope_axes) rope;
  decltype(&fa_rope_axes_paged) rope_paged;
} api{};

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte;
using Shape = std::initializer_list<int64_t>;

// Reads tensors out of Python arguments; after the first that does not fit, `ok` stays false.
struct Args {
  PyObject* const* argv;
  bool ok = true;
  int dev = -1;  // the current device, once a tensor on a GPU has been seen

  const at::Tensor* tensor(int i) {
    if (!ok || !THPVariable_Check(argv[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(argv[i]);
    if (!t.is_cuda()) {
      ok = false;
      return nullptr;
    }
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.get_device() != dev || !t.is_contiguous()) ok = false;
    return ok ? &t : nullptr;
  }
  // A contiguous tensor of this type and shape on the current device: its pointer.
  void* ptr(int i, at::ScalarType type, Shape shape) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape)) ok = false;
    return ok ? t->data_ptr() : nullptr;
  }
  void* ptr_or_none(int i, at::ScalarType type, Shape shape) {
    return argv[i] == Py_None ? nullptr : ptr(i, type, shape);
  }
  // bf16 or fp32 (then *fp32 = 1)
  void* out(int i, Shape shape, int* fp32) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    *fp32 = t->scalar_type() == kF32;
    if ((!*fp32 && t->scalar_type() != kBf16) || t->sizes() != at::IntArrayRef(shape)) ok = false;
    return ok ? t->data_ptr() : nullptr;
  }
  // The sizes of a bf16 tensor of `n` dimensions that fit an int.
  void* sized(int i, int n, int64_t* sizes) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != kBf16 || t->dim() != n) {
      ok = false;
      return nullptr;
    }
    for (int k = 0; k < n; ++k) {
      sizes[k] = t->size(k);
      if (sizes[k] > INT32_MAX) ok = false;
    }
    return ok ? t->data_ptr() : nullptr;
  }
  // A stream handle, or None: torch's current stream.
  void* stream(int i) {
    if (!ok) return nullptr;
    if (argv[i] == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void* s = PyLong_AsVoidPtr(argv[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return s;
  }
  float number(int i) {
    const double x = PyFloat_AsDouble(argv[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(x);
  }
  unsigned long long cycles(int i) {
    const unsigned long long x = PyLong_AsUnsignedLongLong(argv[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return x;
  }
};

// A plan (a ctypes structure) for head dimension d.
struct Plan {
  Py_buffer view{};
  const fa_rope_axes_plan_t* p = nullptr;
  Plan(PyObject* o, int64_t d) {
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      view.obj = nullptr;
    } else if (view.len == sizeof(fa_rope_axes_plan_t) &&
               static_cast<const fa_rope_axes_plan_t*>(view.buf)->d == d) {
      p = static_cast<const fa_rope_axes_plan_t*>(view.buf);
    }
  }
  ~Plan() {
    if (view.obj) PyBuffer_Release(&view);
  }
};

PyObject* status(long st) { return PyLong_FromLong(st); }

// The interpreter's lock is free while the library enqueues: a full launch queue makes the call wait for the GPU, and what
// the GPU is waiting for may be a host function or another thread's call that needs the lock.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
PyObject* enqueue(F f) {
  long st;
  {
    const Unlocked unlocked;
    st = f();
  }
  return status(st);
}

// Scratch for a call on torch's current stream: its memory returns to that stream's pool when the call has been queued.
at::Tensor scratch(size_t bytes, int dev) {
  return at::empty({static_cast<int64_t>(bytes)},
                   at::TensorOptions().dtype(kU8).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
}

// A workspace argument: a 1-dimensional uint8 tensor, or None.
void* workspace(Args& a, int i, size_t* bytes) {
  *bytes = 0;
  if (a.argv[i] == Py_None) return nullptr;
  const at::Tensor* t = a.tensor(i);
  if (!t || t->scalar_type() != kU8 || t->dim() != 1) {
    a.ok = false;
    return nullptr;
  }
  *bytes = static_cast<size_t>(t->numel());
  return t->data_ptr();
}

// q, k, v, o, lse, scale, kv_lens | None, workspace | None (allocated on the current stream), stream | None, cycles
PyObject* cross_fwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) return status(-1);
  Args a{argv};
  int64_t q[4], k[4];
  int fp32 = 0;
  void* pq = a.sized(0, 4, q);
  void* pk = a.sized(1, 4, k);
  if (!a.ok || k[0] != q[0] || k[3] != q[3]) return status(-1);
  void* pv = a.ptr(2, kBf16, {k[0], k[1], k[2], k[3]});
  void* po = a.out(3, {q[0], q[1], q[2], q[3]}, &fp32);
  void* lse = a.ptr(4, kF32, {q[0], q[1], q[2]});
  const float scale = a.number(5);
  void* lens = a.ptr_or_none(6, kI32, {q[0]});
  size_t bytes = 0;
  void* ws = workspace(a, 7, &bytes);
  void* stream = a.stream(8);
  const fa_cross_opts opts{fp32, a.cycles(9)};
  if (!a.ok) return status(-1);
  const int B = q[0], Hq = q[1], Hkv = k[1], Nq = q[2], Nk = k[2], d = q[3];
  return enqueue([&] {
    at::Tensor own;
    if (argv[7] == Py_None && (bytes = api.cross_bytes(B, Hq, Hkv, Nq, Nk, d)) > 0) {
      own = scratch(bytes, a.dev);
      ws = own.data_ptr();
    }
    return api.cross_fwd(pq, pk, pv, static_cast<const int*>(lens), po, static_cast<float*>(lse), B, Hq, Hkv, Nq, Nk, d,
                         scale, ws, bytes, stream, &opts);
  });
  END_HANDLE_TH_ERRORS
}

// q, k, v, o, dout, lse, dq, dk, dv, scale, kv_lens | None, workspace | None, stream | None, cycles
PyObject* cross_bwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) return status(-1);
  Args a{argv};
  int64_t q[4], k[4];
  void* pq = a.sized(0, 4, q);
  void* pk = a.sized(1, 4, k);
  if (!a.ok || k[0] != q[0] || k[3] != q[3]) return status(-1);
  int f0 = 0, f1 = 0, f2 = 0;
  void* pv = a.ptr(2, kBf16, {k[0], k[1], k[2], k[3]});
  void* po = a.ptr(3, kBf16, {q[0], q[1], q[2], q[3]});
  void* pdo = a.ptr(4, kBf16, {q[0], q[1], q[2], q[3]});
  void* lse = a.ptr(5, kF32, {q[0], q[1], q[2]});
  void* dq = a.out(6, {q[0], q[1], q[2], q[3]}, &f0);
  void* dk = a.out(7, {k[0], k[1], k[2], k[3]}, &f1);
  void* dv = a.out(8, {k[0], k[1], k[2], k[3]}, &f2);
  const float scale = a.number(9);
  void* lens = a.ptr_or_none(10, kI32, {q[0]});
  size_t bytes = 0;
  void* ws = workspace(a, 11, &bytes);
  void* stream = a.stream(12);
  const fa_bwd_opts opts{a.cycles(13)};
  if (!a.ok || f0 != f1 || f0 != f2) return status(-1);
  const int B = q[0], Hq = q[1], Hkv = k[1], Nq = q[2], Nk = k[2], d = q[3];
  return enqueue([&] {
    at::Tensor own;
    if (argv[11] == Py_None && (bytes = api.cross_bwd_bytes(B, Hq, Hkv, Nq, Nk, d)) > 0) {
      own = scratch(bytes, a.dev);
      ws = own.data_ptr();
    }
    return api.cross_bwd(pq, pk, pv, static_cast<const int*>(lens), po, pdo, static_cast<const float*>(lse), dq, dk, dv, B,
                         Hq, Hkv, Nq, Nk, d, scale, f0, ws, bytes, stream, &opts);
  });
  END_HANDLE_TH_ERRORS
}

// q, k | None, pos, plan, q_out, k_out | None, inverse, stream | None
PyObject* rope_axes(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return status(-1);
  Args a{argv};
  int64_t q[4], k[4] = {0, 0, 0, 0};
  void* pq = a.sized(0, 4, q);
  void *pk = nullptr, *ko = nullptr;
  if (a.ok && argv[1] != Py_None) {
    pk = a.sized(1, 4, k);
    if (!a.ok || k[0] != q[0] || k[2] != q[2] || k[3] != q[3]) return status(-1);
    ko = a.ptr(5, kBf16, {k[0], k[1], k[2], k[3]});
  } else if (argv[5] != Py_None) {
    return status(-1);
  }
  if (!a.ok) return status(-1);
  const Plan plan(argv[3], q[3]);
  if (!plan.p) return status(-1);
  void* pos = a.ptr(2, kI32, {plan.p->n_axes, q[0], q[2]});
  void* qo = a.ptr(4, kBf16, {q[0], q[1], q[2], q[3]});
  void* stream = a.stream(7);
  const int inverse = PyObject_IsTrue(argv[6]);
  if (!a.ok || inverse < 0) {
    PyErr_Clear();
    return status(-1);
  }
  return enqueue([&] {
    return api.rope(pq, pk, static_cast<const int*>(pos), qo, ko, q[0], q[1], k[1], q[2], plan.p, inverse, stream);
  });
  END_HANDLE_TH_ERRORS
}

// q, k, v, pos, plan, q_out, k_pages, v_pages, block_table, seq_lens, new_lens | None, stream | None
PyObject* rope_axes_paged(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) return status(-1);
  Args a{argv};
  int64_t q[4], k[4], pool[4];
  void* pq = a.sized(0, 4, q);
  void* pk = a.sized(1, 4, k);
  void* kp = a.sized(6, 4, pool);
  if (!a.ok || k[0] != q[0] || k[2] != q[2] || k[3] != q[3] || pool[1] != k[1] || pool[3] != q[3]) return status(-1);
  const at::Tensor* table = a.tensor(8);
  if (!table || table->dim() != 2) return status(-1);
  const int64_t max_pages = table->size(1);
  const Plan plan(argv[4], q[3]);
  if (!plan.p || max_pages > INT32_MAX) return status(-1);
  void* pv = a.ptr(2, kBf16, {k[0], k[1], k[2], k[3]});
  void* pos = a.ptr(3, kI32, {plan.p->n_axes, q[0], q[2]});
  void* qo = a.ptr(5, kBf16, {q[0], q[1], q[2], q[3]});
  void* vp = a.ptr(7, kBf16, {pool[0], pool[1], pool[2], pool[3]});
  void* bt = a.ptr(8, kI32, {q[0], max_pages});
  void* lens = a.ptr(9, kI32, {q[0]});
  void* news = a.ptr_or_none(10, kI32, {q[0]});
  void* stream = a.stream(11);
  if (!a.ok) return status(-1);
  return enqueue([&] {
    return api.rope_paged(pq, pk, pv, static_cast<const int*>(pos), qo, kp, vp, static_cast<const int*>(bt),
                          static_cast<const int*>(lens), static_cast<const int*>(news), q[0], q[1], k[1], q[2], pool[2],
                          max_pages, pool[0], plan.p, stream);
  });
  END_HANDLE_TH_ERRORS
}

// Addresses of fa_cross_fwd, fa_cross_workspace_bytes, fa_cross_bwd, fa_cross_bwd_workspace_bytes, fa_rope_axes,
// fa_rope_axes_paged in the loaded library.
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes 6 addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(argv[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  api.cross_fwd = reinterpret_cast<decltype(api.cross_fwd)>(p[0]);
  api.cross_bytes = reinterpret_cast<decltype(api.cross_bytes)>(p[1]);
  api.cross_bwd = reinterpret_cast<decltype(api.cross_bwd)>(p[2]);
  api.cross_bwd_bytes = reinterpret_cast<decltype(api.cross_bwd_bytes)>(p[3]);
  api.rope = reinterpret_cast<decltype(api.rope)>(p[4]);
  api.rope_paged = reinterpret_cast<decltype(api.rope_paged)>(p[5]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"cross_fwd", fast(cross_fwd), METH_FASTCALL, nullptr},
                         {"cross_bwd", fast(cross_bwd), METH_FASTCALL, nullptr},
                         {"rope_axes", fast(rope_axes), METH_FASTCALL, nullptr},
                         {"rope_axes_paged", fast(rope_axes_paged), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", FATTN_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
