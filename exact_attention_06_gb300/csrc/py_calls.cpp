// The binding's side of the calls that a decode or training step makes most often (cross attention, sliding windows,
// rotary positions and norms, the cache's pages), as a CPython module: argument checks, pointers and the stream are taken from the torch tensors here,
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
  decltype(&fa_window_fwd) window_fwd;
  decltype(&fa_window_bwd) window_bwd;
  decltype(&fa_window_bwd_workspace_bytes) window_bwd_bytes;
  decltype(&fa_window_decode_paged) window_decode;
  decltype(&fa_window_decode_paged_workspace_bytes) window_decode_bytes;
  decltype(&fa_norm_rope_axes) norm_rope;
  decltype(&fa_norm_rope_axes_bwd) norm_rope_bwd;
  decltype(&fa_norm_rope_axes_bwd_workspace_bytes) norm_rope_bwd_bytes;
  decltype(&fa_norm_rope_axes_paged) norm_rope_paged;
  decltype(&fa_pages_extend) pages_extend;
} api{};

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong, kU8 = at::kByte;
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
  // An int; the library checks its range.
  int integer(int i) {
    const long x = PyLong_AsLong(argv[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    } else if (x != static_cast<int>(x)) {
      ok = false;
    }
    return static_cast<int>(x);
  }
  // Two weights [d], both bf16 or both fp32 (then *fp32 = 1), either of them None.
  void weights(int i, int64_t d, void** w0, void** w1, int* fp32) {
    *fp32 = 0;
    for (int k = i; k < i + 2; ++k)
      if (ok && argv[k] != Py_None) {
        const at::Tensor* t = tensor(k);
        if (t) *fp32 = t->scalar_type() == kF32;
      }
    *w0 = ptr_or_none(i, *fp32 ? kF32 : kBf16, {d});
    *w1 = ptr_or_none(i + 1, *fp32 ? kF32 : kBf16, {d});
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

// q, k, v, o, lse, scale, window, sinks, stream | None, cycles
PyObject* window_fwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
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
  const int window = a.integer(6), sinks = a.integer(7);
  void* stream = a.stream(8);
  const fa_window_opts opts{fp32, a.cycles(9)};
  if (!a.ok) return status(-1);
  return enqueue([&] {
    return api.window_fwd(pq, pk, pv, po, static_cast<float*>(lse), q[0], q[1], k[1], q[2], k[2], q[3], scale, window, sinks,
                          stream, &opts);
  });
  END_HANDLE_TH_ERRORS
}

// q, k, v, o, dout, lse, dq, dk, dv, scale, window, sinks, workspace | None, stream | None, cycles
PyObject* window_bwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) return status(-1);
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
  const int window = a.integer(10), sinks = a.integer(11);
  size_t bytes = 0;
  void* ws = workspace(a, 12, &bytes);
  void* stream = a.stream(13);
  const fa_bwd_opts opts{a.cycles(14)};
  if (!a.ok || f0 != f1 || f0 != f2) return status(-1);
  const int B = q[0], Hq = q[1], Hkv = k[1], N = q[2], Nk = k[2], d = q[3];
  return enqueue([&] {
    at::Tensor own;
    if (argv[12] == Py_None && (bytes = api.window_bwd_bytes(B, Hq, Hkv, N, Nk, d, window, sinks)) > 0) {
      own = scratch(bytes, a.dev);
      ws = own.data_ptr();
    }
    return api.window_bwd(pq, pk, pv, po, pdo, static_cast<const float*>(lse), dq, dk, dv, B, Hq, Hkv, N, Nk, d, scale, window,
                          sinks, f0, ws, bytes, stream, &opts);
  });
  END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, block_table, seq_lens, o, lse, scale, max_seq_len, window, sinks, workspace | None, stream | None,
// cycles
PyObject* window_decode_paged(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) return status(-1);
  Args a{argv};
  int64_t q[3], pool[4];
  int fp32 = 0;
  void* pq = a.sized(0, 3, q);
  void* kp = a.sized(1, 4, pool);
  if (!a.ok || pool[3] != q[2]) return status(-1);
  const at::Tensor* table = a.tensor(3);
  if (!table || table->dim() != 2) return status(-1);
  const int64_t max_pages = table->size(1);
  if (max_pages > INT32_MAX) return status(-1);
  void* vp = a.ptr(2, kBf16, {pool[0], pool[1], pool[2], pool[3]});
  void* bt = a.ptr(3, kI32, {q[0], max_pages});
  void* lens = a.ptr(4, kI32, {q[0]});
  void* po = a.out(5, {q[0], q[1], q[2]}, &fp32);
  void* lse = a.ptr(6, kF32, {q[0], q[1]});
  const float scale = a.number(7);
  const int max_seq_len = a.integer(8), window = a.integer(9), sinks = a.integer(10);
  size_t bytes = 0;
  void* ws = workspace(a, 11, &bytes);
  void* stream = a.stream(12);
  const fa_decode_opts opts{fp32, a.cycles(13)};
  if (!a.ok) return status(-1);
  const int B = q[0], Hq = q[1], Hkv = pool[1], d = q[2], page_size = pool[2];
  return enqueue([&] {
    at::Tensor own;
    if (argv[11] == Py_None &&
        (bytes = api.window_decode_bytes(B, Hq, Hkv, d, page_size, max_pages, max_seq_len, window, sinks)) > 0) {
      own = scratch(bytes, a.dev);
      ws = own.data_ptr();
    }
    return api.window_decode(pq, kp, vp, static_cast<const int*>(bt), static_cast<const int*>(lens), po,
                             static_cast<float*>(lse), B, Hq, Hkv, d, page_size, max_pages, pool[0], max_seq_len, scale,
                             window, sinks, ws, bytes, stream, &opts);
  });
  END_HANDLE_TH_ERRORS
}

// q and k (or None) of a norm's call: pointers and sizes, k[1] = 0 without k.
bool norm_inputs(Args& a, int64_t* q, int64_t* k, void** pq, void** pk) {
  k[1] = 0;
  *pk = nullptr;
  *pq = a.sized(0, 4, q);
  if (a.ok && a.argv[1] != Py_None) {
    *pk = a.sized(1, 4, k);
    if (a.ok && (k[0] != q[0] || k[2] != q[2] || k[3] != q[3])) a.ok = false;
  }
  return a.ok;
}

// q, k | None, q_weight | None, k_weight | None, pos, plan, q_out, k_out | None, eps, stream | None
PyObject* norm_rope_axes(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) return status(-1);
  Args a{argv};
  int64_t q[4], k[4];
  void *pq, *pk, *wq, *wk, *ko = nullptr;
  int fp32 = 0;
  if (!norm_inputs(a, q, k, &pq, &pk) || (!pk && argv[7] != Py_None)) return status(-1);
  const Plan plan(argv[5], q[3]);
  if (!plan.p) return status(-1);
  a.weights(2, q[3], &wq, &wk, &fp32);
  void* pos = a.ptr(4, kI32, {plan.p->n_axes, q[0], q[2]});
  void* qo = a.ptr(6, kBf16, {q[0], q[1], q[2], q[3]});
  if (pk) ko = a.ptr(7, kBf16, {k[0], k[1], k[2], k[3]});
  const float eps = a.number(8);
  void* stream = a.stream(9);
  if (!a.ok) return status(-1);
  return enqueue([&] {
    return api.norm_rope(pq, pk, wq, wk, fp32, static_cast<const int*>(pos), qo, ko, q[0], q[1], k[1], q[2], eps, plan.p,
                         stream);
  });
  END_HANDLE_TH_ERRORS
}

// q, k | None, q_weight | None, k_weight | None, pos, plan, dq_out, dk_out | None, dq, dk | None, dq_weight | None,
// dk_weight | None, eps, workspace | None, stream | None
PyObject* norm_rope_axes_bwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) return status(-1);
  Args a{argv};
  int64_t q[4], k[4];
  void *pq, *pk, *wq, *wk, *gk = nullptr, *dk = nullptr;
  int fp32 = 0;
  if (!norm_inputs(a, q, k, &pq, &pk)) return status(-1);
  if (!pk && (argv[7] != Py_None || argv[9] != Py_None || argv[11] != Py_None)) return status(-1);
  const Plan plan(argv[5], q[3]);
  if (!plan.p) return status(-1);
  a.weights(2, q[3], &wq, &wk, &fp32);
  void* pos = a.ptr(4, kI32, {plan.p->n_axes, q[0], q[2]});
  void* gq = a.ptr(6, kBf16, {q[0], q[1], q[2], q[3]});
  void* dq = a.ptr(8, kBf16, {q[0], q[1], q[2], q[3]});
  if (pk) {
    gk = a.ptr(7, kBf16, {k[0], k[1], k[2], k[3]});
    dk = a.ptr(9, kBf16, {k[0], k[1], k[2], k[3]});
  }
  void* dwq = a.ptr_or_none(10, kF32, {q[3]});
  void* dwk = a.ptr_or_none(11, kF32, {q[3]});
  const float eps = a.number(12);
  size_t bytes = 0;
  void* ws = workspace(a, 13, &bytes);
  void* stream = a.stream(14);
  if (!a.ok) return status(-1);
  return enqueue([&] {
    at::Tensor own;
    if (argv[13] == Py_None && (dwq || dwk) && (bytes = api.norm_rope_bwd_bytes(q[0], q[1], k[1], q[2], q[3])) > 0) {
      own = scratch(bytes, a.dev);
      ws = own.data_ptr();
    }
    return api.norm_rope_bwd(pq, pk, wq, wk, fp32, static_cast<const int*>(pos), gq, gk, dq, dk, static_cast<float*>(dwq),
                             static_cast<float*>(dwk), q[0], q[1], k[1], q[2], eps, plan.p, ws, bytes, stream);
  });
  END_HANDLE_TH_ERRORS
}

// q, k, v, q_weight | None, k_weight | None, pos, plan, q_out, k_pages, v_pages, slots, new_lens | None, eps, stream | None
PyObject* norm_rope_axes_paged(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) return status(-1);
  Args a{argv};
  int64_t q[4], k[4], pool[4];
  void *pq, *pk, *wq, *wk;
  int fp32 = 0;
  if (!norm_inputs(a, q, k, &pq, &pk) || !pk) return status(-1);
  void* kp = a.sized(8, 4, pool);
  if (!a.ok || pool[1] != k[1] || pool[3] != q[3]) return status(-1);
  const Plan plan(argv[6], q[3]);
  if (!plan.p) return status(-1);
  a.weights(3, q[3], &wq, &wk, &fp32);
  void* pv = a.ptr(2, kBf16, {k[0], k[1], k[2], k[3]});
  void* pos = a.ptr(5, kI32, {plan.p->n_axes, q[0], q[2]});
  void* qo = a.ptr(7, kBf16, {q[0], q[1], q[2], q[3]});
  void* vp = a.ptr(9, kBf16, {pool[0], pool[1], pool[2], pool[3]});
  void* slots = a.ptr(10, kI64, {q[0], q[2]});
  void* news = a.ptr_or_none(11, kI32, {q[0]});
  const float eps = a.number(12);
  void* stream = a.stream(13);
  if (!a.ok) return status(-1);
  return enqueue([&] {
    return api.norm_rope_paged(pq, pk, pv, wq, wk, fp32, static_cast<const int*>(pos), qo, kp, vp,
                               static_cast<const long long*>(slots), static_cast<const int*>(news), q[0], q[1], k[1], q[2],
                               pool[2], pool[0], eps, plan.p, stream);
  });
  END_HANDLE_TH_ERRORS
}

// block_table, seq_lens, new_lens, free_pages, n_free, granted, slots | None, page_size, stream | None
PyObject* pages_extend(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return status(-1);
  Args a{argv};
  const at::Tensor* table = a.tensor(0);
  if (!table || table->dim() != 2) return status(-1);
  const at::Tensor* stack = a.tensor(3);
  if (!stack || stack->dim() != 1) return status(-1);
  const int64_t B = table->size(0), max_pages = table->size(1), num_pages = stack->size(0);
  int64_t N = 0;
  if (argv[6] != Py_None) {
    const at::Tensor* slots = a.tensor(6);
    if (!slots || slots->dim() != 2) return status(-1);
    N = slots->size(1);
  }
  if (B > INT32_MAX || max_pages > INT32_MAX || num_pages > INT32_MAX || N > INT32_MAX) return status(-1);
  void* bt = a.ptr(0, kI32, {B, max_pages});
  void* lens = a.ptr(1, kI32, {B});
  void* news = a.ptr(2, kI32, {B});
  void* free = a.ptr(3, kI32, {num_pages});
  void* n_free = a.ptr(4, kI32, {1});
  void* granted = a.ptr(5, kI32, {B});
  void* slots = a.ptr_or_none(6, kI64, {B, N});
  const int page_size = a.integer(7);
  void* stream = a.stream(8);
  if (!a.ok) return status(-1);
  return enqueue([&] {
    return api.pages_extend(static_cast<int*>(bt), static_cast<int*>(lens), static_cast<const int*>(news),
                            static_cast<int*>(free), static_cast<int*>(n_free), static_cast<int*>(granted),
                            static_cast<long long*>(slots), B, N, page_size, max_pages, num_pages, stream);
  });
  END_HANDLE_TH_ERRORS
}

// Reads addresses into the entry points, in their order.
template <typename... Fn>
PyObject* set_all(PyObject* const* argv, Py_ssize_t n, Fn&... fn) {
  if (n != static_cast<Py_ssize_t>(sizeof...(fn))) {
    PyErr_Format(PyExc_TypeError, "%d addresses expected", static_cast<int>(sizeof...(fn)));
    return nullptr;
  }
  void* p[sizeof...(fn)];
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(argv[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  int i = 0;
  ((fn = reinterpret_cast<Fn>(p[i++])), ...);
  Py_RETURN_NONE;
}

// Addresses of fa_cross_fwd, fa_cross_workspace_bytes, fa_cross_bwd, fa_cross_bwd_workspace_bytes, fa_rope_axes,
// fa_rope_axes_paged in the loaded library.
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return set_all(argv, n, api.cross_fwd, api.cross_bytes, api.cross_bwd, api.cross_bwd_bytes, api.rope, api.rope_paged);
}

// Those of fa_window_fwd, fa_window_bwd, fa_window_bwd_workspace_bytes, fa_window_decode_paged,
// fa_window_decode_paged_workspace_bytes, fa_norm_rope_axes, fa_norm_rope_axes_bwd,
// fa_norm_rope_axes_bwd_workspace_bytes, fa_norm_rope_axes_paged, fa_pages_extend.
PyObject* bind_layer(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return set_all(argv, n, api.window_fwd, api.window_bwd, api.window_bwd_bytes, api.window_decode, api.window_decode_bytes,
                 api.norm_rope, api.norm_rope_bwd, api.norm_rope_bwd_bytes, api.norm_rope_paged, api.pages_extend);
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"bind_layer", fast(bind_layer), METH_FASTCALL, nullptr},
                         {"cross_fwd", fast(cross_fwd), METH_FASTCALL, nullptr},
                         {"cross_bwd", fast(cross_bwd), METH_FASTCALL, nullptr},
                         {"rope_axes", fast(rope_axes), METH_FASTCALL, nullptr},
                         {"rope_axes_paged", fast(rope_axes_paged), METH_FASTCALL, nullptr},
                         {"window_fwd", fast(window_fwd), METH_FASTCALL, nullptr},
                         {"window_bwd", fast(window_bwd), METH_FASTCALL, nullptr},
                         {"window_decode_paged", fast(window_decode_paged), METH_FASTCALL, nullptr},
                         {"norm_rope_axes", fast(norm_rope_axes), METH_FASTCALL, nullptr},
                         {"norm_rope_axes_bwd", fast(norm_rope_axes_bwd), METH_FASTCALL, nullptr},
                         {"norm_rope_axes_paged", fast(norm_rope_axes_paged), METH_FASTCALL, nullptr},
                         {"pages_extend", fast(pages_extend), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", FATTN_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
