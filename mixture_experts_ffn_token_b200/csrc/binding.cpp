// binding.cpp -- the short way from Python to the operators beside the forward
// pass: abi.py's checks of every tensor (type, size, dense layout, the current
// device) and the call, in one step.  Through ctypes the checks and the
// conversion of the arguments took a call of the dispatch 2.6 us and of the
// 8-bit product 5, as long as the launches themselves.
//
// Each function takes its abi.py namesake's arguments in order, every one of
// them given, and returns the moe_status_t; or -1 where an argument is not as it
// should be, with nothing enqueued: abi.py then checks again in Python, where the
// error's text is.  No exception leaves through the C API.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;
constexpr auto kI8 = at::kChar;
constexpr auto kU8 = at::kByte;

// The entry points, by address, from the library that abi.py has loaded.
struct Entries {
  decltype(&moe_dispatch) dispatch;
  decltype(&moe_dispatch_backward) dispatch_backward;
  decltype(&moe_combine) combine;
  decltype(&moe_combine_backward) combine_backward;
  decltype(&moe_route_backward) route_backward;
  decltype(&moe_dispatch_int8) dispatch_int8;
  decltype(&moe_quantize_rows) quantize_rows;
  decltype(&moe_grouped_linear_int8) grouped_linear_int8;
} g_entry = {};

// One call's arguments; `ok` says whether all were as they should be.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t given, Py_ssize_t wanted) : args_(args) {
    ok = given == wanted && g_entry.dispatch != nullptr;
    if (!ok) return;
    if (PyObject_GetBuffer(args[0], &view_, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      ok = false;
      return;
    }
    held_ = true;
    ok = view_.len == sizeof(moe_config_t);
    if (ok) cfg = *static_cast<const moe_config_t*>(view_.buf);
    R = static_cast<int64_t>(cfg.num_tokens) * cfg.top_k;
  }
  ~Call() {
    if (held_) PyBuffer_Release(&view_);
  }
  Call(const Call&) = delete;
  Call& operator=(const Call&) = delete;

  // Argument i as a dense tensor of `numel` elements on the current device.
  template <typename T = void>
  T* tensor(int i, at::ScalarType type, int64_t numel, bool required = true) {
    if (!ok) return nullptr;
    if (args_[i] == Py_None) {
      ok = !required;
      return nullptr;
    }
    if (!THPVariable_CheckExact(args_[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(args_[i]);
    if (!t.is_cuda() || t.scalar_type() != type || t.numel() != numel || !t.is_contiguous()) {
      ok = false;
      return nullptr;
    }
    if (device_ < 0) device_ = c10::cuda::current_device();
    if (t.get_device() != device_) {
      ok = false;
      return nullptr;
    }
    return static_cast<T*>(t.data_ptr());
  }

  // The type of argument i's rows: bf16 or fp32.
  moe_dtype_t rows_dtype(int i, at::ScalarType* type) {
    *type = kBf16;
    if (!ok || !THPVariable_CheckExact(args_[i])) {
      ok = false;
      return MOE_DTYPE_BF16;
    }
    *type = THPVariable_Unpack(args_[i]).scalar_type();
    ok = *type == kBf16 || *type == kF32;
    return *type == kF32 ? MOE_DTYPE_F32 : MOE_DTYPE_BF16;
  }

  // Argument i as a byte tensor of any size.
  void* bytes(int i, bool required, size_t* n) {
    *n = 0;
    if (!ok) return nullptr;
    if (args_[i] == Py_None || !THPVariable_CheckExact(args_[i])) {
      ok = args_[i] == Py_None && !required;
      return nullptr;
    }
    *n = static_cast<size_t>(THPVariable_Unpack(args_[i]).numel());
    return tensor(i, kU8, static_cast<int64_t>(*n));
  }

  // Argument i as a stream: None is the current one.
  moe_stream_t stream(int i) {
    if (!ok) return nullptr;
    if (args_[i] == Py_None) {
      if (device_ < 0) device_ = c10::cuda::current_device();
      return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream());
    }
    PyObject* handle = PyObject_GetAttrString(args_[i], "cuda_stream");
    void* s = handle != nullptr ? PyLong_AsVoidPtr(handle) : nullptr;
    Py_XDECREF(handle);
    if (PyErr_Occurred() != nullptr) {
      PyErr_Clear();
      ok = false;
    }
    return reinterpret_cast<moe_stream_t>(s);
  }

  moe_config_t cfg = {};
  int64_t R = 0;
  bool ok = false;

 private:
  PyObject* const* args_;
  Py_buffer view_ = {};
  bool held_ = false;
  int device_ = -1;
};

// Runs `body` (which returns a moe_status_t, or -1) and hands its result to Python.
template <typename Body>
PyObject* guarded(Body body) {
  int st = -1;
  try {
    st = body();
  } catch (...) {
    st = -1;  // the careful way says what it was
  }
  if (PyErr_Occurred() != nullptr) PyErr_Clear();
  return PyLong_FromLong(st);
}

// The call itself, without the interpreter's lock.
template <typename F, typename... A>
int enqueue(F entry, A... args) {
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = static_cast<int>(entry(args...));
  Py_END_ALLOW_THREADS;
  return st;
}

int64_t pitch(int64_t n) { return MOE_INT8_PITCH(n); }

// (cfg, x, inverse, rows, expert_weights, stream)
PyObject* py_dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 6);
    const int64_t TH = static_cast<int64_t>(c.cfg.num_tokens) * c.cfg.hidden_dim, RH = c.R * c.cfg.hidden_dim;
    at::ScalarType t;
    const moe_dtype_t dt = c.rows_dtype(1, &t);
    const void* x = c.tensor(1, t, TH);
    const auto* inverse = c.tensor<int32_t>(2, kI32, c.R);
    void* rows = c.tensor(3, t, RH);
    const auto* w = c.tensor<float>(4, kF32, c.R, false);
    const moe_stream_t s = c.stream(5);
    return c.ok ? enqueue(g_entry.dispatch, &c.cfg, dt, x, inverse, w, rows, s) : -1;
  });
}

// (cfg, d_rows, inverse, d_x, x, expert_weights, d_expert_weights, stream)
PyObject* py_dispatch_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 8);
    const int64_t TH = static_cast<int64_t>(c.cfg.num_tokens) * c.cfg.hidden_dim, RH = c.R * c.cfg.hidden_dim;
    at::ScalarType t;
    const moe_dtype_t dt = c.rows_dtype(1, &t);
    const void* d_rows = c.tensor(1, t, RH);
    const auto* inverse = c.tensor<int32_t>(2, kI32, c.R);
    void* d_x = c.tensor(3, t, TH);
    auto* d_w = c.tensor<float>(6, kF32, c.R, false);
    const void* x = c.tensor(4, t, TH, d_w != nullptr);
    const auto* w = c.tensor<float>(5, kF32, c.R, false);
    const moe_stream_t s = c.stream(7);
    return c.ok ? enqueue(g_entry.dispatch_backward, &c.cfg, dt, d_rows, x, inverse, w, d_x, d_w, s) : -1;
  });
}

// (cfg, rows, inverse, out, expert_weights, stream)
PyObject* py_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 6);
    const int64_t TH = static_cast<int64_t>(c.cfg.num_tokens) * c.cfg.hidden_dim, RH = c.R * c.cfg.hidden_dim;
    at::ScalarType t;
    const moe_dtype_t dt = c.rows_dtype(1, &t);
    const void* rows = c.tensor(1, t, RH);
    const auto* inverse = c.tensor<int32_t>(2, kI32, c.R);
    void* out = c.tensor(3, t, TH);
    const auto* w = c.tensor<float>(4, kF32, c.R, false);
    const moe_stream_t s = c.stream(5);
    return c.ok ? enqueue(g_entry.combine, &c.cfg, dt, rows, inverse, w, out, s) : -1;
  });
}

// (cfg, d_out, inverse, d_rows, rows, expert_weights, d_expert_weights, stream)
PyObject* py_combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 8);
    const int64_t TH = static_cast<int64_t>(c.cfg.num_tokens) * c.cfg.hidden_dim, RH = c.R * c.cfg.hidden_dim;
    at::ScalarType t;
    const moe_dtype_t dt = c.rows_dtype(1, &t);
    const void* d_out = c.tensor(1, t, TH);
    const auto* inverse = c.tensor<int32_t>(2, kI32, c.R);
    void* d_rows = c.tensor(3, t, RH);
    auto* d_w = c.tensor<float>(6, kF32, c.R, false);
    const void* rows = c.tensor(4, t, RH, d_w != nullptr);
    const auto* w = c.tensor<float>(5, kF32, c.R, false);
    const moe_stream_t s = c.stream(7);
    return c.ok ? enqueue(g_entry.combine_backward, &c.cfg, dt, d_out, rows, inverse, w, d_rows, d_w, s) : -1;
  });
}

// (cfg, logits, expert_indices, d_expert_weights, d_logits, d_sink_weights, global_scale, d_global_scale, workspace, stream)
PyObject* py_route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 10);
    const int64_t T = c.cfg.num_tokens, all = T * c.cfg.logits_row_stride;
    const at::ScalarType t = c.cfg.logits_dtype == MOE_DTYPE_BF16 ? kBf16 : kF32;
    const void* logits = c.tensor(1, t, all);
    const auto* idx = c.tensor<int32_t>(2, kI32, c.R);
    const auto* d_w = c.tensor<float>(3, kF32, c.R);
    void* d_logits = c.tensor(4, t, all);
    const auto* d_sink = c.tensor<float>(5, kF32, T * c.cfg.num_sink, false);
    const auto* scale = c.tensor<float>(6, kF32, 1, false);
    auto* d_scale = c.tensor<float>(7, kF32, 1, false);
    size_t bytes = 0;
    void* ws = c.bytes(8, false, &bytes);
    const moe_stream_t s = c.stream(9);
    return c.ok ? enqueue(g_entry.route_backward, &c.cfg, logits, scale, idx, d_w, d_sink, d_logits, d_scale, ws, bytes, s)
                : -1;
  });
}

// (cfg, x, inverse, rows_q, row_scales, stream)
PyObject* py_dispatch_int8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 6);
    const void* x = c.tensor(1, kBf16, static_cast<int64_t>(c.cfg.num_tokens) * c.cfg.hidden_dim);
    const auto* inverse = c.tensor<int32_t>(2, kI32, c.R);
    auto* q = c.tensor<int8_t>(3, kI8, c.R * pitch(c.cfg.hidden_dim));
    auto* scales = c.tensor<float>(4, kF32, c.R);
    const moe_stream_t s = c.stream(5);
    return c.ok ? enqueue(g_entry.dispatch_int8, &c.cfg, x, inverse, q, scales, s) : -1;
  });
}

// (cfg, h, expert_offsets, rows_q, row_scales, stream)
PyObject* py_quantize_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 6);
    const void* h = c.tensor(1, kBf16, c.R * c.cfg.moe_dim);
    const auto* off = c.tensor<int32_t>(2, kI32, static_cast<int64_t>(c.cfg.num_experts) + 1, false);
    auto* q = c.tensor<int8_t>(3, kI8, c.R * pitch(c.cfg.moe_dim));
    auto* scales = c.tensor<float>(4, kF32, c.R);
    const moe_stream_t s = c.stream(5);
    return c.ok ? enqueue(g_entry.quantize_rows, &c.cfg, h, off, q, scales, s) : -1;
  });
}

// (cfg, contraction's code, rows_q, row_scales, w_q, w_scales, expert_offsets, out, workspace, bias, stream)
PyObject* py_grouped_linear_int8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Call c(args, n, 11);
    if (!c.ok || !PyLong_CheckExact(args[1])) return -1;
    const bool down = PyLong_AsLong(args[1]) == MOE_DOWN;
    const int64_t H = c.cfg.hidden_dim, D = c.cfg.moe_dim, E = c.cfg.num_experts;
    const int64_t K = down ? D : H, N = down ? H : 2 * D;
    const auto* q = c.tensor<int8_t>(2, kI8, c.R * pitch(K));
    const auto* scales = c.tensor<float>(3, kF32, c.R);
    const auto* w_q = c.tensor<int8_t>(4, kI8, E * N * pitch(K));
    const auto* w_scales = c.tensor<float>(5, kF32, E * N);
    const auto* off = c.tensor<int32_t>(6, kI32, E + 1);
    void* out = c.tensor(7, kBf16, c.R * (down ? H : D));
    size_t bytes = 0;
    void* ws = c.bytes(8, true, &bytes);
    const void* bias = c.tensor(9, kBf16, E * N, false);
    const moe_stream_t s = c.stream(10);
    return c.ok ? enqueue(g_entry.grouped_linear_int8, &c.cfg, down ? MOE_DOWN : MOE_GATE_UP, q, scales, w_q, w_scales, bias,
                          off, out, ws, bytes, s)
                : -1;
  });
}

// (the entry points' addresses, in the order of Entries)
PyObject* py_use(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "use() takes the addresses of eight entry points");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred() != nullptr) return nullptr;
  }
  g_entry.dispatch = reinterpret_cast<decltype(&moe_dispatch)>(p[0]);
  g_entry.dispatch_backward = reinterpret_cast<decltype(&moe_dispatch_backward)>(p[1]);
  g_entry.combine = reinterpret_cast<decltype(&moe_combine)>(p[2]);
  g_entry.combine_backward = reinterpret_cast<decltype(&moe_combine_backward)>(p[3]);
  g_entry.route_backward = reinterpret_cast<decltype(&moe_route_backward)>(p[4]);
  g_entry.dispatch_int8 = reinterpret_cast<decltype(&moe_dispatch_int8)>(p[5]);
  g_entry.quantize_rows = reinterpret_cast<decltype(&moe_quantize_rows)>(p[6]);
  g_entry.grouped_linear_int8 = reinterpret_cast<decltype(&moe_grouped_linear_int8)>(p[7]);
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    METHOD(use),
    METHOD(dispatch),
    METHOD(dispatch_backward),
    METHOD(combine),
    METHOD(combine_backward),
    METHOD(route_backward),
    METHOD(dispatch_int8),
    METHOD(quantize_rows),
    METHOD(grouped_linear_int8),
    {nullptr, nullptr, 0, nullptr},
};
#undef METHOD

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `target`: the torch and Python whose objects this file reads; load_binding()
// refuses to use it under others.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "target", MOE_BINDING_TARGET) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
