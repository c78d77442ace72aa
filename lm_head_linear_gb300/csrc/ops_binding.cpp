// Python side of the operators around the head: checks of the tensors, allocation
// of outputs and workspaces, and the calls of the C ABI.
//
// Why not ctypes, as for the forward and backward: these calls take 2 to 20
// microseconds on the GPU, and attribute lookups, torch.empty() and ctypes
// conversions in Python took 17 to 24 (a norm of one token: 17.2 us through ctypes,
// 6.2 us here, 1.8 us of it the kernel's).  The library itself stays free of torch; this
// module is linked against it and adds no computation.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <stdexcept>
#include <string>

#include "flce.h"

namespace {

using at::ScalarType;
using at::Tensor;

// Raised as ValueError.
struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// A Python exception is set already.
struct Raised {};

[[noreturn]] void bad(const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  throw BadArgument(text);
}

PyObject* g_check = nullptr;  // raises FlceError for a status

void check(flce_status st) {
  if (st == FLCE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", static_cast<int>(st));
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, "the library returned an error status");
  throw Raised{};
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Raised&) {
  } catch (const std::exception&) {
    torch::translate_exception_to_python(std::current_exception());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// ------------------------------------------------------------------ arguments
const Tensor* optional_tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad("%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = optional_tensor(o, name);
  if (!t) bad("%s must be a tensor", name);
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

std::string text_of(const Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] on " + t.device().str();
}

int32_t dtype_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::BFloat16) return FLCE_DTYPE_BF16;
  if (t.scalar_type() == ScalarType::Float) return FLCE_DTYPE_F32;
  bad("%s must be a bfloat16 or float32 tensor, got %s", name, text_of(t).c_str());
}

void matrix(const Tensor& t, const char* name) {
  if (!t.is_cuda() || t.dim() != 2) bad("%s must be a CUDA matrix, got %s", name, text_of(t).c_str());
}

// Row stride of a [rows, cols] matrix on `dev` with contiguous rows.
int64_t rows_of(const Tensor& t, const char* name, int64_t rows, int64_t cols, at::Device dev) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.device() != dev || (cols > 1 && t.stride(1) != 1))
    bad("%s must be a [%lld, %lld] matrix on %s with contiguous rows, got %s", name, (long long)rows, (long long)cols,
        dev.str().c_str(), text_of(t).c_str());
  return rows > 1 ? t.stride(0) : cols;
}

void vector(const Tensor& t, const char* name, int64_t n, ScalarType type, at::Device dev) {
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || t.device() != dev || !t.is_contiguous())
    bad("%s must be a contiguous %s vector of %lld elements on %s, got %s", name, c10::toString(type), (long long)n,
        dev.str().c_str(), text_of(t).c_str());
}

// out[key], checked, or a new tensor.
Tensor output(PyObject* out, const char* key, at::IntArrayRef shape, ScalarType type, const Tensor& like) {
  if (out != Py_None) {
    if (!PyDict_Check(out)) bad("out must be a dict");
    PyObject* o = PyDict_GetItemString(out, key);
    if (o && o != Py_None) {
      const Tensor& t = tensor(o, key);
      if (t.scalar_type() != type || t.sizes() != shape || t.device() != like.device() || !t.is_contiguous())
        bad("out['%s'] must be a contiguous %s tensor of the result's shape on %s, got %s", key, c10::toString(type),
            like.device().str().c_str(), text_of(t).c_str());
      return t;
    }
  }
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// As output(), for a matrix whose rows may lie further apart.
Tensor output_rows(PyObject* out, const char* key, int64_t rows, int64_t cols, ScalarType type, const Tensor& like,
                   int64_t* ld) {
  if (out != Py_None) {
    if (!PyDict_Check(out)) bad("out must be a dict");
    PyObject* o = PyDict_GetItemString(out, key);
    if (o && o != Py_None) {
      const Tensor& t = tensor(o, key);
      if (t.scalar_type() != type) bad("out['%s'] must be %s, got %s", key, c10::toString(type), text_of(t).c_str());
      *ld = rows_of(t, key, rows, cols, like.device());
      return t;
    }
  }
  *ld = cols;
  return at::empty({rows, cols}, at::TensorOptions().dtype(type).device(like.device()));
}

Tensor workspace_of(PyObject* o, size_t bytes, const Tensor& like) {
  if (o == Py_None)
    return at::empty({static_cast<int64_t>(bytes < 256 ? 256 : bytes)},
                     at::TensorOptions().dtype(ScalarType::Byte).device(like.device()));
  const Tensor& t = tensor(o, "workspace");
  if (t.scalar_type() != ScalarType::Byte || t.device() != like.device() || !t.is_contiguous())
    bad("the workspace must be a contiguous uint8 tensor on %s", like.device().str().c_str());
  return t;
}

// The library works on the current device: every entry point makes that the tensors'
// (an OnDevice on its stack) before it allocates or calls, and takes no stream of another.
using OnDevice = c10::cuda::CUDAGuard;

void* stream_of(PyObject* o, const Tensor& like) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
  if (PyObject* d = PyObject_GetAttrString(o, "device")) {
    const bool known = THPDevice_Check(d);
    const at::Device dev = known ? reinterpret_cast<THPDevice*>(d)->device : like.device();
    Py_DECREF(d);
    if (dev != like.device()) bad("the stream is on %s, the tensors are on %s", dev.str().c_str(), like.device().str().c_str());
  } else {
    PyErr_Clear();  // a handle alone
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Raised{};
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!s && PyErr_Occurred()) throw Raised{};
  return s;
}

template <typename E = void>
E* ptr(const Tensor& t) {
  return static_cast<E*>(t.data_ptr());
}
template <typename E = void>
E* ptr(const Tensor* t) {
  return t ? static_cast<E*>(t->data_ptr()) : nullptr;
}
template <typename E = void>
E* defined_ptr(const Tensor& t) {
  return t.defined() ? static_cast<E*>(t.data_ptr()) : nullptr;
}

PyObject* wrapped(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Raised{};
  return o;
}
template <typename... T>
PyObject* tuple_of(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrapped(t)), ...);
  return r;
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) bad("%lld arguments given, %lld wanted", (long long)n, (long long)want);
}

// ------------------------------------------------------------------ norm
int32_t weight_of(const Tensor& w, int64_t Hd, at::Device dev) {
  const int32_t type = dtype_of(w, "weight");
  if (w.dim() != 1 || w.size(0) != Hd || w.device() != dev || !w.is_contiguous())
    bad("weight must be a contiguous vector of %lld elements on %s, got %s", (long long)Hd, dev.str().c_str(),
        text_of(w).c_str());
  return type;
}

// x, weight, residual, eps, normed, fp8, save_rstd, stream, out -> y, h, rstd, q, q_scale
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 9);
    const Tensor& x = tensor(a[0], "x");
    const Tensor& w = tensor(a[1], "weight");
    const Tensor* r = optional_tensor(a[2], "residual");
    matrix(x, "x");
    const at::Device dev = x.device();
    const OnDevice on(dev);
    const int64_t T = x.size(0), Hd = x.size(1);
    const int32_t x_type = dtype_of(x, "x");
    const int64_t ldx = rows_of(x, "x", T, Hd, dev);
    const int32_t w_type = weight_of(w, Hd, dev);
    PyObject* out = a[8];
    Tensor h = x, y, rstd, q, qs;
    int64_t ldr = 0, ldh = 0;
    int32_t r_type = 0;
    if (r) {
      r_type = dtype_of(*r, "residual");
      ldr = rows_of(*r, "residual", T, Hd, dev);
      h = output_rows(out, "h", T, Hd, r->scalar_type(), x, &ldh);
    }
    if (truth(a[4])) y = output(out, "y", {T, Hd}, ScalarType::BFloat16, x);
    if (truth(a[6])) rstd = output(out, "rstd", {T}, ScalarType::Float, x);
    if (truth(a[5])) {
      q = output(out, "q", {T, Hd}, ScalarType::Float8_e4m3fn, x);
      qs = output(out, "q_scale", {T, (Hd + 127) / 128}, ScalarType::Float8_e8m0fnu, x);
    }
    check(flce_add_rms_norm(ptr(x), x_type, ldx, ptr(r), r_type, ldr, ptr(w), w_type, T, Hd,
                            static_cast<float>(number(a[3])), r ? ptr(h) : nullptr, ldh, defined_ptr(y),
                            defined_ptr<float>(rstd), defined_ptr(q), defined_ptr<uint8_t>(qs), stream_of(a[7], x)));
    return tuple_of(y, h, rstd, q, qs);
  });
}

// dy, h, weight, rstd, dh, workspace, stream, out -> dx, dweight, workspace
PyObject* add_rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 8);
    const Tensor& dy = tensor(a[0], "dy");
    const Tensor& h = tensor(a[1], "h");
    const Tensor& w = tensor(a[2], "weight");
    const Tensor& rstd = tensor(a[3], "rstd");
    const Tensor* dh = optional_tensor(a[4], "dh");
    matrix(h, "h");
    const at::Device dev = h.device();
    const OnDevice on(dev);
    const int64_t T = h.size(0), Hd = h.size(1);
    const int32_t h_type = dtype_of(h, "h"), y_type = dtype_of(dy, "dy");
    const int64_t ldh = rows_of(h, "h", T, Hd, dev), lddy = rows_of(dy, "dy", T, Hd, dev);
    const int32_t w_type = weight_of(w, Hd, dev);
    vector(rstd, "rstd", T, ScalarType::Float, dev);
    int64_t lddh = 0;
    if (dh) {
      if (dh->scalar_type() != h.scalar_type()) bad("dh must have h's dtype, got %s", text_of(*dh).c_str());
      lddh = rows_of(*dh, "dh", T, Hd, dev);
    }
    const Tensor dx = output(a[7], "dx", {T, Hd}, h.scalar_type(), h);
    const Tensor dw = output(a[7], "dweight", {Hd}, ScalarType::Float, h);
    const Tensor ws = workspace_of(a[5], flce_add_rms_norm_backward_workspace_size(T, Hd), h);
    check(flce_add_rms_norm_backward(ptr(dy), y_type, lddy, ptr(h), h_type, ldh, ptr(w), w_type, ptr<float>(rstd), ptr(dh),
                                     lddh, T, Hd, ptr(dx), ptr<float>(dw), ptr(ws), ws.numel(), stream_of(a[6], h)));
    return tuple_of(dx, dw, ws);
  });
}

// x, weight, residual, eps, stream, out -> y, h, rstd, hq, hq_scale
PyObject* add_rms_norm_checkpoint(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 6);
    const Tensor& x = tensor(a[0], "x");
    const Tensor& w = tensor(a[1], "weight");
    const Tensor* r = optional_tensor(a[2], "residual");
    matrix(x, "x");
    const at::Device dev = x.device();
    const OnDevice on(dev);
    const int64_t T = x.size(0), Hd = x.size(1);
    const int32_t x_type = dtype_of(x, "x");
    const int64_t ldx = rows_of(x, "x", T, Hd, dev);
    const int32_t w_type = weight_of(w, Hd, dev);
    PyObject* out = a[5];
    Tensor h = x;
    int64_t ldr = 0, ldh = 0;
    int32_t r_type = 0;
    if (r) {
      r_type = dtype_of(*r, "residual");
      ldr = rows_of(*r, "residual", T, Hd, dev);
      h = output_rows(out, "h", T, Hd, r->scalar_type(), x, &ldh);
    }
    const Tensor y = output(out, "y", {T, Hd}, ScalarType::BFloat16, x);
    const Tensor rstd = output(out, "rstd", {T}, ScalarType::Float, x);
    const Tensor q = output(out, "hq", {T, Hd}, ScalarType::Float8_e4m3fn, x);
    const Tensor qs = output(out, "hq_scale", {T, (Hd + 127) / 128}, ScalarType::Float8_e8m0fnu, x);
    check(flce_add_rms_norm_checkpoint(ptr(x), x_type, ldx, ptr(r), r_type, ldr, ptr(w), w_type, T, Hd,
                                       static_cast<float>(number(a[3])), r ? ptr(h) : nullptr, ldh, ptr(y), ptr<float>(rstd),
                                       ptr(q), ptr<uint8_t>(qs), stream_of(a[4], x)));
    return tuple_of(y, h, rstd, q, qs);
  });
}

void blocks(const Tensor& q, const Tensor& s, const char* name, int64_t per, at::Device dev);

// dy, hq, hq_scale, weight, rstd, dh, fp32, workspace, stream, out -> dx, dweight, workspace
PyObject* add_rms_norm_checkpoint_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 10);
    const Tensor& dy = tensor(a[0], "dy");
    const Tensor& q = tensor(a[1], "hq");
    const Tensor& qs = tensor(a[2], "hq_scale");
    const Tensor& w = tensor(a[3], "weight");
    const Tensor& rstd = tensor(a[4], "rstd");
    const Tensor* dh = optional_tensor(a[5], "dh");
    matrix(q, "hq");
    const at::Device dev = q.device();
    const OnDevice on(dev);
    const int64_t T = q.size(0), Hd = q.size(1);
    blocks(q, qs, "hq", 1, dev);
    const bool f32 = truth(a[6]);
    const ScalarType type = f32 ? ScalarType::Float : ScalarType::BFloat16;
    const int32_t y_type = dtype_of(dy, "dy");
    const int64_t lddy = rows_of(dy, "dy", T, Hd, dev);
    const int32_t w_type = weight_of(w, Hd, dev);
    vector(rstd, "rstd", T, ScalarType::Float, dev);
    int64_t lddh = 0;
    if (dh) {
      if (dh->scalar_type() != type) bad("dh must have the dtype of dx, got %s", text_of(*dh).c_str());
      lddh = rows_of(*dh, "dh", T, Hd, dev);
    }
    const Tensor dx = output(a[9], "dx", {T, Hd}, type, q);
    const Tensor dw = output(a[9], "dweight", {Hd}, ScalarType::Float, q);
    const Tensor ws = workspace_of(a[7], flce_add_rms_norm_backward_workspace_size(T, Hd), q);
    check(flce_add_rms_norm_checkpoint_backward(ptr(dy), y_type, lddy, ptr(q), ptr<uint8_t>(qs),
                                                f32 ? FLCE_DTYPE_F32 : FLCE_DTYPE_BF16, ptr(w), w_type, ptr<float>(rstd),
                                                ptr(dh), lddh, T, Hd, ptr(dx), ptr<float>(dw), ptr(ws), ws.numel(),
                                                stream_of(a[8], q)));
    return tuple_of(dx, dw, ws);
  });
}

// ------------------------------------------------------------------ 8 bits
// a, block_rows, stream, out -> q, q_scale
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 4);
    const Tensor& m = tensor(a[0], "a");
    matrix(m, "a");
    const OnDevice on(m.device());
    const int64_t rows = m.size(0), K = m.size(1);
    // 0, which the library refuses, for what it does not know: the number of scales that
    // are allocated and its 32-bit argument have to mean the same
    const int32_t block = integer(a[1]) == 128 ? 128 : integer(a[1]) == 1 ? 1 : 0;
    const int32_t type = dtype_of(m, "a");
    const int64_t ld = rows_of(m, "a", rows, K, m.device());
    const int64_t per = block < 1 ? 1 : block;
    const Tensor q = output(a[3], "q", {rows, K}, ScalarType::Float8_e4m3fn, m);
    const Tensor qs = output(a[3], "q_scale", {(rows + per - 1) / per, (K + 127) / 128}, ScalarType::Float8_e8m0fnu, m);
    check(flce_quantize_fp8(ptr(m), type, ld, rows, K, block, ptr(q), ptr<uint8_t>(qs),
                            stream_of(a[2], m)));
    return tuple_of(q, qs);
  });
}

void blocks(const Tensor& q, const Tensor& s, const char* name, int64_t per, at::Device dev) {
  if (q.scalar_type() != ScalarType::Float8_e4m3fn || q.dim() != 2 || q.device() != dev || !q.is_contiguous())
    bad("%s must be a contiguous float8_e4m3fn matrix on %s, got %s", name, dev.str().c_str(), text_of(q).c_str());
  const int64_t r = (q.size(0) + per - 1) / per, c = (q.size(1) + 127) / 128;
  if ((s.scalar_type() != ScalarType::Float8_e8m0fnu && s.scalar_type() != ScalarType::Byte) || s.dim() != 2 ||
      s.size(0) != r || s.size(1) != c || s.device() != dev || !s.is_contiguous())
    bad("%s's scales must be a contiguous float8_e8m0fnu or uint8 [%lld, %lld] matrix on %s, got %s", name, (long long)r,
        (long long)c, dev.str().c_str(), text_of(s).c_str());
}

// x, x_scale, W, W_scale, fp32, workspace, stream, out -> y, workspace
PyObject* linear_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 8);
    const Tensor& x = tensor(a[0], "x");
    const Tensor& xs = tensor(a[1], "x_scale");
    const Tensor& W = tensor(a[2], "W");
    const Tensor& Ws = tensor(a[3], "W_scale");
    matrix(x, "x");
    matrix(W, "W");
    const OnDevice on(x.device());
    const int64_t T = x.size(0), K = x.size(1), V = W.size(0);
    if (W.size(1) != K) bad("x [T, K] and W [V, K] must have equal K");
    blocks(x, xs, "x", 1, x.device());
    blocks(W, Ws, "W", 128, x.device());
    const bool f32 = truth(a[4]);
    int64_t ldy = 0;
    const Tensor y = output_rows(a[7], "y", T, V, f32 ? ScalarType::Float : ScalarType::BFloat16, x, &ldy);
    const Tensor ws = workspace_of(a[5], flce_linear_fp8_workspace_size(T, K, V), x);
    check(flce_linear_fp8(ptr(x), ptr<uint8_t>(xs), ptr(W), ptr<uint8_t>(Ws), T, K, V, ptr(y),
                          f32 ? FLCE_DTYPE_F32 : FLCE_DTYPE_BF16, ldy, ptr(ws), ws.numel(), stream_of(a[6], x)));
    return tuple_of(y, ws);
  });
}

// ------------------------------------------------------------------ 4 bits
// a, stream, out -> q, q_scale
PyObject* quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 3);
    const Tensor& m = tensor(a[0], "a");
    matrix(m, "a");
    const OnDevice on(m.device());
    const int64_t rows = m.size(0), K = m.size(1), kb = (K + 127) / 128;
    const int32_t type = dtype_of(m, "a");
    const int64_t ld = rows_of(m, "a", rows, K, m.device());
    const Tensor q = output(a[2], "q", {rows, 64 * kb}, ScalarType::Byte, m);
    const Tensor qs = output(a[2], "q_scale", {kb, rows, 4}, ScalarType::Float8_e8m0fnu, m);
    check(flce_quantize_fp4(ptr(m), type, ld, rows, K, ptr(q), ptr<uint8_t>(qs), stream_of(a[1], m)));
    return tuple_of(q, qs);
  });
}

// x, x_scale, W, W_scale, fp32, workspace, stream, out -> y, workspace
PyObject* linear_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 8);
    const Tensor& x = tensor(a[0], "x");
    const Tensor& xs = tensor(a[1], "x_scale");
    const Tensor& W = tensor(a[2], "W");
    const Tensor& Ws = tensor(a[3], "W_scale");
    matrix(x, "x");
    matrix(W, "W");
    const at::Device dev = x.device();
    const OnDevice on(dev);
    const int64_t T = x.size(0), K = x.size(1), V = W.size(0), kb = (K + 127) / 128;
    blocks(x, xs, "x", 1, dev);
    if (W.scalar_type() != ScalarType::Byte || W.size(1) != 64 * kb || W.device() != dev || !W.is_contiguous())
      bad("W must be a contiguous uint8 [V, %lld] matrix on %s, got %s", (long long)(64 * kb), dev.str().c_str(),
          text_of(W).c_str());
    if ((Ws.scalar_type() != ScalarType::Float8_e8m0fnu && Ws.scalar_type() != ScalarType::Byte) || Ws.dim() != 3 ||
        Ws.size(0) != kb || Ws.size(1) != V || Ws.size(2) != 4 || Ws.device() != dev || !Ws.is_contiguous())
      bad("W's scales must be a contiguous float8_e8m0fnu or uint8 [%lld, %lld, 4] tensor on %s, got %s", (long long)kb,
          (long long)V, dev.str().c_str(), text_of(Ws).c_str());
    const bool f32 = truth(a[4]);
    int64_t ldy = 0;
    const Tensor y = output_rows(a[7], "y", T, V, f32 ? ScalarType::Float : ScalarType::BFloat16, x, &ldy);
    const Tensor ws = workspace_of(a[5], flce_linear_fp4_workspace_size(T, K, V), x);
    check(flce_linear_fp4(ptr(x), ptr<uint8_t>(xs), ptr(W), ptr<uint8_t>(Ws), T, K, V, ptr(y),
                          f32 ? FLCE_DTYPE_F32 : FLCE_DTYPE_BF16, ldy, ptr(ws), ws.numel(), stream_of(a[6], x)));
    return tuple_of(y, ws);
  });
}

// ------------------------------------------------------------------ sampling
// A setting of flce_sample: a tensor [T], or a number for all rows.
template <typename E>
const E* setting(PyObject* o, const char* name, int64_t T, ScalarType type, at::Device dev, double* all) {
  *all = 0.0;
  if (!THPVariable_Check(o)) {
    *all = number(o);
    return nullptr;
  }
  const Tensor& t = THPVariable_Unpack(o);
  vector(t, name, T, type, dev);
  return ptr<E>(t);
}

// logits, u, temperature, top_k, top_p, min_p, ignore_index, stream, out -> tokens, logp
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 9);
    const Tensor& l = tensor(a[0], "logits");
    const Tensor& u = tensor(a[1], "u");
    matrix(l, "logits");
    const at::Device dev = l.device();
    const OnDevice on(dev);
    const int64_t T = l.size(0), V = l.size(1);
    const int32_t type = dtype_of(l, "logits");
    const int64_t ld = rows_of(l, "logits", T, V, dev);
    vector(u, "u", T, ScalarType::Float, dev);
    double temperature, top_p, min_p, unused;
    const float* ts = setting<float>(a[2], "temperature", T, ScalarType::Float, dev, &temperature);
    int64_t top_k = 0;
    const int32_t* ks = nullptr;
    if (THPVariable_Check(a[3]))
      ks = setting<int32_t>(a[3], "top_k", T, ScalarType::Int, dev, &unused);
    else
      top_k = integer(a[3]);
    const float* ps = setting<float>(a[4], "top_p", T, ScalarType::Float, dev, &top_p);
    const float* ms = setting<float>(a[5], "min_p", T, ScalarType::Float, dev, &min_p);
    const Tensor tokens = output(a[8], "tokens", {T}, ScalarType::Long, l);
    const Tensor logp = output(a[8], "logp", {T}, ScalarType::Float, l);
    check(flce_sample(ptr(l), type, ld, ptr<float>(u), T, V, ts, temperature, ks, top_k, ps, top_p, ms, min_p, integer(a[6]),
                      ptr<int64_t>(tokens), ptr<float>(logp), stream_of(a[7], l)));
    return tuple_of(tokens, logp);
  });
}

// ------------------------------------------------------------------ losses
const Tensor& logp_of(PyObject* o) {
  const Tensor& t = tensor(o, "logp");
  if (!t.is_cuda() || t.dim() != 1) bad("logp must be a CUDA tensor [T], got %s", text_of(t).c_str());
  return t;
}

// A gradient of a loss with `n` entries, or nullptr.
const float* gradient(PyObject* o, int64_t n, const Tensor& like) {
  const Tensor* t = optional_tensor(o, "dloss");
  if (!t) return nullptr;
  if (t->scalar_type() != ScalarType::Float || t->numel() != n || t->device() != like.device() || !t->is_contiguous())
    bad("dloss must be a contiguous Float tensor of %lld elements on %s, got %s", (long long)n,
        like.device().str().c_str(), text_of(*t).c_str());
  return ptr<float>(t);
}

// logp, old_logp, advantages, targets, ref_logp, cu_seqlens, per_sequence, ignore_index, reduction, clip_low, clip_high,
// dual_clip, kl_coef, kl, dloss, forward, grad, workspace, stream, out -> loss, dlogp, stats, n_valid, workspace
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 20);
    const Tensor& logp = logp_of(a[0]);
    const Tensor& old = tensor(a[1], "old_logp");
    const Tensor& adv = tensor(a[2], "advantages");
    const Tensor& y = tensor(a[3], "targets");
    const Tensor* ref = optional_tensor(a[4], "ref_logp");
    const Tensor* cu = optional_tensor(a[5], "cu_seqlens");
    const at::Device dev = logp.device();
    const OnDevice on(dev);
    const int64_t T = logp.size(0);
    const bool per_seq = truth(a[6]);
    int64_t S = 0;
    if (cu) {
      if (cu->dim() != 1 || cu->size(0) < 1) bad("cu_seqlens must be a tensor [n_seqs + 1], got %s", text_of(*cu).c_str());
      S = cu->size(0) - 1;
      vector(*cu, "cu_seqlens", S + 1, ScalarType::Long, dev);
    }
    vector(logp, "logp", T, ScalarType::Float, dev);
    vector(old, "old_logp", T, ScalarType::Float, dev);
    vector(adv, "advantages", per_seq ? S : T, ScalarType::Float, dev);
    vector(y, "targets", T, ScalarType::Long, dev);
    if (ref) vector(*ref, "ref_logp", T, ScalarType::Float, dev);
    const int32_t red = static_cast<int32_t>(integer(a[8]));
    const int64_t entries = red == FLCE_REDUCTION_NONE ? T : 1;
    const float* dloss = gradient(a[14], entries, logp);
    Tensor loss, dlogp;
    if (truth(a[15])) loss = output(a[19], "loss", {entries}, ScalarType::Float, logp);
    if (truth(a[16])) dlogp = output(a[19], "dlogp", {T}, ScalarType::Float, logp);
    const Tensor stats = output(a[19], "stats", {4}, ScalarType::Float, logp);
    const Tensor n_valid = output(a[19], "n_valid", {1}, ScalarType::Long, logp);
    const Tensor ws = workspace_of(a[17], flce_policy_loss_workspace_size(T, S), logp);
    check(flce_policy_loss(dloss, ptr<float>(logp), ptr<float>(old), ptr<float>(ref), ptr<float>(adv), per_seq,
                           ptr<int64_t>(y), ptr<int64_t>(cu), S, T, integer(a[7]), red, static_cast<float>(number(a[9])),
                           static_cast<float>(number(a[10])), static_cast<float>(number(a[11])),
                           static_cast<float>(number(a[12])), static_cast<int32_t>(integer(a[13])),
                           defined_ptr<float>(loss), defined_ptr<float>(dlogp), ptr<float>(stats), ptr<int64_t>(n_valid),
                           ptr(ws), ws.numel(), stream_of(a[18], logp)));
    return tuple_of(loss, dlogp, stats, n_valid, ws);
  });
}

// logp, targets, cu_seqlens, ref_logp, ignore_index, reduction, kind, beta, label_smoothing, margin, length_normalize,
// dloss, forward, grad, workspace, stream, out -> loss, dlogp, chosen, rejected, workspace
PyObject* preference_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 17);
    const Tensor& logp = logp_of(a[0]);
    const Tensor& y = tensor(a[1], "targets");
    const Tensor& cu = tensor(a[2], "cu_seqlens");
    const Tensor* ref = optional_tensor(a[3], "ref_logp");
    const at::Device dev = logp.device();
    const OnDevice on(dev);
    const int64_t T = logp.size(0);
    if (cu.dim() != 1 || cu.size(0) % 2 == 0) bad("cu_seqlens must be a tensor [2 n_pairs + 1], got %s", text_of(cu).c_str());
    const int64_t P = cu.size(0) / 2;
    vector(cu, "cu_seqlens", 2 * P + 1, ScalarType::Long, dev);
    vector(logp, "logp", T, ScalarType::Float, dev);
    vector(y, "targets", T, ScalarType::Long, dev);
    if (ref) vector(*ref, "ref_logp", T, ScalarType::Float, dev);
    const int32_t red = static_cast<int32_t>(integer(a[5]));
    const int64_t entries = red == FLCE_REDUCTION_NONE ? P : 1;
    const float* dloss = gradient(a[11], entries, logp);
    Tensor loss, dlogp;
    if (truth(a[12])) loss = output(a[16], "loss", {entries}, ScalarType::Float, logp);
    if (truth(a[13])) dlogp = output(a[16], "dlogp", {T}, ScalarType::Float, logp);
    const Tensor chosen = output(a[16], "chosen", {P}, ScalarType::Float, logp);
    const Tensor rejected = output(a[16], "rejected", {P}, ScalarType::Float, logp);
    const Tensor ws = workspace_of(a[14], flce_preference_loss_workspace_size(P), logp);
    check(flce_preference_loss(dloss, ptr<float>(logp), ptr<float>(ref), ptr<int64_t>(y), ptr<int64_t>(cu), P, T,
                               integer(a[4]), red, static_cast<int32_t>(integer(a[6])), static_cast<float>(number(a[7])),
                               static_cast<float>(number(a[8])), static_cast<float>(number(a[9])), truth(a[10]),
                               defined_ptr<float>(loss), defined_ptr<float>(dlogp), ptr<float>(chosen),
                               ptr<float>(rejected), ptr(ws), ws.numel(), stream_of(a[15], logp)));
    return tuple_of(loss, dlogp, chosen, rejected, ws);
  });
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(add_rms_norm),
                         FAST(add_rms_norm_backward),
                         FAST(add_rms_norm_checkpoint),
                         FAST(add_rms_norm_checkpoint_backward),
                         FAST(quantize_fp8),
                         FAST(linear_fp8),
                         FAST(quantize_fp4),
                         FAST(linear_fp4),
                         FAST(sample),
                         FAST(policy_loss),
                         FAST(preference_loss),
                         {"set_check", set_check, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "flce_ops", "Calls of the operators around the LM head.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_flce_ops(void) { return PyModule_Create(&module); }
