// The operators on feature rows for Python: checks of torch tensors, outputs from torch's
// allocator on its current stream, and the calls of the C ABI. A call of one row takes
// the GPU about five microseconds; through ctypes the host took nine for it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "overlap.hpp"
#include "topo.h"

namespace {

using at::Tensor;

PyObject* g_topo_error = nullptr;  // binding.TopoError

struct Refused {
  PyObject* type;
  std::string what;
};

[[noreturn]] void bad_type(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void bad_value(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

struct Failed {
  int status;
};
void check(int status) {
  if (status != TC_OK) throw Failed{status};
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int dtype_id(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return TC_F32;
    case at::kHalf: return TC_F16;
    case at::kBFloat16: return TC_BF16;
    default: bad_type(std::string("dtype must be float32, float16 or bfloat16, not ") + c10::toString(t));
  }
}

// The device of `t`, which has to be the current one.
int device_of(const Tensor& t, int current) {
  if (!t.is_cuda()) bad_type("the tensors must be cuda tensors");
  if (t.get_device() != current) bad_value("the tensors are not on the current device");
  return current;
}

void check_kind(const Tensor& t, const char* name, at::ScalarType dtype, int device) {
  if (!t.is_cuda() || t.scalar_type() != dtype)
    bad_type(std::string(name) + " must be a cuda " + c10::toString(dtype) + " tensor");
  if (t.get_device() != device) bad_value("the tensors are on different devices");
}

struct Matrix {
  void* p = nullptr;
  int64_t stride = 0, rows = 0, cols = 0;
};
// A device matrix with unit channel stride (any strides where it has no rows), any row stride; rows or cols of -1 may be any.
Matrix matrix(const Tensor& t, const char* name, at::ScalarType dtype, int device, int64_t rows = -1,
              int64_t cols = -1) {
  check_kind(t, name, dtype, device);
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols))
    bad_value(std::string(name) + " has the wrong shape: expected [" + (rows < 0 ? "rows" : std::to_string(rows)) +
              ", " + (cols < 0 ? "channels" : std::to_string(cols)) + "]");
  if (t.stride(1) != 1 && t.size(1) > 1 && t.size(0) > 0) bad_value(std::string(name) + " must have unit channel stride");
  return {t.data_ptr(), t.stride(0), t.size(0), t.size(1)};
}

void* vector(const Tensor& t, const char* name, at::ScalarType dtype, int device, int64_t n) {
  check_kind(t, name, dtype, device);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    bad_value(std::string(name) + " must be a contiguous vector of " + std::to_string(n));
  return t.data_ptr();
}

// An output on the current device, which `like` is on. torch's dispatcher takes a third of a microsecond for each, so its own
// allocator is asked directly, but where a mode answers for the dispatcher (one of fake tensors, or one that watches). Which
// allocator that is, the first output that the dispatcher makes by itself tells.
Tensor empty(const Tensor& like, at::IntArrayRef shape, at::ScalarType dtype) {
  auto ask = [&](at::IntArrayRef shape) {
    return at::empty(shape, like.options().dtype(dtype).requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
  };
  const auto answers = c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set;
  if (!answers.empty()) return ask(shape);
  static c10::Allocator* const allocator = ask({1}).storage().allocator();
  return at::detail::empty_generic(shape, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), dtype,
                                   at::MemoryFormat::Contiguous);
}

int32_t channels_of(int64_t n, const char* name) {  // the C ABI refuses what is too many for it
  if (n > INT32_MAX) bad_value(std::string(name) + " has too many channels");
  return (int32_t)n;
}

struct Args {
  PyObject* const* a;
  int current;
  void* stream;
};

struct NormIn {
  const Tensor* x;
  Matrix xm, rm;
  void* w = nullptr;
  int dt, wdt;
  bool residual;
};
NormIn norm_in(PyObject* const* a, int current) {
  NormIn n{};
  n.x = &tensor(a[0], "x");
  const auto type = n.x->scalar_type();
  n.wdt = n.dt = dtype_id(type);
  const int device = device_of(*n.x, current);
  n.xm = matrix(*n.x, "x", type, device);
  n.residual = a[2] != Py_None;
  if (n.residual) n.rm = matrix(tensor(a[2], "residual"), "residual", type, device, n.xm.rows, n.xm.cols);
  if (a[1] != Py_None) {
    const Tensor& w = tensor(a[1], "weight");
    n.wdt = dtype_id(w.scalar_type());
    n.w = vector(w, "weight", w.scalar_type(), device, n.xm.cols);
  }
  channels_of(n.xm.cols, "x");
  return n;
}

template <size_t N>
PyObject* tuple(const std::optional<Tensor> (&t)[N]) {
  PyObject* r = PyTuple_New(N);
  if (!r) return nullptr;
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = t[i] ? THPVariable_Wrap(*t[i]) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// Runs a call of the C ABI without the interpreter's lock.
template <typename F>
void unlocked(F&& f) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(state);
  check(status);
}

// (x, weight, residual, eps) -> (out, h, rstd), or in 8 bits (q, scale, h)
template <bool kI8>
PyObject* rms_norm(const Args& g) {
  const NormIn n = norm_in(g.a, g.current);
  const double eps = PyFloat_AsDouble(g.a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const auto type = n.x->scalar_type();
  Tensor out = empty(*n.x, {n.xm.rows, n.xm.cols}, kI8 ? at::kChar : type);
  Tensor per_row = empty(*n.x, {n.xm.rows}, at::kFloat);
  Tensor h = n.residual ? empty(*n.x, {n.xm.rows, n.xm.cols}, type) : *n.x;
  void *ph = n.residual ? h.data_ptr() : nullptr, *po = out.data_ptr();
  float* ps = static_cast<float*>(per_row.data_ptr());
  const int32_t channels = (int32_t)n.xm.cols;
  unlocked([&]() {
    return kI8 ? tc_rms_norm_i8(n.xm.p, n.xm.stride, n.rm.p, n.rm.stride, n.w, n.wdt, n.xm.rows, channels, n.dt,
                                (float)eps, ph, static_cast<int8_t*>(po), ps, g.stream)
               : tc_rms_norm(n.xm.p, n.xm.stride, n.rm.p, n.rm.stride, n.w, n.wdt, n.xm.rows, channels, n.dt,
                             (float)eps, ph, po, ps, g.stream);
  });
  if (!n.residual) {  // h is the caller's own tensor
    PyObject *a = THPVariable_Wrap(out), *b = THPVariable_Wrap(per_row);
    PyObject* r = !a || !b ? nullptr : kI8 ? PyTuple_Pack(3, a, b, g.a[0]) : PyTuple_Pack(3, a, g.a[0], b);
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
  }
  if (kI8) return tuple<3>({out, per_row, h});
  return tuple<3>({out, h, per_row});
}

// (grad_out, h, weight, rstd, grad_h) -> (grad_x, grad_weight)
PyObject* rms_norm_backward(const Args& g) {
  const Tensor& h = tensor(g.a[1], "h");
  const auto type = h.scalar_type();
  const int dt = dtype_id(type), device = device_of(h, g.current);
  const Matrix hm = matrix(h, "h", type, device);
  const Matrix gm = matrix(tensor(g.a[0], "grad_out"), "grad_out", type, device, hm.rows, hm.cols);
  Matrix dm;
  if (g.a[4] != Py_None) dm = matrix(tensor(g.a[4], "grad_h"), "grad_h", type, device, hm.rows, hm.cols);
  const float* rstd = static_cast<float*>(vector(tensor(g.a[3], "rstd"), "rstd", at::kFloat, device, hm.rows));
  const int32_t channels = channels_of(hm.cols, "h");
  int wdt = dt;
  void* w = nullptr;
  std::optional<Tensor> grad_weight;
  Tensor work;
  int64_t bytes = 0;
  if (g.a[2] != Py_None) {
    const Tensor& wt = tensor(g.a[2], "weight");
    wdt = dtype_id(wt.scalar_type());
    w = vector(wt, "weight", wt.scalar_type(), device, hm.cols);
    grad_weight = empty(h, {hm.cols}, at::kFloat);
    bytes = tc_rms_norm_backward_workspace(hm.rows, channels);
    work = empty(h, {std::max<int64_t>(bytes, 1)}, at::kByte);
  }
  Tensor grad_x = empty(h, {hm.rows, hm.cols}, type);
  void *px = grad_x.data_ptr(), *pwork = w ? work.data_ptr() : nullptr;
  float* pw = grad_weight ? static_cast<float*>(grad_weight->data_ptr()) : nullptr;
  unlocked([&]() {
    return tc_rms_norm_backward(gm.p, gm.stride, dm.p, dm.stride, hm.p, hm.stride, w, wdt, rstd, hm.rows, channels, dt,
                                px, pw, pwork, bytes, g.stream);
  });
  return tuple<2>({grad_x, grad_weight});
}

// The caller's own tensor as a result: autograd sees that it was written.
PyObject* written(PyObject* out) {
  const Tensor& t = THPVariable_Unpack(out);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return Py_NewRef(out);
}

// A vector of one number a channel, in 32 bits or the rows' own type; none: nullptr.
struct Params {
  void* p = nullptr;
  int dt;
};
Params params(PyObject* o, const char* name, at::ScalarType rows_type, int device, int64_t n) {
  Params r{nullptr, dtype_id(rows_type)};
  if (o == Py_None) return r;
  const Tensor& t = tensor(o, name);
  r.dt = dtype_id(t.scalar_type());
  r.p = vector(t, name, t.scalar_type(), device, n);
  return r;
}

// (x, weight, bias, residual, eps) -> (out, h, mean, rstd)
PyObject* layer_norm(const Args& g) {
  const Tensor& x = tensor(g.a[0], "x");
  const auto type = x.scalar_type();
  const int dt = dtype_id(type), device = device_of(x, g.current);
  const Matrix xm = matrix(x, "x", type, device);
  const bool residual = g.a[3] != Py_None;
  Matrix rm;
  if (residual) rm = matrix(tensor(g.a[3], "residual"), "residual", type, device, xm.rows, xm.cols);
  const Params w = params(g.a[1], "weight", type, device, xm.cols), b = params(g.a[2], "bias", type, device, xm.cols);
  const int32_t channels = channels_of(xm.cols, "x");
  const double eps = PyFloat_AsDouble(g.a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  Tensor out = empty(x, {xm.rows, xm.cols}, type), mean = empty(x, {xm.rows}, at::kFloat),
         rstd = empty(x, {xm.rows}, at::kFloat);
  Tensor h = residual ? empty(x, {xm.rows, xm.cols}, type) : x;
  void *ph = residual ? h.data_ptr() : nullptr, *po = out.data_ptr();
  float *pm = static_cast<float*>(mean.data_ptr()), *ps = static_cast<float*>(rstd.data_ptr());
  unlocked([&]() {
    return tc_layer_norm(xm.p, xm.stride, rm.p, rm.stride, w.p, w.dt, b.p, b.dt, xm.rows, channels, dt, (float)eps, ph,
                         po, pm, ps, g.stream);
  });
  if (residual) return tuple<4>({out, h, mean, rstd});
  PyObject* r = tuple<4>({out, std::nullopt, mean, rstd});
  if (r) {  // h is the caller's own tensor
    Py_DECREF(PyTuple_GET_ITEM(r, 1));
    PyTuple_SET_ITEM(r, 1, Py_NewRef(g.a[0]));
  }
  return r;
}

// (grad_out, h, weight, mean, rstd, grad_h, with_bias) -> (grad_x, grad_weight, grad_bias)
PyObject* layer_norm_backward(const Args& g) {
  const Tensor& h = tensor(g.a[1], "h");
  const auto type = h.scalar_type();
  const int dt = dtype_id(type), device = device_of(h, g.current);
  const Matrix hm = matrix(h, "h", type, device);
  const Matrix gm = matrix(tensor(g.a[0], "grad_out"), "grad_out", type, device, hm.rows, hm.cols);
  Matrix dm;
  if (g.a[5] != Py_None) dm = matrix(tensor(g.a[5], "grad_h"), "grad_h", type, device, hm.rows, hm.cols);
  const float* mean = static_cast<float*>(vector(tensor(g.a[3], "mean"), "mean", at::kFloat, device, hm.rows));
  const float* rstd = static_cast<float*>(vector(tensor(g.a[4], "rstd"), "rstd", at::kFloat, device, hm.rows));
  const Params w = params(g.a[2], "weight", type, device, hm.cols);
  const int32_t channels = channels_of(hm.cols, "h");
  const int with_bias = PyObject_IsTrue(g.a[6]);
  if (with_bias < 0) return nullptr;
  std::optional<Tensor> grad_weight, grad_bias;
  Tensor work;
  int64_t bytes = 0;
  if (g.a[2] != Py_None) grad_weight = empty(h, {hm.cols}, at::kFloat);
  if (with_bias) grad_bias = empty(h, {hm.cols}, at::kFloat);
  if (grad_weight || grad_bias) {
    bytes = tc_layer_norm_backward_workspace(hm.rows, channels);
    work = empty(h, {std::max<int64_t>(bytes, 1)}, at::kByte);
  }
  Tensor grad_x = empty(h, {hm.rows, hm.cols}, type);
  void *px = grad_x.data_ptr(), *pwork = bytes ? work.data_ptr() : nullptr;
  float* pw = grad_weight ? static_cast<float*>(grad_weight->data_ptr()) : nullptr;
  float* pb = grad_bias ? static_cast<float*>(grad_bias->data_ptr()) : nullptr;
  unlocked([&]() {
    return tc_layer_norm_backward(gm.p, gm.stride, dm.p, dm.stride, hm.p, hm.stride, w.p, w.dt, mean, rstd, hm.rows,
                                  channels, dt, px, pw, pb, pwork, bytes, g.stream);
  });
  return tuple<3>({grad_x, grad_weight, grad_bias});
}

struct Heads {
  void* p;
  int64_t row, head, rows;
  int32_t heads, dim;
};
// [rows, heads, dim], or [rows, dim] (one head), with unit stride in a head.
Heads heads_of(const Tensor& t, const char* name, at::ScalarType type, int device) {
  check_kind(t, name, type, device);
  if (t.dim() != 2 && t.dim() != 3) bad_value(std::string(name) + " must be [rows, heads, dim] or [rows, dim]");
  const int64_t last = t.dim() - 1, heads = t.dim() == 3 ? t.size(1) : 1;
  if (t.stride(last) != 1 && t.size(last) > 1 && t.numel() > 0)
    bad_value(std::string(name) + " must have unit stride in a head");
  if (heads > INT32_MAX || t.size(last) > INT32_MAX) bad_value(std::string(name) + " has too many channels");
  return {t.data_ptr(), t.stride(0), t.dim() == 3 ? t.stride(1) : 0, t.size(0), (int32_t)heads, (int32_t)t.size(last)};
}

// (x, positions, freqs, sections, interleaved, inverse, out) -> out
PyObject* rotary(const Args& g) {
  const Tensor &x = tensor(g.a[0], "x"), &positions = tensor(g.a[1], "positions"), &freqs = tensor(g.a[2], "freqs");
  const auto type = x.scalar_type();
  const int dt = dtype_id(type), device = device_of(x, g.current);
  const Heads h = heads_of(x, "x", type, device);
  const Matrix pm = matrix(positions, "positions", at::kInt, device, h.rows);
  int32_t sections[4];
  int64_t axes = pm.cols, pairs = 0;
  if (axes < 1 || axes > 4) bad_value("positions must have 1 to 4 axes");
  if (g.a[3] == Py_None) {
    if (axes != 1) bad_value("sections are needed where positions have more than one axis");
    pairs = freqs.numel();
    if (pairs > INT32_MAX) bad_value("too many frequencies");
    sections[0] = (int32_t)pairs;
  } else {
    PyObject* list = PySequence_Fast(g.a[3], "sections must be a sequence of integers");
    if (!list) return nullptr;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
    bool ok = n == axes;
    for (Py_ssize_t i = 0; ok && i < n; ++i) {
      int over = 0;
      const long v = PyLong_AsLongAndOverflow(PySequence_Fast_GET_ITEM(list, i), &over);
      if (v == -1 && PyErr_Occurred()) {
        Py_DECREF(list);
        return nullptr;
      }
      ok = !over && v >= 0 && v <= INT32_MAX;
      sections[i] = (int32_t)v;
      pairs += v;
    }
    Py_DECREF(list);
    if (!ok) bad_value("sections must be a number of pairs for each axis of positions");
  }
  const float* pf = static_cast<float*>(vector(freqs, "freqs", at::kFloat, device, pairs));
  const int interleaved = PyObject_IsTrue(g.a[4]), inverse = PyObject_IsTrue(g.a[5]);
  if (interleaved < 0 || inverse < 0) return nullptr;
  std::optional<Tensor> made;
  Heads o;
  if (g.a[6] == Py_None) {
    made = empty(x, x.sizes(), type);
    o = {made->data_ptr(), (int64_t)h.heads * h.dim, h.dim, h.rows, h.heads, h.dim};
  } else {
    const Tensor& out = tensor(g.a[6], "out");
    if (c10::GradMode::is_enabled() && out.requires_grad())
      bad_value("out requires a gradient, which this call has none for");
    if (out.sizes() != x.sizes()) bad_value("out has another shape than x");
    o = heads_of(out, "out", type, device);
    // x itself, or apart from it
    const bool same = o.p == h.p && (h.rows < 2 || o.row == h.row) && (h.heads < 2 || o.head == h.head);
    if (x.numel() > 0 && !same &&
        tc::overlap({h.p, h.row, h.head}, {o.p, o.row, o.head}, h.rows, h.heads, h.dim, x.element_size()) != tc::Overlap::none)
      bad_value("out overlaps x without being x");
  }
  if (h.heads > 0)
    unlocked([&]() {
      return tc_rotary(h.p, h.row, h.head, h.rows, h.heads, h.dim, dt, static_cast<int32_t*>(pm.p), pm.stride,
                       (int32_t)axes, sections, pf, interleaved, inverse, o.p, o.row, o.head, g.stream);
    });
  return made ? THPVariable_Wrap(*made) : written(g.a[6]);
}

// (x) -> (q, scale)
PyObject* quantise_mx4(const Args& g) {
  const Tensor& x = tensor(g.a[0], "x");
  const auto type = x.scalar_type();
  const int dt = dtype_id(type);
  const Matrix xm = matrix(x, "x", type, device_of(x, g.current));
  const int32_t channels = channels_of(xm.cols, "x");
  Tensor q = empty(x, {xm.rows, (xm.cols + 1) / 2}, at::kByte), scale = empty(x, {xm.rows, (xm.cols + 31) / 32}, at::kByte);
  uint8_t *pq = static_cast<uint8_t*>(q.data_ptr()), *ps = static_cast<uint8_t*>(scale.data_ptr());
  unlocked([&]() { return tc_quantise_mx4(xm.p, xm.stride, xm.rows, channels, dt, pq, ps, g.stream); });
  return tuple<2>({q, scale});
}

struct Mx4 {
  Matrix q, scale;
};
Mx4 mx4(PyObject* q, PyObject* scale, const char* name, int device, int64_t channels) {
  const std::string s = std::string(name) + "_scale";
  return {matrix(tensor(q, name), name, at::kByte, device, -1, (channels + 1) / 2),
          matrix(tensor(scale, s.c_str()), s.c_str(), at::kByte, device, tensor(q, name).size(0), (channels + 31) / 32)};
}
// The channels of rows packed two a byte: as given, or all that the bytes hold. False with a Python error.
bool channels_of_mx4(PyObject* given, const Tensor& q, const char* name, int64_t& channels) {
  if (q.dim() != 2) bad_value(std::string(name) + " must be a [rows, bytes] tensor");
  channels = 2 * q.size(1);
  if (given != Py_None) {
    const int64_t bytes = q.size(1);
    channels = PyLong_AsLongLong(given);
    if (channels == -1 && PyErr_Occurred()) return false;
    if (channels < 0 || channels > 2 * bytes || channels < 2 * bytes - 1)
      bad_value(std::string(name) + " holds " + std::to_string(2 * bytes) + " channels, or one less");
  }
  channels_of(channels, name);
  return true;
}

struct ProductIn {
  const Tensor* x;
  Matrix xm;
  float *xs, *ws, *bias = nullptr;
  int device;
};
ProductIn product_in(PyObject* x, PyObject* x_scale, PyObject* w_scale, PyObject* bias, int64_t c_out, int current) {
  ProductIn p{};
  p.x = &tensor(x, "x");
  p.device = device_of(*p.x, current);
  p.xm = matrix(*p.x, "x", at::kChar, p.device);
  p.xs = static_cast<float*>(vector(tensor(x_scale, "x_scale"), "x_scale", at::kFloat, p.device, p.xm.rows));
  p.ws = static_cast<float*>(vector(tensor(w_scale, "w_scale"), "w_scale", at::kFloat, p.device, c_out));
  if (bias != Py_None) p.bias = static_cast<float*>(vector(tensor(bias, "bias"), "bias", at::kFloat, p.device, c_out));
  channels_of(p.xm.cols, "x");
  channels_of(c_out, "w");
  return p;
}

struct ProductOut {
  std::optional<Tensor> made;
  Matrix m;
  int dt;
};
ProductOut product_out(const Tensor& like, int device, PyObject* out, PyObject* out_dtype, int64_t rows, int64_t cols) {
  ProductOut o;
  auto type = at::kBFloat16;
  if (out_dtype != Py_None) {
    if (!THPDtype_Check(out_dtype)) bad_type("out_dtype must be a torch dtype");
    type = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
  }
  if (out == Py_None) {
    o.dt = dtype_id(type);
    o.made = empty(like, {rows, cols}, type);
    o.m = {o.made->data_ptr(), cols, rows, cols};
    return o;
  }
  const Tensor& t = tensor(out, "out");
  if (c10::GradMode::is_enabled() && t.requires_grad()) bad_value("out requires a gradient, which this call has none for");
  if (out_dtype != Py_None && type != t.scalar_type()) bad_value("out is of another type than out_dtype");
  o.dt = dtype_id(t.scalar_type());
  o.m = matrix(t, "out", t.scalar_type(), device, rows, cols);
  if (o.m.stride < cols && rows > 1) bad_value("the rows of out overlap");
  o.m.stride = std::max(o.m.stride, cols);
  return o;
}
PyObject* result(const ProductOut& o, PyObject* out) {
  return o.made ? THPVariable_Wrap(*o.made) : written(out);
}

// (x, x_scale, w, w_scale, bias, out_dtype, out) -> out
PyObject* matmul_i8(const Args& g) {
  const Tensor& w = tensor(g.a[2], "w");
  if (w.dim() != 2) bad_value("w must be a [c_out, c_in] tensor");
  const ProductIn p = product_in(g.a[0], g.a[1], g.a[3], g.a[4], w.size(0), g.current);
  const Matrix wm = matrix(w, "w", at::kChar, p.device, -1, p.xm.cols);
  const ProductOut o = product_out(*p.x, p.device, g.a[6], g.a[5], p.xm.rows, wm.rows);
  unlocked([&]() {
    return tc_matmul_i8(static_cast<int8_t*>(p.xm.p), p.xm.stride, p.xs, static_cast<int8_t*>(wm.p), wm.stride, p.ws,
                        p.bias, p.xm.rows, (int32_t)wm.rows, (int32_t)p.xm.cols, o.dt, o.m.p, o.m.stride, g.stream);
  });
  return result(o, g.a[6]);
}

// (x, x_scale, kmap, w, w_scale, bias, out_dtype, out) -> out
PyObject* sparse_conv_i8(const Args& g) {
  const Tensor &kmap = tensor(g.a[2], "kmap"), &w = tensor(g.a[3], "w");
  if (w.dim() != 3) bad_value("w must be a contiguous [taps, c_out, c_in] tensor");
  const ProductIn p = product_in(g.a[0], g.a[1], g.a[4], g.a[5], w.size(1), g.current);
  check_kind(kmap, "kmap", at::kInt, p.device);
  if (kmap.dim() != 2 || !kmap.is_contiguous()) bad_value("kmap must be a contiguous [n_dst, taps] tensor");
  check_kind(w, "w", at::kChar, p.device);
  const int64_t n_dst = kmap.size(0), taps = kmap.size(1);
  if (w.size(0) != taps || w.size(2) != p.xm.cols || !w.is_contiguous())
    bad_value("w must be a contiguous [" + std::to_string(taps) + ", c_out, " + std::to_string(p.xm.cols) + "] tensor");
  if (taps > INT32_MAX) bad_value("kmap has too many taps");
  const ProductOut o = product_out(*p.x, p.device, g.a[7], g.a[6], n_dst, w.size(1));
  const int32_t* pm = static_cast<int32_t*>(kmap.data_ptr());
  const int8_t* pw = static_cast<int8_t*>(w.data_ptr());
  unlocked([&]() {
    return tc_sparse_conv_i8(static_cast<int8_t*>(p.xm.p), p.xm.stride, p.xs, p.xm.rows, pm, n_dst, (int32_t)taps, pw,
                             p.ws, p.bias, (int32_t)w.size(1), (int32_t)p.xm.cols, o.dt, o.m.p, o.m.stride, g.stream);
  });
  return result(o, g.a[7]);
}

// (q, scale, channels, out_dtype) -> out
PyObject* dequantise_mx4(const Args& g) {
  const Tensor& q = tensor(g.a[0], "q");
  int64_t channels;
  if (!channels_of_mx4(g.a[2], q, "q", channels)) return nullptr;
  const int device = device_of(q, g.current);
  const Mx4 m = mx4(g.a[0], g.a[1], "q", device, channels);
  const ProductOut o = product_out(q, device, Py_None, g.a[3], m.q.rows, channels);
  unlocked([&]() {
    return tc_dequantise_mx4(static_cast<uint8_t*>(m.q.p), m.q.stride, static_cast<uint8_t*>(m.scale.p), m.scale.stride,
                             m.q.rows, (int32_t)channels, o.dt, o.m.p, g.stream);
  });
  return THPVariable_Wrap(*o.made);
}

// (x, x_scale, w, w_scale, channels, bias, out_dtype, out) -> out
PyObject* matmul_mx4(const Args& g) {
  const Tensor &x = tensor(g.a[0], "x"), &wt = tensor(g.a[2], "w");
  int64_t channels;
  if (!channels_of_mx4(g.a[4], x, "x", channels)) return nullptr;
  const int device = device_of(x, g.current);
  const Mx4 xm = mx4(g.a[0], g.a[1], "x", device, channels);
  if (wt.dim() != 2) bad_value("w must be a [c_out, bytes] tensor");
  const Mx4 wm = mx4(g.a[2], g.a[3], "w", device, channels);
  const int64_t c_out = wt.size(0);
  channels_of(c_out, "w");
  const float* bias =
      g.a[5] == Py_None ? nullptr : static_cast<float*>(vector(tensor(g.a[5], "bias"), "bias", at::kFloat, device, c_out));
  const ProductOut o = product_out(x, device, g.a[7], g.a[6], xm.q.rows, c_out);
  auto bytes = [](const Matrix& m) { return static_cast<uint8_t*>(m.p); };
  unlocked([&]() {
    return tc_matmul_mx4(bytes(xm.q), xm.q.stride, bytes(xm.scale), xm.scale.stride, bytes(wm.q), wm.q.stride,
                         bytes(wm.scale), wm.scale.stride, bias, xm.q.rows, (int32_t)c_out, (int32_t)channels, o.dt,
                         o.m.p, o.m.stride, g.stream);
  });
  return result(o, g.a[7]);
}

// The last two arguments of every call: the current device and its current stream's handle.
template <PyObject* (*F)(const Args&), int kArgs>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs + 2) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[kArgs]);
  void* stream = PyLong_AsVoidPtr(args[kArgs + 1]);
  if (PyErr_Occurred()) return nullptr;
  try {
    return F(Args{args, (int)device, stream});
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const Failed& e) {
    PyObject* a = Py_BuildValue("(is)", e.status, tc_last_error());
    if (a) PyErr_SetObject(g_topo_error, a);
    Py_XDECREF(a);
  } catch (...) {  // torch's own errors as its operators raise them (no memory for an output: OutOfMemoryError)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// Whether autograd records a call on these (what is no tensor is passed over): it is on and one
// requires a gradient, or one has a forward-mode tangent.
PyObject* records(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const bool on = c10::GradMode::is_enabled();
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (!THPVariable_Check(args[i])) continue;
    const Tensor& t = THPVariable_Unpack(args[i]);
    if ((on && t.requires_grad()) || t._fw_grad(0).defined()) Py_RETURN_TRUE;
  }
  Py_RETURN_FALSE;
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_topo_error, type);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(const Args&), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rms_norm<false>, 4>("rms_norm"),
                           method<rms_norm<true>, 4>("rms_norm_i8"),
                           method<rms_norm_backward, 5>("rms_norm_backward"),
                           method<matmul_i8, 7>("matmul_i8"),
                           method<sparse_conv_i8, 8>("sparse_conv_i8"),
                           method<layer_norm, 5>("layer_norm"),
                           method<layer_norm_backward, 7>("layer_norm_backward"),
                           method<rotary, 7>("rotary"),
                           method<quantise_mx4, 1>("quantise_mx4"),
                           method<dequantise_mx4, 4>("dequantise_mx4"),
                           method<matmul_mx4, 8>("matmul_mx4"),
                           {"records", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&records)),
                            METH_FASTCALL, nullptr},
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_features", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__features() { return PyModule_Create(&g_module); }
