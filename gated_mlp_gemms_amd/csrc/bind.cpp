// The Python side of moe.h's, norm.h's and mx4.h's entry points: checks a call's tensors, turns them into device pointers and
// makes the call, as functions of positional arguments that moe.py, norm.py and mx4.py wrap. A call of a few tokens takes the
// GPU 2-4 us; checking 3 to 8 tensors and passing 10 to 17 arguments from Python took 4 to 7 us a call, more than
// the launch itself, here it takes well under one.
//
// Errors leave as Python exceptions, and no C++ exception passes a C frame: ValueError for what a tensor is
// wrong in, MlpError for a status of the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string>

#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"
#include "mx4.h"
#include "norm.h"

namespace {

// What _lib.py hands over once (setup): the library's entry points, and its own objects.
struct Entry {
  decltype(&::moe_route) route;
  decltype(&::moe_route_bwd) route_bwd;
  decltype(&::moe_sort_workspace_bytes) sort_bytes;
  decltype(&::moe_sort) sort;
  decltype(&::moe_gather) gather;
  decltype(&::moe_gather_bwd) gather_bwd;
  decltype(&::moe_combine) combine;
  decltype(&::moe_combine_bwd) combine_bwd;
  decltype(&::linear_workspace_bytes) linear_bytes;
  decltype(&::linear_fwd) fwd;
  decltype(&::linear_bwd) bwd;
  decltype(&::moe_balance_workspace_bytes) balance_bytes;
  decltype(&::moe_balance) balance;
  decltype(&::moe_balance_bwd) balance_bwd;
  decltype(&::norm_fwd) norm_fwd;
  decltype(&::norm_workspace_bytes) norm_bytes;
  decltype(&::norm_bwd) norm_bwd;
  decltype(&::mx4_planes) mx4_planes;
  decltype(&::mx4_scale_rows) mx4_scale_rows;
  decltype(&::mx4_quantize) mx4_quantize;
  decltype(&::mx4_dequantize) mx4_dequantize;
  decltype(&::mx4_linear_workspace_bytes) mx4_bytes;
  decltype(&::mx4_linear_fwd) mx4_fwd;
} lib;
PyObject *py_error, *py_workspace, *py_raw_stream;   // owned for good

using at::ScalarType;
constexpr ScalarType kI32 = ScalarType::Int, kF32 = ScalarType::Float;

struct PyFailed {};   // a Python exception is set

int code_of(ScalarType t) {   // mlp_dtype, or -1
  switch (t) {
    case ScalarType::Float: return MLP_F32;
    case ScalarType::BFloat16: return MLP_BF16;
    case ScalarType::Half: return MLP_F16;
    default: return -1;
  }
}
ScalarType type_of(int code) {   // (the library refuses another code)
  return code == MLP_BF16 ? ScalarType::BFloat16 : code == MLP_F16 ? ScalarType::Half : kF32;
}

using Shape = at::IntArrayRef;

[[noreturn]] void raise(PyObject* kind, const std::string& text) {
  PyErr_SetString(kind, text.c_str());
  throw PyFailed{};
}

std::string type_name(ScalarType t) {   // as torch prints it
  switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Bool: return "torch.bool";
    default: return c10::toString(t);
  }
}
std::string list(Shape v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

// One call's tensors. The first one sets the device; all of them are looked at before a GPU is required.
class Args {
 public:
  void* operator()(PyObject* o, const char* name, ScalarType type, Shape shape) {
    if (!THPVariable_Check(o)) raise(PyExc_ValueError, std::string(name) + " must be a tensor, not " + Py_TYPE(o)->tp_name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || t.sizes() != shape)
      raise(PyExc_ValueError, name + (" must be " + type_name(type)) + " " + list(shape) + ", not " +
                                  type_name(t.scalar_type()) + " " + list(t.sizes()));
    if (t.layout() != at::kStrided || !t.is_contiguous())
      raise(PyExc_ValueError, std::string(name) + " must be contiguous" +
                                  (t.layout() == at::kStrided ? ", not of strides " + list(t.strides()) : ""));
    const bool gpu = t.is_cuda();
    const int dev = gpu ? (int)t.get_device() : -1;
    if (dev_ == kUnset) dev_ = dev;
    if ((!gpu || dev != dev_) && far_ == nullptr) far_ = &t, far_name_ = name;
    return gpu ? t.data_ptr() : nullptr;
  }
  void* opt(PyObject* o, const char* name, ScalarType type, Shape shape) {
    return o == Py_None ? nullptr : (*this)(o, name, type, shape);
  }
  template <typename P> P* as(PyObject* o, const char* name, ScalarType type, Shape shape) {
    return static_cast<P*>((*this)(o, name, type, shape));
  }
  // The tensors' device: called once all of them have been checked.
  int device() const {
    if (far_ != nullptr)
      raise(PyExc_ValueError, std::string(far_name_) + " must be on the GPU of the other tensors, not on " + far_->device().str());
    return dev_;
  }

 private:
  static constexpr int kUnset = -2;
  int dev_ = kUnset;
  const at::Tensor* far_ = nullptr;
  const char* far_name_ = nullptr;
};

// A tensor's sizes, when it has `n` of them (its type is checked with the others).
Shape dims(PyObject* o, const char* name, int64_t n) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != n)
    raise(PyExc_ValueError, std::string(name) + " must be a tensor of " + std::to_string(n) + " dimensions");
  return THPVariable_Unpack(o).sizes();
}
ScalarType float_type(PyObject* o, const char* name) {
  const ScalarType t = THPVariable_Check(o) ? THPVariable_Unpack(o).scalar_type() : ScalarType::Undefined;
  if (code_of(t) < 0) raise(PyExc_ValueError, std::string(name) + " must be a float32, bfloat16 or float16 tensor");
  return t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailed{};
  return v;
}

// The call's stream: the one passed (a torch stream or its handle), or the device's current one.
void* stream_of(PyObject* o, int dev) {
  PyObject* h;
  if (o == Py_None) {
    PyObject* d = PyLong_FromLong(dev);
    h = d == nullptr ? nullptr : PyObject_CallOneArg(py_raw_stream, d);
    Py_XDECREF(d);
  } else if (PyLong_Check(o)) {
    Py_INCREF(o);
    h = o;
  } else {
    h = PyObject_GetAttrString(o, "cuda_stream");
  }
  if (h == nullptr) throw PyFailed{};
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (s == nullptr && PyErr_Occurred()) throw PyFailed{};
  return s;
}

// The caller's workspace, or a new one of need() bytes that lives until the call has been made: torch's
// allocator hands it on in the order of the stream it was allocated on, which is the call's.
class Workspace {
 public:
  template <typename Need> Workspace(PyObject* o, int dev, void* stream, Need need) {
    if (o == Py_None) {
      own_ = PyObject_CallFunction(py_workspace, "KiK", (unsigned long long)need(), dev,
                                   (unsigned long long)reinterpret_cast<uintptr_t>(stream));
      if (own_ == nullptr) throw PyFailed{};
      o = own_;
    }
    if (!THPVariable_Check(o)) raise(PyExc_ValueError, "workspace must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_contiguous() || !t.is_cuda() || t.get_device() != dev)
      raise(PyExc_ValueError, "workspace must be contiguous and on the GPU of the other tensors");
    ptr = t.data_ptr();
    bytes = t.nbytes();
  }
  ~Workspace() { Py_XDECREF(own_); }
  Workspace(const Workspace&) = delete;
  void* ptr;
  size_t bytes;

 private:
  PyObject* own_ = nullptr;
};

// Raises for a status that is not MLP_OK.
void check(mlp_status st, const char* where) {
  if (st == MLP_OK) return;
  PyObject* e = PyObject_CallFunction(py_error, "is", (int)st, where);
  if (e != nullptr) {
    PyErr_SetObject(py_error, e);
    Py_DECREF(e);
  }
  throw PyFailed{};
}

size_t needed(size_t bytes, const char* where) {   // 0: the library refuses the sizes
  if (bytes == 0) check(MLP_ERR_INVALID_ARG, where);
  return bytes;
}

// Makes the library's call on the tensors' device, without the interpreter's lock (the status and the text
// of an error belong to this thread).
template <typename F> void call(int dev, const char* where, F f) {
  mlp_status st;
  {
    const c10::DeviceGuard guard(c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)dev));
    PyThreadState* save = PyEval_SaveThread();
    st = f();
    PyEval_RestoreThread(save);
  }
  check(st, where);
}

// Every function below: its number of positional arguments, and its body.
template <Py_ssize_t N, void (*BODY)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", N, n);
    return nullptr;
  }
  if (py_error == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "setup has not been called");
    return nullptr;
  }
  try {
    BODY(a);
    Py_RETURN_NONE;
  } catch (const PyFailed&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// logits, ids, weights, score, renorm, stream
void route(PyObject* const* a) {
  Args arg;
  const ScalarType dt = float_type(a[0], "logits");
  const Shape te = dims(a[0], "logits", 2);
  const int64_t T = te[0], E = te[1], k = dims(a[1], "ids", 2)[1];
  const void* logits = arg(a[0], "logits", dt, te);
  auto* ids = arg.as<int32_t>(a[1], "ids", kI32, {T, k});
  auto* w = arg.as<float>(a[2], "weights", kF32, {T, k});
  const int score = (int)integer(a[3]), renorm = (int)integer(a[4]), dev = arg.device();
  void* s = stream_of(a[5], dev);
  call(dev, "moe_route", [&] { return lib.route(logits, code_of(dt), T, E, k, score, renorm, ids, w, s); });
}

// logits, ids, dweights, dlogits, score, renorm, stream
void route_bwd(PyObject* const* a) {
  Args arg;
  const ScalarType dt = float_type(a[0], "logits");
  const Shape te = dims(a[0], "logits", 2);
  const int64_t T = te[0], E = te[1], k = dims(a[1], "ids", 2)[1];
  const void* logits = arg(a[0], "logits", dt, te);
  auto* ids = arg.as<int32_t>(a[1], "ids", kI32, {T, k});
  auto* dw = arg.as<float>(a[2], "dweights", kF32, {T, k});
  void* dl = arg(a[3], "dlogits", dt, te);
  const int score = (int)integer(a[4]), renorm = (int)integer(a[5]), dev = arg.device();
  void* s = stream_of(a[6], dev);
  call(dev, "moe_route_bwd", [&] { return lib.route_bwd(logits, ids, dw, code_of(dt), T, E, k, score, renorm, dl, s); });
}

// logits, ids, mask, counts, shares, loss, score, workspace, stream
void balance(PyObject* const* a) {
  Args arg;
  const ScalarType dt = float_type(a[0], "logits");
  const Shape te = dims(a[0], "logits", 2);
  const int64_t T = te[0], E = te[1], k = dims(a[1], "ids", 2)[1];
  const void* logits = arg(a[0], "logits", dt, te);
  auto* ids = arg.as<int32_t>(a[1], "ids", kI32, {T, k});
  auto* mask = static_cast<uint8_t*>(arg.opt(a[2], "mask", ScalarType::Bool, {T}));
  auto* counts = arg.as<int32_t>(a[3], "counts", kI32, {E + 1});
  auto* shares = arg.as<float>(a[4], "shares", kF32, {E});
  auto* loss = arg.as<float>(a[5], "loss", kF32, {1});
  const int score = (int)integer(a[6]), dev = arg.device();
  void* s = stream_of(a[8], dev);
  const Workspace ws(a[7], dev, s, [&] { return needed(lib.balance_bytes(T, E), "moe_balance_workspace_bytes"); });
  call(dev, "moe_balance", [&] {
    return lib.balance(logits, ids, mask, code_of(dt), T, E, k, score, counts, shares, loss, ws.ptr, ws.bytes, s);
  });
}

// logits, ids, mask, counts, dloss, dweights, dlogits, score, renorm, stream
void balance_bwd(PyObject* const* a) {
  Args arg;
  const ScalarType dt = float_type(a[0], "logits");
  const Shape te = dims(a[0], "logits", 2);
  const int64_t T = te[0], E = te[1], k = dims(a[1], "ids", 2)[1];
  const void* logits = arg(a[0], "logits", dt, te);
  auto* ids = arg.as<int32_t>(a[1], "ids", kI32, {T, k});
  auto* mask = static_cast<uint8_t*>(arg.opt(a[2], "mask", ScalarType::Bool, {T}));
  auto* counts = arg.as<int32_t>(a[3], "counts", kI32, {E + 1});
  auto* dloss = static_cast<float*>(arg.opt(a[4], "dloss", kF32, {1}));
  auto* dw = static_cast<float*>(arg.opt(a[5], "dweights", kF32, {T, k}));
  void* dl = arg(a[6], "dlogits", dt, te);
  const int score = (int)integer(a[7]), renorm = (int)integer(a[8]), dev = arg.device();
  void* s = stream_of(a[9], dev);
  call(dev, "moe_balance_bwd", [&] {
    return lib.balance_bwd(logits, ids, mask, counts, dloss, dw, code_of(dt), T, E, k, score, renorm, dl, s);
  });
}

// ids (any shape, taken in order), experts, offsets, row_of, slot_of, workspace, stream
void sort(PyObject* const* a) {
  Args arg;
  const int64_t E = integer(a[1]), n = THPVariable_Check(a[0]) ? THPVariable_Unpack(a[0]).numel() : 0;
  auto* ids = arg.as<int32_t>(a[0], "ids", kI32, THPVariable_Check(a[0]) ? THPVariable_Unpack(a[0]).sizes() : Shape());
  auto* offsets = arg.as<int32_t>(a[2], "offsets", kI32, {E + 1});
  auto* row_of = arg.as<int32_t>(a[3], "row_of", kI32, {n});
  auto* slot_of = arg.as<int32_t>(a[4], "slot_of", kI32, {n});
  const int dev = arg.device();
  void* s = stream_of(a[6], dev);
  const Workspace ws(a[5], dev, s, [&] { return needed(lib.sort_bytes(n, E), "moe_sort_workspace_bytes"); });
  call(dev, "moe_sort", [&] { return lib.sort(ids, n, E, offsets, row_of, slot_of, ws.ptr, ws.bytes, s); });
}

// The sizes of a [T, d] tensor and the [T k, d] rows that belong to it.
struct Rows {
  ScalarType dt;
  int code;
  int64_t T, E, k, d;
  Rows(PyObject* tokens, const char* name, PyObject* sorted, const char* sorted_name, PyObject* offsets) {
    dt = float_type(tokens, name);
    code = code_of(dt);
    const Shape td = dims(tokens, name, 2);
    T = td[0];
    d = td[1];
    const int64_t n = dims(sorted, sorted_name, 2)[0];
    E = dims(offsets, "offsets", 1)[0] - 1;
    if ((T ? n % T : n) != 0)
      raise(PyExc_ValueError, std::string(sorted_name) + " has " + std::to_string(n) + " rows, not a multiple of the " +
                                  std::to_string(T) + " tokens");
    k = T ? n / T : 1;
  }
  int64_t n() const { return T * k; }
};

// x, slot_of, offsets, xs, stream
void gather(PyObject* const* a) {
  Args arg;
  const Rows r(a[0], "x", a[3], "xs", a[2]);
  const void* x = arg(a[0], "x", r.dt, {r.T, r.d});
  auto* slot_of = arg.as<int32_t>(a[1], "slot_of", kI32, {r.n()});
  auto* offsets = arg.as<int32_t>(a[2], "offsets", kI32, {r.E + 1});
  void* xs = arg(a[3], "xs", r.dt, {r.n(), r.d});
  const int dev = arg.device();
  void* s = stream_of(a[4], dev);
  call(dev, "moe_gather", [&] { return lib.gather(x, slot_of, offsets, r.code, r.T, r.E, r.k, r.d, xs, s); });
}

// dxs, row_of, offsets, dx, stream
void gather_bwd(PyObject* const* a) {
  Args arg;
  const Rows r(a[3], "dx", a[0], "dxs", a[2]);
  const void* dxs = arg(a[0], "dxs", r.dt, {r.n(), r.d});
  auto* row_of = arg.as<int32_t>(a[1], "row_of", kI32, {r.n()});
  auto* offsets = arg.as<int32_t>(a[2], "offsets", kI32, {r.E + 1});
  void* dx = arg(a[3], "dx", r.dt, {r.T, r.d});
  const int dev = arg.device();
  void* s = stream_of(a[4], dev);
  call(dev, "moe_gather_bwd", [&] { return lib.gather_bwd(dxs, row_of, offsets, r.code, r.T, r.E, r.k, r.d, dx, s); });
}

// ys, weights, row_of, offsets, out, residual, stream
void combine(PyObject* const* a) {
  Args arg;
  const Rows r(a[4], "out", a[0], "ys", a[3]);
  const void* ys = arg(a[0], "ys", r.dt, {r.n(), r.d});
  auto* w = arg.as<float>(a[1], "weights", kF32, {r.T, r.k});
  auto* row_of = arg.as<int32_t>(a[2], "row_of", kI32, {r.n()});
  auto* offsets = arg.as<int32_t>(a[3], "offsets", kI32, {r.E + 1});
  const void* res = arg.opt(a[5], "residual", r.dt, {r.T, r.d});
  void* out = arg(a[4], "out", r.dt, {r.T, r.d});
  const int dev = arg.device();
  void* s = stream_of(a[6], dev);
  call(dev, "moe_combine",
       [&] { return lib.combine(ys, w, row_of, offsets, res, r.code, r.T, r.E, r.k, r.d, out, s); });
}

// dout, ys, weights, row_of, slot_of, offsets, dys, dweights, stream
void combine_bwd(PyObject* const* a) {
  Args arg;
  const Rows r(a[0], "dout", a[1], "ys", a[5]);
  arg(a[3], "row_of", kI32, {r.n()});
  const void* dout = arg(a[0], "dout", r.dt, {r.T, r.d});
  const void* ys = arg(a[1], "ys", r.dt, {r.n(), r.d});
  auto* w = arg.as<float>(a[2], "weights", kF32, {r.T, r.k});
  auto* slot_of = arg.as<int32_t>(a[4], "slot_of", kI32, {r.n()});
  auto* offsets = arg.as<int32_t>(a[5], "offsets", kI32, {r.E + 1});
  void* dys = arg(a[6], "dys", r.dt, {r.n(), r.d});
  auto* dw = arg.as<float>(a[7], "dweights", kF32, {r.T, r.k});
  const int dev = arg.device();
  void* s = stream_of(a[8], dev);
  call(dev, "moe_combine_bwd",
       [&] { return lib.combine_bwd(dout, ys, w, slot_of, offsets, r.code, r.T, r.E, r.k, r.d, dys, dw, s); });
}

// A linear_desc (moe.py's ctypes structure) and the shapes that it gives the tensors.
struct Desc {
  linear_desc d;
  ScalarType dt;
  int64_t P;
  explicit Desc(PyObject* o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw PyFailed{};
    const bool fits = b.len == (Py_ssize_t)sizeof d;
    if (fits) memcpy(&d, b.buf, sizeof d);
    PyBuffer_Release(&b);
    if (!fits) raise(PyExc_ValueError, "desc must be a LinearDesc");
    dt = type_of(d.dtype);
    const bool gated = d.act == MLP_ACT_SWIGLU || d.act == MLP_ACT_GEGLU || d.act == MLP_ACT_REGLU || d.act == MLP_ACT_GLU;
    P = gated ? 2 * d.N : d.N;
    weight_[0] = bias_[0] = d.experts;
    weight_[1] = bias_[1] = d.N;
    weight_[2] = d.K;
  }
  Shape weight() const { return d.experts ? Shape(weight_, 3) : Shape(weight_ + 1, 2); }
  Shape bias() const { return d.experts ? Shape(bias_, 2) : Shape(bias_ + 1, 1); }

 private:
  int64_t weight_[3], bias_[2];
};

// desc, x, w, y, w_up, bias, bias_up, residual, offsets, preact, workspace, stream
void fwd(PyObject* const* a) {
  Args arg;
  const Desc q(a[0]);
  const int64_t M = q.d.M, K = q.d.K, N = q.d.N;
  const void* x = arg(a[1], "x", q.dt, {M, K});
  const void* w = arg(a[2], "w", q.dt, q.weight());
  const void* w_up = arg.opt(a[4], "w_up", q.dt, q.weight());
  const void* bias = arg.opt(a[5], "bias", q.dt, q.bias());
  const void* bias_up = arg.opt(a[6], "bias_up", q.dt, q.bias());
  const void* res = arg.opt(a[7], "residual", q.dt, {M, N});
  auto* offsets = static_cast<int32_t*>(arg.opt(a[8], "offsets", kI32, {q.d.experts + 1}));
  void* y = arg(a[3], "y", q.dt, {M, N});
  void* preact = arg.opt(a[9], "preact", q.dt, {M, q.P});
  const int dev = arg.device();
  void* s = stream_of(a[11], dev);
  const Workspace ws(a[10], dev, s, [&] { return needed(lib.linear_bytes(&q.d, LINEAR_FWD), "linear_workspace_bytes"); });
  call(dev, "linear_fwd",
       [&] { return lib.fwd(&q.d, x, w, w_up, bias, bias_up, res, offsets, y, preact, ws.ptr, ws.bytes, s); });
}

// desc, dy, x, w, w_up, preact, offsets, dx, dw, dw_up, dbias, dbias_up, grad_accum, workspace, stream
void bwd(PyObject* const* a) {
  Args arg;
  const Desc q(a[0]);
  const int64_t M = q.d.M, K = q.d.K, N = q.d.N;
  const int accum = (int)integer(a[12]);
  const ScalarType gt = accum ? kF32 : q.dt;
  const void* dy = arg(a[1], "dy", q.dt, {M, N});
  const void* x = arg(a[2], "x", q.dt, {M, K});
  const void* w = arg(a[3], "w", q.dt, q.weight());
  const void* w_up = arg.opt(a[4], "w_up", q.dt, q.weight());
  const void* preact = arg.opt(a[5], "preact", q.dt, {M, q.P});
  auto* offsets = static_cast<int32_t*>(arg.opt(a[6], "offsets", kI32, {q.d.experts + 1}));
  void* dx = arg.opt(a[7], "dx", q.dt, {M, K});
  void* dw = arg.opt(a[8], "dw", gt, q.weight());
  void* dw_up = arg.opt(a[9], "dw_up", gt, q.weight());
  void* dbias = arg.opt(a[10], "dbias", gt, q.bias());
  void* dbias_up = arg.opt(a[11], "dbias_up", gt, q.bias());
  const int dev = arg.device();
  void* s = stream_of(a[14], dev);
  const Workspace ws(a[13], dev, s, [&] { return needed(lib.linear_bytes(&q.d, LINEAR_BWD), "linear_workspace_bytes"); });
  call(dev, "linear_bwd", [&] {
    return lib.bwd(&q.d, dy, x, w, w_up, preact, offsets, dx, dw, dw_up, dbias, dbias_up, accum, ws.ptr, ws.bytes, s);
  });
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFailed{};
  return (float)v;
}

// A norm_desc from the rows' tensor and the weight's; the first of `given` that is a tensor has the weights' type.
norm_desc norm_of(PyObject* rows, const char* name, std::initializer_list<PyObject*> given, PyObject* kind, PyObject* eps) {
  const ScalarType dt = float_type(rows, name);
  const Shape md = dims(rows, name, 2);
  ScalarType wt = dt;
  for (PyObject* o : given)
    if (o != Py_None) {
      wt = float_type(o, "weight");
      break;
    }
  return {md[0], md[1], code_of(dt), code_of(wt), (int32_t)integer(kind), eps == nullptr ? 0.0f : real(eps)};
}

// x, y, weight, bias, residual, h, mean, rstd, kind, eps, stream
void norm_fwd(PyObject* const* a) {
  Args arg;
  const norm_desc q = norm_of(a[0], "x", {a[2], a[3]}, a[8], a[9]);
  const ScalarType dt = type_of(q.dtype), wt = type_of(q.wdtype);
  const void* x = arg(a[0], "x", dt, {q.M, q.d});
  void* y = arg(a[1], "y", dt, {q.M, q.d});
  const void* w = arg.opt(a[2], "weight", wt, {q.d});
  const void* b = arg.opt(a[3], "bias", wt, {q.d});
  const void* res = arg.opt(a[4], "residual", dt, {q.M, q.d});
  void* h = arg.opt(a[5], "h", dt, {q.M, q.d});
  auto* mean = static_cast<float*>(arg.opt(a[6], "mean", kF32, {q.M}));
  auto* rstd = static_cast<float*>(arg.opt(a[7], "rstd", kF32, {q.M}));
  const int dev = arg.device();
  void* s = stream_of(a[10], dev);
  call(dev, "norm_fwd", [&] { return lib.norm_fwd(&q, x, res, w, b, y, h, mean, rstd, s); });
}

// dy, h, mean, rstd, weight, dresidual, dx, dweight, dbias, kind, grad_accum, workspace, stream
void norm_bwd(PyObject* const* a) {
  Args arg;
  const int accum = (int)integer(a[10]);
  // (gradients that are added to are fp32 whatever the weights are)
  const norm_desc q = accum ? norm_of(a[0], "dy", {a[4]}, a[9], nullptr) : norm_of(a[0], "dy", {a[4], a[7], a[8]}, a[9], nullptr);
  const ScalarType dt = type_of(q.dtype), wt = type_of(q.wdtype), gt = accum ? kF32 : wt;
  const void* dy = arg(a[0], "dy", dt, {q.M, q.d});
  const void* h = arg(a[1], "h", dt, {q.M, q.d});
  auto* mean = static_cast<float*>(arg.opt(a[2], "mean", kF32, {q.M}));
  auto* rstd = arg.as<float>(a[3], "rstd", kF32, {q.M});
  const void* w = arg.opt(a[4], "weight", wt, {q.d});
  const void* dres = arg.opt(a[5], "dresidual", dt, {q.M, q.d});
  void* dx = arg.opt(a[6], "dx", dt, {q.M, q.d});
  void* dw = arg.opt(a[7], "dweight", gt, {q.d});
  void* db = arg.opt(a[8], "dbias", gt, {q.d});
  const int dev = arg.device();
  void* s = stream_of(a[12], dev);
  auto run = [&](void* ws, size_t bytes) {
    call(dev, "norm_bwd", [&] { return lib.norm_bwd(&q, dy, h, mean, rstd, w, dres, dx, dw, db, accum, ws, bytes, s); });
  };
  if (dw == nullptr && db == nullptr) return run(nullptr, 0);   // no sums, no workspace
  const Workspace ws(a[11], dev, s, [&] { return needed(lib.norm_bytes(q.M, q.d), "norm_workspace_bytes"); });
  run(ws.ptr, ws.bytes);
}

constexpr ScalarType kU8 = ScalarType::Byte;

// The codes and scales of [batch][rows][K] (n dimensions with the batch, or two without), and their device pointers.
struct Blocks {
  Blocks(int64_t n, int64_t batch, int64_t rows, int64_t K)
      : codes_{batch, rows, K / 2}, scales_{batch, lib.mx4_planes(K), lib.mx4_scale_rows(rows), 8}, skip_(n == 3 ? 0 : 1) {}
  Shape codes() const { return Shape(codes_ + skip_, 3 - skip_); }
  Shape scales() const { return Shape(scales_ + skip_, 4 - skip_); }

 private:
  int64_t codes_[3], scales_[4];
  int skip_;
};

// A matrix, or a batch of them.
struct Matrix {
  int64_t n, batch, rows, cols;
  Matrix(PyObject* o, const char* name) {
    n = THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 3 ? 3 : 2;
    const Shape s = dims(o, name, n);
    batch = n == 3 ? s[0] : 1;
    rows = s[n - 2];
    cols = s[n - 1];
  }
};

// x, codes, scales, codes_t, scales_t, stream
void mx4_quantize(PyObject* const* a) {
  Args arg;
  const ScalarType dt = float_type(a[0], "x");
  const Matrix m(a[0], "x");
  const Blocks b(m.n, m.batch, m.rows, m.cols), t(m.n, m.batch, m.cols, (m.rows + 31) / 32 * 32);
  const void* x = arg(a[0], "x", dt, THPVariable_Unpack(a[0]).sizes());
  void* codes = arg.opt(a[1], "codes", kU8, b.codes());
  void* scales = arg.opt(a[2], "scales", kU8, b.scales());
  void* codes_t = arg.opt(a[3], "codes_t", kU8, t.codes());
  void* scales_t = arg.opt(a[4], "scales_t", kU8, t.scales());
  const int dev = arg.device();
  void* s = stream_of(a[5], dev);
  call(dev, "mx4_quantize", [&] {
    return lib.mx4_quantize(x, code_of(dt), m.batch, m.rows, m.cols, codes, scales, codes_t, scales_t, s);
  });
}

// codes, scales, out, stream
void mx4_dequantize(PyObject* const* a) {
  Args arg;
  const ScalarType dt = float_type(a[2], "out");
  const Matrix m(a[2], "out");
  const Blocks b(m.n, m.batch, m.rows, m.cols);
  const void* codes = arg(a[0], "codes", kU8, b.codes());
  const void* scales = arg(a[1], "scales", kU8, b.scales());
  void* out = arg(a[2], "out", dt, THPVariable_Unpack(a[2]).sizes());
  const int dev = arg.device();
  void* s = stream_of(a[3], dev);
  call(dev, "mx4_dequantize", [&] { return lib.mx4_dequantize(codes, scales, code_of(dt), m.batch, m.rows, m.cols, out, s); });
}

// desc, x, x_scales, w, w_scales, y, w_up, w_up_scales, bias, bias_up, residual, offsets, preact, workspace, stream
void mx4_fwd(PyObject* const* a) {
  Args arg;
  const Desc q(a[0]);
  const int64_t M = q.d.M, K = q.d.K, N = q.d.N, E = q.d.experts;
  const Blocks bx(2, 1, M, K), bw(E ? 3 : 2, E ? E : 1, N, K);
  const void* x = arg(a[1], "x", kU8, bx.codes());
  const void* xs = arg(a[2], "x_scales", kU8, bx.scales());
  const void* w = arg(a[3], "w", kU8, bw.codes());
  const void* wsc = arg(a[4], "w_scales", kU8, bw.scales());
  void* y = arg(a[5], "y", q.dt, {M, N});
  const void* w_up = arg.opt(a[6], "w_up", kU8, bw.codes());
  const void* w_ups = arg.opt(a[7], "w_up_scales", kU8, bw.scales());
  const void* bias = arg.opt(a[8], "bias", q.dt, q.bias());
  const void* bias_up = arg.opt(a[9], "bias_up", q.dt, q.bias());
  const void* res = arg.opt(a[10], "residual", q.dt, {M, N});
  auto* offsets = static_cast<int32_t*>(arg.opt(a[11], "offsets", kI32, {E + 1}));
  void* preact = arg.opt(a[12], "preact", q.dt, {M, q.P});
  const int dev = arg.device();
  void* s = stream_of(a[14], dev);
  const Workspace ws(a[13], dev, s, [&] { return needed(lib.mx4_bytes(&q.d), "mx4_linear_workspace_bytes"); });
  call(dev, "mx4_linear_fwd", [&] {
    return lib.mx4_fwd(&q.d, x, xs, w, wsc, w_up, w_ups, bias, bias_up, res, offsets, y, preact, ws.ptr, ws.bytes, s);
  });
}

// addresses of the library's entry points in Entry's order, MlpError, workspace(bytes, device, stream), raw_stream(device)
PyObject* setup(PyObject*, PyObject* args) {
  PyObject *at, *error, *workspace, *raw_stream;
  if (!PyArg_ParseTuple(args, "O!OOO", &PyTuple_Type, &at, &error, &workspace, &raw_stream)) return nullptr;
  constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);
  if (PyTuple_GET_SIZE(at) != kEntries) {
    PyErr_SetString(PyExc_ValueError, "wrong number of entry points");
    return nullptr;
  }
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i));
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is NULL");
      return nullptr;
    }
  }
  memcpy(&lib, p, sizeof lib);
  Py_INCREF(error);
  Py_INCREF(workspace);
  Py_INCREF(raw_stream);
  py_error = error;
  py_workspace = workspace;
  py_raw_stream = raw_stream;
  Py_RETURN_NONE;
}

#define BIND_ENTRY(name, n, body) {name, (PyCFunction)(void (*)(void))entry<n, body>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    BIND_ENTRY("moe_route", 6, route),
    BIND_ENTRY("moe_route_bwd", 7, route_bwd),
    BIND_ENTRY("moe_sort", 7, sort),
    BIND_ENTRY("moe_gather", 5, gather),
    BIND_ENTRY("moe_gather_bwd", 5, gather_bwd),
    BIND_ENTRY("moe_combine", 7, combine),
    BIND_ENTRY("moe_combine_bwd", 9, combine_bwd),
    BIND_ENTRY("linear_fwd", 12, fwd),
    BIND_ENTRY("linear_bwd", 15, bwd),
    BIND_ENTRY("moe_balance", 9, balance),
    BIND_ENTRY("moe_balance_bwd", 10, balance_bwd),
    BIND_ENTRY("norm_fwd", 11, norm_fwd),
    BIND_ENTRY("norm_bwd", 13, norm_bwd),
    BIND_ENTRY("mx4_quantize", 6, mx4_quantize),
    BIND_ENTRY("mx4_dequantize", 4, mx4_dequantize),
    BIND_ENTRY("mx4_linear_fwd", 15, mx4_fwd),
    {"setup", setup, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
