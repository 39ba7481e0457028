// torch_binding.cpp -- marshalling of torch tensors for the entry points whose
// device time can be a few microseconds (4-bit weights, 8-bit checkpoints, the
// backward pass): tensor checks, outputs and workspaces, the current stream.
// lynx.py is in front of it; every step of the operators is behind lynx.h.
//
// Each function takes its arguments by position.  It returns its tensors, or a
// lynx_status that is not LYNX_OK as an int; a tensor that does not fit raises.
// The same checks through Python attributes took 8 us a call of the 12.
#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "lynx.h"

namespace {

struct Refused {
  PyObject* type;
  std::string text;
};

[[noreturn]] void refuse(PyObject* type, std::string text) { throw Refused{type, std::move(text)}; }

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

// One call: its positional arguments, the current device and the stream.
class Call {
 public:
  // `first`: the name of the first argument, a tensor
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, const char* first) : args_(args) {
    if (n != want) refuse(PyExc_TypeError, "wrong number of arguments");
    if (!tensor(0, first).is_cuda()) refuse(PyExc_ValueError, std::string(first) + " must be a CUDA tensor");
    here_ = c10::cuda::current_device();
    PyObject* s = args_[want - 1];
    if (s == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream(here_).stream();
      return;
    }
    const long handle = attribute(s, "cuda_stream"), device = attribute(s, "device_index");
    if (device != here_)
      refuse(PyExc_ValueError, "stream is on cuda:" + std::to_string(device) + ", the current device is cuda:" +
                                   std::to_string(here_));
    stream_ = reinterpret_cast<cudaStream_t>(handle);
    // buffers made here come from the pool of the stream they are used on
    guard_.emplace(c10::cuda::getStreamFromExternal(stream_, static_cast<c10::DeviceIndex>(here_)));
  }

  bool given(int i) const { return args_[i] != Py_None; }

  const at::Tensor& tensor(int i, const char* name) const {
    if (args_[i] == Py_None) refuse(PyExc_ValueError, std::string(name) + " is required");
    if (!THPVariable_Check(args_[i])) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(args_[i]);
  }

  // a matrix's two extents
  std::pair<int64_t, int64_t> matrix(int i, const char* name) const {
    const at::Tensor& t = tensor(i, name);
    if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must be a matrix");
    return {t.size(0), t.size(1)};
  }

  void* in(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return check(tensor(i, name), name, type, shape);
  }

  void* optional_in(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return given(i) ? in(i, name, type, shape) : nullptr;
  }

  // the caller's tensor, or a new one kept in `made`
  void* out(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, at::Tensor& made) const {
    if (given(i)) {
      made = tensor(i, name);
      return check(made, name, type, shape);
    }
    made = at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(here_)));
    return made.data_ptr();
  }

  // (address, bytes) of the caller's workspace, or of one kept in `made`
  std::pair<void*, size_t> workspace(int i, size_t need, at::Tensor& made) const {
    if (given(i)) {
      made = tensor(i, "workspace");
      void* p = check(made, "workspace", at::kByte, {made.numel()});
      return {p, static_cast<size_t>(made.numel())};
    }
    if (need == 0) return {nullptr, 0};
    void* p = out(i, "workspace", at::kByte, {static_cast<int64_t>(need)}, made);
    return {p, need};
  }

  int integer(int i) const {
    const long v = PyLong_AsLong(args_[i]);
    const bool failed = v == -1 && PyErr_Occurred();
    if (failed) PyErr_Clear();
    if (failed || v != static_cast<int>(v)) refuse(PyExc_TypeError, "an integer is required");
    return static_cast<int>(v);
  }

  bool truth(int i) const {
    const int v = PyObject_IsTrue(args_[i]);
    if (v < 0) {
      PyErr_Clear();
      refuse(PyExc_TypeError, "a truth value is required");
    }
    return v == 1;
  }

  void* stream() const { return stream_; }

 private:
  static long attribute(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    const long r = v ? PyLong_AsLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse(PyExc_TypeError, "stream must be a torch.cuda.Stream");
    }
    return r;
  }

  void* check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (!(t.is_cuda() && t.get_device() == here_ && t.scalar_type() == type && t.sizes() == shape &&
          t.is_contiguous())) {
      const std::string n = name;
      if (!t.is_cuda()) refuse(PyExc_ValueError, n + " must be a CUDA tensor");
      if (!t.is_contiguous()) refuse(PyExc_ValueError, n + " must be contiguous");
      if (t.scalar_type() != type)
        refuse(PyExc_TypeError, n + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
      if (t.sizes() != shape)
        refuse(PyExc_ValueError, n + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
      refuse(PyExc_ValueError, n + " is on cuda:" + std::to_string(t.get_device()) + ", the current device is cuda:" +
                                   std::to_string(here_));
    }
    return t.data_ptr();
  }

  PyObject* const* args_;
  int here_ = 0;
  cudaStream_t stream_ = nullptr;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = t.defined() ? wrap(t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// No exception leaves an entry.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// N, K and groups of Wq [N,K/2] and scales [K/group,N]
struct W4 {
  int64_t N, K, groups;
  W4(const Call& c, int wq, int scales) {
    const auto q = c.matrix(wq, "Wq"), s = c.matrix(scales, "scales");
    N = q.first;
    K = 2 * q.second;
    groups = s.first;
    if (s.second != N || groups == 0 || K % groups != 0) refuse(PyExc_ValueError, "scales must be [K/group,N]");
  }
  int group() const { return K / groups > 1024 ? 1024 : static_cast<int>(K / groups); }
};

// M, K and format of a checkpoint: the dtype of q says which format it is
struct Ckpt {
  int64_t M, K;
  int format;
  at::ScalarType type;
  Ckpt(const Call& c, int q) {
    const auto s = c.matrix(q, "q");
    M = s.first;
    K = s.second;
    type = c.tensor(q, "q").scalar_type();
    if (type == at::kChar)
      format = LYNX_CKPT8_INT8;
    else if (type == at::kFloat8_e4m3fn)
      format = LYNX_CKPT8_E4M3;
    else
      refuse(PyExc_TypeError, std::string("q must be int8 or float8_e4m3fn, got ") + c10::toString(type));
  }
};

// W, group, zero_points, Wq, scales, zeros, stream
PyObject* w4_quantize(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 7, "W");
  const auto [N, K] = c.matrix(0, "W");
  const int group = c.integer(1);
  if ((group != 32 && group != 64 && group != 128) || K % group != 0) return PyLong_FromLong(LYNX_ERR_UNSUPPORTED_SHAPE);
  at::Tensor wq, scales, zeros;
  const void* w = c.in(0, "W", at::kBFloat16, {N, K});
  void* q = c.out(3, "Wq", at::kByte, {N, K / 2}, wq);
  void* s = c.out(4, "scales", at::kBFloat16, {K / group, N}, scales);
  void* z = nullptr;
  if (c.given(5) || c.truth(2)) z = c.out(5, "zeros", at::kByte, {K / group, N}, zeros);
  const int st = lynx_w4_quantize(w, N, K, group, q, s, z, c.stream());
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap_all({wq, scales, zeros});
}

// Wq, scales, zeros, W, stream
PyObject* w4_dequantize(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 5, "Wq");
  const W4 g(c, 0, 1);
  at::Tensor W;
  const void* q = c.in(0, "Wq", at::kByte, {g.N, g.K / 2});
  const void* s = c.in(1, "scales", at::kBFloat16, {g.groups, g.N});
  const void* z = c.optional_in(2, "zeros", at::kByte, {g.groups, g.N});
  void* w = c.out(3, "W", at::kBFloat16, {g.N, g.K}, W);
  const int st = lynx_w4_dequantize(q, s, z, g.N, g.K, g.group(), w, c.stream());
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap(W);
}

// X, Wq, scales, zeros, bias, A, B, act, Y, workspace, stream
PyObject* linear_w4(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 11, "X");
  const W4 g(c, 1, 2);
  const auto [M, k] = c.matrix(0, "X");
  if (k != g.K) refuse(PyExc_ValueError, "X must be [M,K] with K = 2 * Wq.shape[1]");
  at::Tensor Y, ws;
  const void* x = c.in(0, "X", at::kBFloat16, {M, g.K});
  const void* q = c.in(1, "Wq", at::kByte, {g.N, g.K / 2});
  const void* s = c.in(2, "scales", at::kBFloat16, {g.groups, g.N});
  const void* z = c.optional_in(3, "zeros", at::kByte, {g.groups, g.N});
  const void* bias = c.optional_in(4, "bias", at::kBFloat16, {g.N});
  const void *a = nullptr, *b = nullptr;
  int64_t r = 0;
  std::pair<void*, size_t> work{nullptr, 0};
  if (c.given(5) != c.given(6)) refuse(PyExc_ValueError, "A and B must both be given or both be None");
  if (c.given(5)) {
    r = c.matrix(5, "A").first;
    a = c.in(5, "A", at::kBFloat16, {r, g.K});
    b = c.in(6, "B", at::kBFloat16, {g.N, r});
    work = c.workspace(9, lynx_linear_w4_workspace_bytes(M, g.N, g.K, r), ws);
  }
  void* y = c.out(8, "Y", at::kBFloat16, {M, g.N}, Y);
  const int st = lynx_linear_w4(x, q, s, z, bias, a, b, M, g.N, g.K, r, g.group(), c.integer(7), y,
                                work.first, work.second, c.stream());
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap(Y);
}

// X, format, q, e, stream
PyObject* ckpt8_store(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 5, "X");
  const auto [M, K] = c.matrix(0, "X");
  const int format = c.integer(1);
  if (format != LYNX_CKPT8_INT8 && format != LYNX_CKPT8_E4M3) return PyLong_FromLong(LYNX_ERR_INVALID_ARG);
  at::Tensor q, e;
  const void* x = c.in(0, "X", at::kBFloat16, {M, K});
  void* qp = c.out(2, "q", format == LYNX_CKPT8_INT8 ? at::kChar : at::kFloat8_e4m3fn, {M, K}, q);
  void* ep = c.out(3, "e", at::kByte, {M, K / 32}, e);
  const int st = lynx_ckpt8_store(x, M, K, format, qp, ep, c.stream());
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap_all({q, e});
}

// q, e, X, stream
PyObject* ckpt8_restore(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 4, "q");
  const Ckpt k(c, 0);
  at::Tensor X;
  const void* q = c.in(0, "q", k.type, {k.M, k.K});
  const void* e = c.in(1, "e", at::kByte, {k.M, k.K / 32});
  void* x = c.out(2, "X", at::kBFloat16, {k.M, k.K}, X);
  const int st = lynx_ckpt8_restore(q, e, k.M, k.K, k.format, x, c.stream());
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap(X);
}

// dY, q, e, A, B, dA, dB, dT, workspace, stream
PyObject* lora_backward(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 10, "dY");
  const Ckpt k(c, 1);
  const auto [m, N] = c.matrix(0, "dY");
  if (m != k.M) refuse(PyExc_ValueError, "dY must be [M,N] with the checkpoint's M");
  const int64_t r = c.matrix(3, "A").first;
  at::Tensor dA, dB, dT, ws;
  const void* dy = c.in(0, "dY", at::kBFloat16, {k.M, N});
  const void* q = c.in(1, "q", k.type, {k.M, k.K});
  const void* e = c.in(2, "e", at::kByte, {k.M, k.K / 32});
  const void* a = c.in(3, "A", at::kBFloat16, {r, k.K});
  const void* b = c.in(4, "B", at::kBFloat16, {N, r});
  void* da = c.out(5, "dA", at::kBFloat16, {r, k.K}, dA);
  void* db = c.out(6, "dB", at::kBFloat16, {N, r}, dB);
  void* dt = c.out(7, "dT", at::kBFloat16, {k.M, r}, dT);
  const auto work = c.workspace(8, lynx_lora_backward_workspace_bytes(k.M, N, k.K, r), ws);
  const int st = lynx_lora_backward(dy, q, e, a, b, k.M, N, k.K, r, k.format, da, db, dt, work.first, work.second,
                                    c.stream());
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap_all({dA, dB, dT});
}

// G, q, e, dT, A, dX, workspace, meta, stream
PyObject* sparsify_backward(PyObject* const* args, Py_ssize_t n) {
  const Call c(args, n, 9, "G");
  const Ckpt k(c, 1);
  at::Tensor dX, ws;
  const void* g = c.in(0, "G", at::kBFloat16, {k.M, k.K});
  const void* q = c.in(1, "q", k.type, {k.M, k.K});
  const void* e = c.in(2, "e", at::kByte, {k.M, k.K / 32});
  const void *dt = nullptr, *a = nullptr;
  int64_t r = 0;
  if (c.given(3) != c.given(4)) refuse(PyExc_ValueError, "dT and A must both be given or both be None");
  if (c.given(4)) {
    r = c.matrix(4, "A").first;
    a = c.in(4, "A", at::kBFloat16, {r, k.K});
    dt = c.in(3, "dT", at::kBFloat16, {k.M, r});
  }
  void* dx = c.out(5, "dX", at::kBFloat16, {k.M, k.K}, dX);
  const auto work = c.workspace(6, lynx_sparsify_backward_workspace_bytes(k.M, k.K), ws);
  int st;
  if (c.given(7)) {
    const at::Tensor& t = c.tensor(7, "meta");
    const void* meta = c.in(7, "meta", at::kByte, {t.numel()});
    if (static_cast<size_t>(t.numel()) < lynx_meta_bytes(k.M, k.K))
      refuse(PyExc_ValueError, "meta must have lynx_meta_bytes(M, K) bytes");
    st = lynx_sparsify_backward_meta(g, q, e, meta, dt, a, k.M, k.K, r, k.format, dx, work.first, work.second,
                                     c.stream());
  } else {
    st = lynx_sparsify_backward(g, q, e, dt, a, k.M, k.K, r, k.format, dx, work.first, work.second, c.stream());
  }
  return st != LYNX_OK ? PyLong_FromLong(st) : wrap(dX);
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<w4_quantize>("w4_quantize"),
                           method<w4_dequantize>("w4_dequantize"),
                           method<linear_w4>("linear_w4"),
                           method<ckpt8_store>("ckpt8_store"),
                           method<ckpt8_restore>("ckpt8_restore"),
                           method<lora_backward>("lora_backward"),
                           method<sparsify_backward>("sparsify_backward"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_lynx_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lynx_torch(void) { return PyModule_Create(&g_module); }
