// Argument marshalling of the operators around the layer, as a Python module.
//
// A decode step makes several of these calls a token and their kernels run for two
// to twenty microseconds, about as long as Python takes to check the tensors and to
// fill a ctypes structure (measured: 12 us a call of causal_conv on one token
// through ctypes).  This module checks shapes, types, strides and devices,
// allocates the outputs through torch's allocator and calls the C ABI of
// include/ittt.h; it computes nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>

#include "ittt.h"

namespace {

decltype(&ittt_linear) f_linear;
decltype(&ittt_causal_conv) f_conv;
decltype(&ittt_selective_scan_workspace_size) f_scan_ws;
decltype(&ittt_selective_scan) f_scan;
PyObject* g_error;  // IttTError(status, where)

struct Refused {
  PyObject* type;
  std::string text;
};
struct Failed {
  ittt_status status;
  const char* where;
};

template <typename... Ts>
[[noreturn]] void refuse(const Ts&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Refused{PyExc_ValueError, s.str()};
}

void check(ittt_status s, const char* where) {
  if (s != ITTT_OK) throw Failed{s, where};
}

using Shape = c10::SmallVector<int64_t, 6>;

std::string text_of(at::IntArrayRef v) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < v.size(); ++i) s << (i ? ", " : "") << v[i];
  s << (v.size() == 1 ? ",)" : ")");
  return s.str();
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

int32_t dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return ITTT_BF16;
  if (t.scalar_type() == at::kFloat) return ITTT_F32;
  throw Refused{PyExc_TypeError, std::string("unsupported dtype ") + name_of(t.scalar_type())};
}

void fits(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype,
          c10::DeviceIndex dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(name, " is on ", t.device().str(), ", expected cuda:", int(dev));
  if (t.scalar_type() != dtype)
    refuse(name, " has dtype ", name_of(t.scalar_type()), ", expected ", name_of(dtype));
  if (t.sizes() != shape)
    refuse(name, " has shape ", text_of(t.sizes()), ", expected ", text_of(shape));
}

// The address of a dense tensor of this shape, type and device (nullptr for None).
void* dense(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype,
            c10::DeviceIndex dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  fits(t, name, shape, dtype, dev);
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
  return t.data_ptr();
}

// Elements between the rows of a [..., width] tensor whose rows are a fixed distance
// apart (dense: 0; or a column slice of a dense tensor).  `inner` trailing dimensions
// make up a row.
int64_t row_stride(const at::Tensor& t, const char* name, int inner = 1) {
  if (t.is_contiguous()) return 0;
  const auto sizes = t.sizes(), strides = t.strides();
  const int rows = int(sizes.size()) - inner;
  int64_t width = 1;
  bool ok = true;
  for (int i = int(sizes.size()) - 1; i >= rows; --i) {
    ok = ok && (sizes[i] == 1 || strides[i] == width);
    width *= sizes[i];
  }
  if (!ok && inner > 1)
    refuse("the groups of ", name, " must stand side by side (strides ", text_of(strides), ")");
  int64_t ld = -1, step = 0;
  for (int i = rows - 1; i >= 0; --i) {
    if (sizes[i] == 1) continue;
    if (ld < 0) ld = step = strides[i];
    ok = ok && strides[i] == step;
    step *= sizes[i];
  }
  if (ld < 0) ld = width;
  if (!ok || ld < width)
    refuse(name, " must be dense, or a column slice of a dense tensor (shape ", text_of(sizes),
           ", strides ", text_of(strides), ")");
  return ld;
}

struct Rows {
  void* ptr = nullptr;
  int64_t ld = 0;
};

Rows rows(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype,
          c10::DeviceIndex dev, int inner = 1) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor(o, name);
  fits(t, name, shape, dtype, dev);
  return {t.data_ptr(), row_stride(t, name, inner)};
}

c10::DeviceIndex gpu_of(const at::Tensor& t) {
  if (!t.is_cuda()) refuse("the operands must be CUDA tensors");
  return c10::DeviceIndex(t.get_device());
}

// The call's device made current, and its stream: the given one, or the device's
// current one.  What is made for work on a given stream comes from that stream's
// memory (no earlier work elsewhere may still use it) and is marked as used on the
// current stream, where the caller goes on (it is not given out again before the
// work queued there by the time it is freed).
struct Place {
  c10::cuda::CUDAGuard guard;
  c10::cuda::CUDAStream current;
  std::optional<c10::cuda::CUDAStream> given;

  Place(c10::DeviceIndex dev, PyObject* stream)
      : guard(dev), current(c10::cuda::getCurrentCUDAStream(dev)) {
    if (stream == Py_None) return;
    if (!THPStream_Check(stream)) throw Refused{PyExc_TypeError, "stream must be a torch.cuda.Stream"};
    const auto* s = reinterpret_cast<THPStream*>(stream);
    const c10::Stream g = c10::Stream::unpack3(s->stream_id, c10::DeviceIndex(s->device_index),
                                               static_cast<c10::DeviceType>(s->device_type));
    if (g.device_type() != c10::DeviceType::CUDA || g.device_index() != dev)
      refuse("stream belongs to another device than the operands");
    given.emplace(g);
  }

  cudaStream_t raw() const { return given ? given->stream() : current.stream(); }

  at::Tensor make(at::IntArrayRef shape, at::ScalarType dtype, bool zeros = false) {
    const c10::Device dev(c10::DeviceType::CUDA, current.device_index());
    std::optional<c10::cuda::CUDAStreamGuard> on;
    if (given) on.emplace(*given);
    at::Tensor t = at::detail::empty_cuda(shape, dtype, dev, std::nullopt);
    if (zeros && t.numel()) t.zero_();
    if (given && t.numel()) t.record_stream(current.unwrap());
    return t;
  }
};

PyObject* given_or(PyObject* o, at::Tensor& made) {
  if (o != Py_None) {
    Py_INCREF(o);
    return o;
  }
  return THPVariable_Wrap(std::move(made));
}

PyObject* pair_of(PyObject* a, PyObject* b) {
  if (!a || !b) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    return nullptr;
  }
  PyObject* t = PyTuple_Pack(2, a, b);
  Py_DECREF(a);
  Py_DECREF(b);
  return t;
}

template <typename Fn>
PyObject* guarded(Fn&& fn) {
  try {
    return fn();
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const Failed& e) {
    PyObject* v = PyObject_CallFunction(g_error, "is", int(e.status), e.where);
    if (v) {
      PyErr_SetObject(g_error, v);
      Py_DECREF(v);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

bool arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return false;
}

// linear(X, W, bias, residual, act, out, stream)
PyObject* py_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "W");
    const at::ScalarType dt = X.scalar_type();
    ittt_linear_problem p{};
    p.dtype = dtype_code(X);
    if (X.dim() < 1 || W.dim() != 2) refuse("X must have shape [..., K] and W [N, K]");
    p.N = W.size(0);
    p.K = W.size(1);
    if (X.size(-1) != p.K) refuse("X has ", X.size(-1), " columns, W ", p.K);
    p.act = int32_t(PyLong_AsLong(a[4]));
    const c10::DeviceIndex dev = gpu_of(X);
    Shape shape(X.sizes().begin(), X.sizes().end());
    shape.back() = p.N;
    p.M = 1;
    for (size_t i = 0; i + 1 < shape.size(); ++i) p.M *= shape[i];
    p.ldx = row_stride(X, "X");
    const void* w = dense(a[1], "W", W.sizes(), dt, dev);
    const void* bias = dense(a[2], "bias", {p.N}, dt, dev);
    const Rows r = rows(a[3], "residual", shape, dt, dev);
    Rows y = rows(a[5], "out", shape, dt, dev);
    Place at_(dev, a[6]);
    at::Tensor out;
    if (a[5] == Py_None) {
      out = at_.make(shape, dt);
      y.ptr = out.data_ptr();
    }
    p.ldr = r.ld;
    p.ldy = y.ld;
    check(f_linear(&p, X.data_ptr(), w, bias, r.ptr, y.ptr, at_.raw()), "ittt_linear");
    return given_or(a[5], out);
  });
}

// causal_conv(X, conv_kernel, bias, act, state, lengths, out, state_out, stream)
PyObject* py_conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &X = tensor(a[0], "X"), &w = tensor(a[1], "conv_kernel");
    const at::ScalarType dt = X.scalar_type();
    ittt_conv_problem p{};
    p.dtype = dtype_code(X);
    if (X.dim() != 3 || w.dim() != 2) refuse("X must have shape [B, T, d] and conv_kernel [d, k]");
    p.B = X.size(0);
    p.T = X.size(1);
    p.d = X.size(2);
    p.k = int32_t(std::min<int64_t>(w.size(1), 1 << 20));
    p.act = int32_t(PyLong_AsLong(a[3]));
    const c10::DeviceIndex dev = gpu_of(X);
    p.ldx = row_stride(X, "X");
    const void* taps = dense(a[1], "conv_kernel", {p.d, w.size(1)}, dt, dev);
    const void* bias = dense(a[2], "bias", {p.d}, dt, dev);
    const Shape state_shape{p.B, std::max<int64_t>(p.k - 1, 0), p.d};
    const void* s_in = dense(a[4], "state", state_shape, dt, dev);
    const void* len = dense(a[5], "lengths", {p.B}, at::kInt, dev);
    Rows y = rows(a[6], "out", X.sizes(), dt, dev);
    void* s_out = dense(a[7], "state_out", state_shape, dt, dev);
    Place at_(dev, a[8]);
    at::Tensor out, state;
    if (a[6] == Py_None) {
      // rows behind a sequence's end are not written: they come out as zeros
      out = at_.make(X.sizes(), dt, len != nullptr);
      y.ptr = out.data_ptr();
    }
    if (a[7] == Py_None) {
      state = at_.make(state_shape, dt);
      s_out = state.data_ptr();
    }
    p.ldy = y.ld;
    check(f_conv(&p, X.data_ptr(), taps, bias, s_in, static_cast<const int32_t*>(len), y.ptr, s_out, at_.raw()),
          "ittt_causal_conv");
    return pair_of(given_or(a[6], out), given_or(a[7], state));
  });
}

// selective_scan(U, delta, A, Bm, Cm, D, Z, dt_bias, flags, state, lengths, out,
//                state_out, workspace, stream)
PyObject* py_scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 15)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &U = tensor(a[0], "U"), &A = tensor(a[2], "A"), &Bm = tensor(a[3], "Bm");
    const at::ScalarType dt = U.scalar_type();
    ittt_scan_problem p{};
    p.dtype = dtype_code(U);
    const bool grouped = Bm.dim() == 4;
    if (U.dim() != 3 || A.dim() != 2 || (Bm.dim() != 3 && !grouped))
      refuse("U must have shape [B, T, d], A [d, N], Bm and Cm [B, T, N] or [B, T, G, N]");
    p.B = U.size(0);
    p.T = U.size(1);
    p.d = U.size(2);
    p.N = int32_t(std::min<int64_t>(A.size(1), 1 << 20));
    p.G = grouped ? int32_t(std::min<int64_t>(Bm.size(2), 1 << 30)) : 1;
    p.flags = int32_t(PyLong_AsLong(a[8]));
    const c10::DeviceIndex dev = gpu_of(U);
    p.ldu = row_stride(U, "U");
    const Rows delta = rows(a[1], "delta", U.sizes(), dt, dev), z = rows(a[6], "Z", U.sizes(), dt, dev);
    Shape bc{p.B, p.T};
    if (grouped) bc.push_back(p.G);
    bc.push_back(A.size(1));
    const Rows bm = rows(a[3], "Bm", bc, dt, dev, grouped ? 2 : 1);
    const Rows cm = rows(a[4], "Cm", bc, dt, dev, grouped ? 2 : 1);
    const auto* av = static_cast<const float*>(dense(a[2], "A", {p.d, A.size(1)}, at::kFloat, dev));
    const auto* d = static_cast<const float*>(dense(a[5], "D", {p.d}, at::kFloat, dev));
    const auto* db = static_cast<const float*>(dense(a[7], "dt_bias", {p.d}, at::kFloat, dev));
    const Shape state_shape{p.B, p.d, A.size(1)};
    const auto* s_in = static_cast<const float*>(dense(a[9], "state", state_shape, at::kFloat, dev));
    const auto* len = static_cast<const int32_t*>(dense(a[10], "lengths", {p.B}, at::kInt, dev));
    Rows y = rows(a[11], "out", U.sizes(), dt, dev);
    auto* s_out = static_cast<float*>(dense(a[12], "state_out", state_shape, at::kFloat, dev));
    Place at_(dev, a[14]);
    p.ldt = delta.ld;
    p.ldb = bm.ld;
    p.ldc = cm.ld;
    p.ldz = z.ld;
    p.ldy = y.ld;
    size_t need = 0;
    check(f_scan_ws(&p, &need), "ittt_selective_scan_workspace_size");
    at::Tensor out, state, scratch;
    void* ws = nullptr;
    if (need) {
      if (a[13] != Py_None) {
        const at::Tensor& w = tensor(a[13], "workspace");
        if (!w.is_cuda() || w.get_device() != dev || !w.is_contiguous())
          refuse("workspace must be a dense tensor on cuda:", int(dev));
        if (size_t(w.numel()) * w.element_size() >= need) ws = w.data_ptr();
      }
      if (!ws) {
        scratch = at_.make({int64_t(need)}, at::kByte);
        ws = scratch.data_ptr();
      }
    }
    if (a[11] == Py_None) {
      out = at_.make(U.sizes(), dt, len != nullptr);
      y.ptr = out.data_ptr();
    }
    if (a[12] == Py_None) {
      state = at_.make(state_shape, at::kFloat);
      s_out = state.data_ptr<float>();
    }
    check(f_scan(&p, U.data_ptr(), delta.ptr, av, bm.ptr, cm.ptr, d, db, z.ptr, s_in, len, y.ptr, s_out, ws,
                 need, at_.raw()),
          "ittt_selective_scan");
    return pair_of(given_or(a[11], out), given_or(a[12], state));
  });
}

// row_stride(t, inner): the row stride by which the calls describe t.
PyObject* py_row_stride(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 2)) return nullptr;
  return guarded([&]() -> PyObject* {
    return PyLong_FromLongLong(row_stride(tensor(a[0], "t"), "t", int(PyLong_AsLong(a[1]))));
  });
}

// bind(path of libittt.so, IttTError)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 2)) return nullptr;
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) return nullptr;
  void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_Format(PyExc_RuntimeError, "cannot load %s: %s", path, dlerror());
    return nullptr;
  }
  f_linear = reinterpret_cast<decltype(f_linear)>(dlsym(lib, "ittt_linear"));
  f_conv = reinterpret_cast<decltype(f_conv)>(dlsym(lib, "ittt_causal_conv"));
  f_scan_ws = reinterpret_cast<decltype(f_scan_ws)>(dlsym(lib, "ittt_selective_scan_workspace_size"));
  f_scan = reinterpret_cast<decltype(f_scan)>(dlsym(lib, "ittt_selective_scan"));
  if (!f_linear || !f_conv || !f_scan_ws || !f_scan) {
    PyErr_Format(PyExc_RuntimeError, "%s lacks an entry point", path);
    return nullptr;
  }
  Py_XDECREF(g_error);
  Py_INCREF(a[1]);
  g_error = a[1];
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", FAST(py_bind), nullptr},
    {"linear", FAST(py_linear), nullptr},
    {"causal_conv", FAST(py_conv), nullptr},
    {"selective_scan", FAST(py_scan), nullptr},
    {"row_stride", FAST(py_row_stride), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
