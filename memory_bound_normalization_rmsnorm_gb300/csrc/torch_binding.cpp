// torch_binding.cpp -- the tensor side of the dropout and group-normalisation
// entry points: argument checks, output and workspace allocation, the
// current stream, and the C ABI call, in one native call.
//
// These operators run in 2 to 10 us on small tensors, less than a binding
// costs that checks, allocates and calls step by step from Python: 26 us for
// a group-norm forward whose kernel takes 3.6 us (Neoverse V2 host).  The
// functions take positional arguments from _binding.py, which owns the
// documented signatures, and return a tuple of tensors, or the status code
// (an int) that the library refused with.  Nothing is computed here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <optional>
#include <string>
#include <utility>

#include "../../include/gbnorm.h"

namespace {

struct PyFail {};  // a Python error is set

[[noreturn]] void fail(const std::string &msg) {
  PyErr_SetString(PyExc_ValueError, msg.c_str());
  throw PyFail{};
}

std::string show(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument, or undefined for None.
const at::Tensor &tensor(PyObject *o, const char *name, bool optional = false) {
  static const at::Tensor none;
  if (o == Py_None && optional) return none;
  if (!THPVariable_Check(o)) fail(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void check(const at::Tensor &t, const char *name, at::ScalarType dt, c10::IntArrayRef shape,
           c10::Device dev) {
  if (!t.defined()) return;
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  if (t.device() != dev)
    fail(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (t.scalar_type() != dt)
    fail(std::string(name) + " must be " + c10::toString(dt) + ", got " +
         c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) fail(std::string(name) + " must be contiguous");
  if (t.sizes() != shape)
    fail(std::string(name) + " has shape " + show(t.sizes()) + ", expected " + show(shape));
}

// The leading tensor argument of a call: its device is the call's.
const at::Tensor &lead(PyObject *o, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  if (!t.is_contiguous()) fail(std::string(name) + " must be contiguous");
  return t;
}

norm_dtype_t dtype_code(const at::Tensor &x) {
  switch (x.scalar_type()) {
    case at::kBFloat16: return NORM_BF16;
    case at::kHalf: return NORM_FP16;
    case at::kFloat: return NORM_FP32;
    default:
      fail(std::string("x must be bfloat16, float16 or float32, got ") +
           c10::toString(x.scalar_type()));
  }
}

// Lets other Python threads run in its scope.  A call may wait there, for
// memory, for a kernel to be loaded, or in a launch for room in a full queue;
// inside, no Python object is touched.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked &) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A new contiguous tensor over `bytes` of the current device's and stream's
// memory, at least those of its elements.  (The allocator is asked directly: by
// way of at::detail::empty_cuda, which sets the device and the sizes once more,
// a call with three outputs takes 0.5 us longer.)
at::Tensor device_tensor(int64_t bytes, at::ScalarType dt, c10::IntArrayRef shape) {
  c10::Allocator *const alloc = c10::cuda::CUDACachingAllocator::get();
  const size_t n = static_cast<size_t>(bytes);
  auto storage = c10::make_intrusive<c10::StorageImpl>(
      c10::StorageImpl::use_byte_size_t(), n, alloc->allocate(n), alloc, /*resizable=*/true);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(std::move(storage)), c10::DispatchKeySet(c10::DispatchKey::CUDA),
      c10::scalarTypeToTypeMeta(dt));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// An output: the given tensor, checked, or one that make() allocates (on the
// current device and stream).  A new one owns its memory: callers release and
// grow the storages of activations one by one, and the statistics that a
// backward pass reads must outlive that.  (One allocation shared by the outputs
// of a small call saved 0.7 us of host time and broke there.)  Its storage is a
// whole number of the caching allocator's 512-byte blocks, the memory that it
// takes either way.
struct Output {
  at::Tensor t;
  at::ScalarType dt;
  c10::DimVector shape;
  bool wanted;

  // `wanted`: None asks for a new tensor (else for no output).
  Output(PyObject *o, const char *name, at::ScalarType type, c10::IntArrayRef sizes,
         c10::Device dev, bool want = true)
      : dt(type), shape(sizes.begin(), sizes.end()), wanted(want) {
    if (o == Py_None) return;
    t = tensor(o, name);
    check(t, name, dt, sizes, dev);
  }
  void make() {
    if (t.defined() || !wanted) return;
    const int64_t bytes =
        static_cast<int64_t>(c10::elementSize(dt)) * c10::multiply_integers(shape);
    t = device_tensor((bytes + 511) & ~int64_t(511), dt, shape);
  }
};

void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFail{};
  return v;
}

// A mode or activation: -1, which the library refuses, for what an int
// cannot hold.
int code_of(PyObject *o) {
  const int64_t v = integer(o);
  return v < 0 || v > 255 ? -1 : static_cast<int>(v);
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFail{};
  return v;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyFail{};
  return v != 0;
}

uint64_t word(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);
  if (!i) throw PyFail{};
  const unsigned long long v = PyLong_AsUnsignedLongLong(i);
  Py_DECREF(i);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    fail(std::string(name) + " must be in [0, 2**64)");
  }
  return v;
}

// p, seed, offset, offset_dev of a call.
struct Rng {
  float p;
  uint64_t seed, offset;
  const void *dev_word = nullptr;

  Rng(PyObject *const *a, c10::Device dev)
      : p(static_cast<float>(number(a[0]))), seed(word(a[1], "seed")), offset(word(a[2], "offset")) {
    const at::Tensor &t = tensor(a[3], "offset_dev", true);
    if (!t.defined()) return;
    if ((t.scalar_type() != at::kLong && t.scalar_type() != at::kUInt64) || t.numel() != 1 ||
        t.device() != dev)
      fail("offset_dev must be one int64 or uint64 on " + dev.str());
    dev_word = t.data_ptr();
  }
};

// The stream argument of a call: None (the device's current stream) or a
// handle.
struct StreamArg {
  std::optional<uintptr_t> handle;

  explicit StreamArg(PyObject *o) {
    if (o == Py_None) return;
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw PyFail{};
    handle = static_cast<uintptr_t>(v);
  }
};

// The device is current inside the scope, and so is the stream, so outputs
// and workspaces come from that stream's memory: a workspace that is freed
// when the call returns is used again by later work of the same stream only.
struct StreamScope {
  norm_stream_t s;
  std::optional<c10::cuda::CUDAStreamGuard> stream;
  std::optional<c10::cuda::CUDAGuard> device;

  StreamScope(const StreamArg &arg, c10::Device dev) {
    if (!arg.handle) {
      device.emplace(dev);
      s = reinterpret_cast<norm_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
      return;
    }
    s = reinterpret_cast<norm_stream_t>(*arg.handle);
    stream.emplace(
        c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(s), dev.index()));
  }
};

// The given workspace, checked, or one that make() allocates of the bytes that
// `query` asks for.
struct Workspace {
  at::Tensor t;
  size_t bytes = 0;

  Workspace(PyObject *o, c10::Device dev) {
    if (o == Py_None) return;
    t = tensor(o, "workspace");
    if (t.device() != dev || !t.is_contiguous())
      fail("workspace must be contiguous and on " + dev.str());
    bytes = t.nbytes();
  }
  template <typename Query>
  norm_status_t make(Query query) {
    if (t.defined()) return NORM_OK;
    const norm_status_t st = query(&bytes);
    const int64_t n = static_cast<int64_t>(bytes);
    if (st == NORM_OK && n) t = device_tensor(n, at::kByte, {n});
    return st;
  }
};

PyObject *tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw PyFail{};
  Py_ssize_t i = 0;
  for (const at::Tensor &t : ts) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw PyFail{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

PyObject *result(norm_status_t st, std::initializer_list<at::Tensor> ts) {
  return st == NORM_OK ? tuple_of(ts) : PyLong_FromLong(st);
}

// No C++ exception leaves a function of the module.
template <Py_ssize_t N, typename Body>
PyObject *guarded(Py_ssize_t n, Body body) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const PyFail &) {
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// (x, p, seed, offset, offset_dev, y, stream) -> y
PyObject *dropout(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<7>(n, [&]() -> PyObject * {
    const at::Tensor &x = lead(a[0], "x");
    const norm_dtype_t dt = dtype_code(x);
    const c10::Device dev = x.device();
    const Rng rng(a + 1, dev);
    const StreamArg stream(a[6]);
    Output y(a[5], "y", x.scalar_type(), x.sizes(), dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      y.make();
      st = norm_dropout(ptr(x), x.numel(), rng.p, rng.seed, rng.offset, rng.dev_word, dt, ptr(y.t),
                        on.s);
    }
    return result(st, {y.t});
  });
}

struct Rows {
  int64_t M, N;
  c10::IntArrayRef shape, lead;
  explicit Rows(const at::Tensor &x) : shape(x.sizes()) {
    if (x.dim() < 1) fail("x must have at least one dimension");
    N = x.size(-1);
    M = N ? x.numel() / N : 0;
    lead = shape.slice(0, shape.size() - 1);
  }
};

// (x, r, gamma, beta, eps, mode, p, seed, offset, offset_dev, h, y, rstd,
// mean, stream) -> (h, y, rstd, mean)
PyObject *dropout_add_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<15>(n, [&]() -> PyObject * {
    const at::Tensor &x = lead(a[0], "x");
    const c10::Device dev = x.device();
    const Rows d(x);
    const at::ScalarType bf = at::kBFloat16;
    const at::Tensor &r = tensor(a[1], "r"), &gamma = tensor(a[2], "gamma"),
                     &beta = tensor(a[3], "beta", true);
    check(x, "x", bf, d.shape, dev);
    check(r, "r", bf, d.shape, dev);
    check(gamma, "gamma", bf, {d.N}, dev);
    check(beta, "beta", bf, {d.N}, dev);
    const float eps = static_cast<float>(number(a[4]));
    const int mode = code_of(a[5]);
    const Rng rng(a + 6, dev);
    const StreamArg stream(a[14]);
    Output h(a[10], "h", bf, d.shape, dev), y(a[11], "y", bf, d.shape, dev);
    Output rstd(a[12], "rstd", at::kFloat, d.lead, dev);
    Output mean(a[13], "mean", at::kFloat, d.lead, dev, mode == NORM_LAYER);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      for (Output *o : {&h, &y, &rstd, &mean}) o->make();
      st = norm_dropout_add_fwd(ptr(x), ptr(r), ptr(gamma), ptr(beta), d.M, d.N, eps,
                                static_cast<norm_mode_t>(mode), rng.p, rng.seed, rng.offset,
                                rng.dev_word, ptr(h.t), ptr(y.t), static_cast<float *>(ptr(rstd.t)),
                                static_cast<float *>(ptr(mean.t)), on.s);
    }
    return result(st, {h.t, y.t, rstd.t, mean.t});
  });
}

// (dy, dh, h, gamma, rstd, mean, mode, p, seed, offset, offset_dev, dx, dr,
// dgamma, dbeta, want_dbeta, workspace, stream) -> (dx, dr, dgamma, dbeta)
PyObject *dropout_add_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<18>(n, [&]() -> PyObject * {
    const at::Tensor &h = lead(a[2], "h");
    const c10::Device dev = h.device();
    const Rows d(h);
    const at::ScalarType bf = at::kBFloat16, f32 = at::kFloat;
    const at::Tensor &dy = tensor(a[0], "dy"), &dh = tensor(a[1], "dh"),
                     &gamma = tensor(a[3], "gamma"), &rstd = tensor(a[4], "rstd"),
                     &mean = tensor(a[5], "mean", true);
    check(h, "h", bf, d.shape, dev);
    check(dy, "dy", bf, d.shape, dev);
    check(dh, "dh", bf, d.shape, dev);
    check(gamma, "gamma", bf, {d.N}, dev);
    check(rstd, "rstd", f32, d.lead, dev);
    check(mean, "mean", f32, d.lead, dev);
    const norm_mode_t mode = static_cast<norm_mode_t>(code_of(a[6]));
    const Rng rng(a + 7, dev);
    const StreamArg stream(a[17]);
    Output dx(a[11], "dx", bf, d.shape, dev), dr(a[12], "dr", bf, d.shape, dev);
    Output dg(a[13], "dgamma", f32, {d.N}, dev);
    Output db(a[14], "dbeta", f32, {d.N}, dev, mode == NORM_LAYER && truth(a[15]));
    Workspace ws(a[16], dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      for (Output *o : {&dx, &dr, &dg, &db}) o->make();
      st = ws.make([&](size_t *b) { return norm_dropout_add_bwd_workspace_bytes(d.M, d.N, mode, b); });
      if (st == NORM_OK)
        st = norm_dropout_add_bwd(ptr(dy), ptr(dh), ptr(h), ptr(gamma),
                                  static_cast<const float *>(ptr(rstd)),
                                  static_cast<const float *>(ptr(mean)), d.M, d.N, mode, rng.p,
                                  rng.seed, rng.offset, rng.dev_word, ptr(dx.t), ptr(dr.t),
                                  static_cast<float *>(ptr(dg.t)), static_cast<float *>(ptr(db.t)),
                                  ptr(ws.t), ws.bytes, on.s);
    }
    return result(st, {dx.t, dr.t, dg.t, db.t});
  });
}

struct Samples {
  int64_t B, S, C;
  explicit Samples(const at::Tensor &x) {
    if (x.dim() < 2) fail("x must be [B, ..., C]");
    B = x.size(0);
    C = x.size(-1);
    S = B && C ? x.numel() / (B * C) : 0;
  }
};

// (x, gamma, beta, groups, eps, act, p, seed, offset, offset_dev, y, rstd,
// mean, workspace, stream) -> (y, rstd, mean)
PyObject *group_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<15>(n, [&]() -> PyObject * {
    const at::Tensor &x = lead(a[0], "x");
    const norm_dtype_t code = dtype_code(x);
    const c10::Device dev = x.device();
    const at::ScalarType dt = x.scalar_type();
    const Samples d(x);
    const at::Tensor &gamma = tensor(a[1], "gamma"), &beta = tensor(a[2], "beta", true);
    check(gamma, "gamma", dt, {d.C}, dev);
    check(beta, "beta", dt, {d.C}, dev);
    const int64_t groups = integer(a[3]);
    if (groups < 1 || groups > d.C) return PyLong_FromLong(NORM_ERR_SHAPE);
    const float eps = static_cast<float>(number(a[4]));
    const norm_act_t act = static_cast<norm_act_t>(code_of(a[5]));
    const Rng rng(a + 6, dev);
    const StreamArg stream(a[14]);
    Output y(a[10], "y", dt, x.sizes(), dev);
    Output rstd(a[11], "rstd", at::kFloat, {d.B, groups}, dev);
    Output mean(a[12], "mean", at::kFloat, {d.B, groups}, dev);
    Workspace ws(a[13], dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      for (Output *o : {&y, &rstd, &mean}) o->make();
      st = ws.make([&](size_t *b) {
        return norm_group_fwd_workspace_bytes(d.B, d.S, d.C, groups, code, b);
      });
      if (st == NORM_OK)
        st = norm_group_fwd(ptr(x), ptr(gamma), ptr(beta), d.B, d.S, d.C, groups, eps, act, code,
                            rng.p, rng.seed, rng.offset, rng.dev_word, ptr(y.t),
                            static_cast<float *>(ptr(rstd.t)), static_cast<float *>(ptr(mean.t)),
                            ptr(ws.t), ws.bytes, on.s);
    }
    return result(st, {y.t, rstd.t, mean.t});
  });
}

// (dy, x, gamma, beta, rstd, mean, groups, act, p, seed, offset, offset_dev,
// dx, dgamma, dbeta, want_dbeta, workspace, stream) -> (dx, dgamma, dbeta)
PyObject *group_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<18>(n, [&]() -> PyObject * {
    const at::Tensor &x = lead(a[1], "x");
    const norm_dtype_t code = dtype_code(x);
    const c10::Device dev = x.device();
    const at::ScalarType dt = x.scalar_type(), f32 = at::kFloat;
    const Samples d(x);
    const at::Tensor &dy = tensor(a[0], "dy"), &gamma = tensor(a[2], "gamma"),
                     &beta = tensor(a[3], "beta", true), &rstd = tensor(a[4], "rstd"),
                     &mean = tensor(a[5], "mean");
    const int64_t groups = integer(a[6]);
    if (groups < 1 || groups > d.C) return PyLong_FromLong(NORM_ERR_SHAPE);
    check(dy, "dy", dt, x.sizes(), dev);
    check(gamma, "gamma", dt, {d.C}, dev);
    check(beta, "beta", dt, {d.C}, dev);
    check(rstd, "rstd", f32, {d.B, groups}, dev);
    check(mean, "mean", f32, {d.B, groups}, dev);
    const norm_act_t act = static_cast<norm_act_t>(code_of(a[7]));
    const Rng rng(a + 8, dev);
    const StreamArg stream(a[17]);
    Output dx(a[12], "dx", dt, x.sizes(), dev);
    Output dg(a[13], "dgamma", f32, {d.C}, dev);
    Output db(a[14], "dbeta", f32, {d.C}, dev, truth(a[15]));
    Workspace ws(a[16], dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      for (Output *o : {&dx, &dg, &db}) o->make();
      st = ws.make([&](size_t *b) {
        return norm_group_bwd_workspace_bytes(d.B, d.S, d.C, groups, code, b);
      });
      if (st == NORM_OK)
        st = norm_group_bwd(ptr(dy), ptr(x), ptr(gamma), ptr(beta),
                            static_cast<const float *>(ptr(rstd)),
                            static_cast<const float *>(ptr(mean)), d.B, d.S, d.C, groups, act, code,
                            rng.p, rng.seed, rng.offset, rng.dev_word, ptr(dx.t),
                            static_cast<float *>(ptr(dg.t)), static_cast<float *>(ptr(db.t)),
                            ptr(ws.t), ws.bytes, on.s);
    }
    return result(st, {dx.t, dg.t, db.t});
  });
}

template <typename F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"dropout", as_method(dropout), METH_FASTCALL, nullptr},
    {"dropout_add_fwd", as_method(dropout_add_fwd), METH_FASTCALL, nullptr},
    {"dropout_add_bwd", as_method(dropout_add_bwd), METH_FASTCALL, nullptr},
    {"group_fwd", as_method(group_fwd), METH_FASTCALL, nullptr},
    {"group_bwd", as_method(group_bwd), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gbnorm_torch", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gbnorm_torch() { return PyModule_Create(&module); }
