// torch_binding.cpp -- the tensor side of the dropout, group-normalisation and
// head-rotation and linear-layer entry points: argument checks, output and workspace allocation, the
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

// A tensor of heads [..., H, D] whose leading dimensions are evenly strided
// tokens, as the library's view of it.
struct Heads {
  norm_heads_t v = {nullptr, 0, 0};
  int64_t T = 0, H = 0, D = 0;

  Heads() = default;
  Heads(const at::Tensor &t, const char *name) {
    if (t.dim() < 3) fail(std::string(name) + " must be [..., heads, head size]");
    const int64_t n = t.dim();
    D = t.size(n - 1);
    H = t.size(n - 2);
    if (D > 1 && t.stride(n - 1) != 1)
      fail(std::string(name) + " must be contiguous in its last dimension");
    T = 1;
    bool any = false;
    for (int64_t i = n - 3; i >= 0; --i) {
      if (t.size(i) == 1) continue;
      if (!any)
        v.token_stride = t.stride(i);
      else if (t.stride(i) != v.token_stride * T)
        fail(std::string(name) + " must have evenly strided tokens in its leading dimensions");
      any = true;
      T *= t.size(i);
    }
    v.head_stride = H > 1 ? t.stride(n - 2) : 0;
    v.data = t.numel() ? t.data_ptr() : nullptr;
  }
};

void check_like(const at::Tensor &t, const char *name, at::ScalarType dt, c10::IntArrayRef shape,
                c10::Device dev) {
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  if (t.device() != dev)
    fail(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (t.scalar_type() != dt)
    fail(std::string(name) + " must be " + c10::toString(dt) + ", got " +
         c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    fail(std::string(name) + " has shape " + show(t.sizes()) + ", expected " + show(shape));
}

// An output of heads: the given tensor (any strides that Heads takes) or a new
// contiguous one.
struct HeadsOut {
  at::Tensor t;
  at::ScalarType dt;
  c10::DimVector shape;
  const char *name;

  HeadsOut(PyObject *o, const char *what, const at::Tensor &like, c10::Device dev)
      : dt(like.scalar_type()), shape(like.sizes().begin(), like.sizes().end()), name(what) {
    if (o == Py_None) return;
    t = tensor(o, name);
    check_like(t, name, dt, shape, dev);
    Heads checked(t, name);
  }
  Heads make() {
    if (!t.defined()) {
      const int64_t bytes =
          static_cast<int64_t>(c10::elementSize(dt)) * c10::multiply_integers(shape);
      t = device_tensor((bytes + 511) & ~int64_t(511), dt, shape);
    }
    return Heads(t, name);
  }
};

// pos, inv_freq and the sections of a call.
struct Rotation {
  const void *pos;
  const double *inv_freq;
  int pos_bits, axes = 1;
  int64_t pos_stride = 0, rd;
  uint8_t axis[128] = {};

  Rotation(PyObject *p, PyObject *f, PyObject *sections, const at::Tensor &q, c10::Device dev) {
    const at::Tensor &freq = tensor(f, "inv_freq"), &ps = tensor(p, "pos");
    if (freq.dim() != 1 || freq.numel() > 128) fail("inv_freq must be [pairs], 128 at most");
    check(freq, "inv_freq", at::kDouble, freq.sizes(), dev);
    rd = 2 * freq.numel();
    inv_freq = static_cast<const double *>(freq.data_ptr());
    if (sections != Py_None) {
      PyObject *seq = PySequence_Fast(sections, "sections must be a sequence of pair counts");
      if (!seq) throw PyFail{};
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
      int64_t at = 0;
      bool good = n >= 1 && n <= 4;
      for (Py_ssize_t i = 0; good && i < n; ++i) {
        const long long c = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
        if (PyErr_Occurred()) {
          Py_DECREF(seq);
          throw PyFail{};
        }
        good = c >= 0 && c <= rd / 2 - at;
        for (long long j = 0; good && j < c; ++j) axis[at++] = static_cast<uint8_t>(i);
      }
      Py_DECREF(seq);
      if (!good || at != rd / 2)
        fail("sections must be 1 to 4 pair counts that add up to the length of inv_freq");
      axes = static_cast<int>(n);
    }
    const c10::IntArrayRef lead = q.sizes().slice(0, q.dim() - 2);
    if (!ps.is_cuda() || ps.device() != dev) fail("pos must be on " + dev.str());
    if (ps.scalar_type() != at::kInt && ps.scalar_type() != at::kLong)
      fail("pos must be int32 or int64");
    const bool rows = axes > 1 || ps.dim() == q.dim() - 1;
    c10::DimVector want;
    if (rows) want.push_back(axes);
    want.insert(want.end(), lead.begin(), lead.end());
    if (ps.sizes() != c10::IntArrayRef(want))
      fail("pos has shape " + show(ps.sizes()) + ", expected " + show(want));
    int64_t step = 1;
    for (int64_t i = ps.dim() - 1; i >= (rows ? 1 : 0); --i) {
      if (ps.size(i) != 1 && ps.stride(i) != step)
        fail("pos must be contiguous in its token dimensions");
      step *= ps.size(i);
    }
    if (axes > 1) pos_stride = ps.stride(0);
    pos = ps.numel() ? ps.data_ptr() : nullptr;
    pos_bits = ps.scalar_type() == at::kInt ? 32 : 64;
  }
};

// The head tensor `o`, or an undefined one for None.
const at::Tensor &heads_arg(PyObject *o, const char *name, bool optional, at::ScalarType dt,
                            c10::Device dev) {
  const at::Tensor &t = tensor(o, name, optional);
  if (!t.defined()) return t;
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  if (t.device() != dev)
    fail(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (t.scalar_type() != dt)
    fail(std::string(name) + " must be " + c10::toString(dt) + ", got " +
         c10::toString(t.scalar_type()));
  return t;
}

// Keys have the tokens and the head size of the queries.
void check_keys(const at::Tensor &q, const at::Tensor &k, const char *name) {
  if (k.dim() != q.dim() || k.size(-1) != q.size(-1) ||
      k.sizes().slice(0, k.dim() - 2) != q.sizes().slice(0, q.dim() - 2))
    fail(std::string(name) + " has shape " + show(k.sizes()) +
         ", expected that of the queries but for the heads, " + show(q.sizes()));
}

// (q, k, pos, inv_freq, gamma_q, gamma_k, beta_q, beta_k, eps, mode, sections,
// interleaved, yq, yk, stream) -> (yq, yk)
PyObject *rope_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<15>(n, [&]() -> PyObject * {
    const at::Tensor &q = tensor(a[0], "q");
    if (!q.is_cuda()) fail("q must be a CUDA tensor");
    const norm_dtype_t code = dtype_code(q);
    const c10::Device dev = q.device();
    const at::ScalarType dt = q.scalar_type();
    const at::Tensor &k = heads_arg(a[1], "k", true, dt, dev);
    const Heads hq(q, "q");
    Heads hk;
    if (k.defined()) {
      hk = Heads(k, "k");
      check_keys(q, k, "k");
    }
    const Rotation rot(a[2], a[3], a[10], q, dev);
    const at::Tensor *par[4];
    static const char *const names[4] = {"gamma_q", "gamma_k", "beta_q", "beta_k"};
    for (int i = 0; i < 4; ++i) {
      par[i] = &tensor(a[4 + i], names[i], true);
      check(*par[i], names[i], dt, {hq.D}, dev);
    }
    const float eps = static_cast<float>(number(a[8]));
    const norm_mode_t mode = static_cast<norm_mode_t>(code_of(a[9]));
    const bool inter = truth(a[11]);
    const StreamArg stream(a[14]);
    HeadsOut yq(a[12], "yq", q, dev), yk(k.defined() ? a[13] : Py_None, "yk", k.defined() ? k : q, dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      const Heads oq = yq.make();
      const Heads ok = k.defined() ? yk.make() : Heads();
      st = norm_rope_fwd(&hq.v, &hk.v, hq.T, hq.H, hk.H, hq.D, rot.rd, rot.pos, rot.pos_bits,
                         rot.pos_stride, rot.inv_freq, rot.axis, rot.axes, inter, ptr(*par[0]),
                         ptr(*par[1]), ptr(*par[2]), ptr(*par[3]), eps, mode, code, &oq.v, &ok.v,
                         on.s);
    }
    return result(st, {yq.t, yk.t});
  });
}

// (dyq, dyk, q, k, pos, inv_freq, gamma_q, gamma_k, eps, mode, sections,
// interleaved, dq, dk, dgamma_q, dgamma_k, dbeta_q, dbeta_k, want_dbeta,
// workspace, stream) -> (dq, dk, dgamma_q, dgamma_k, dbeta_q, dbeta_k)
PyObject *rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<21>(n, [&]() -> PyObject * {
    const at::Tensor &dyq = tensor(a[0], "dyq");
    if (!dyq.is_cuda()) fail("dyq must be a CUDA tensor");
    const norm_dtype_t code = dtype_code(dyq);
    const c10::Device dev = dyq.device();
    const at::ScalarType dt = dyq.scalar_type(), f32 = at::kFloat;
    const at::Tensor &dyk = heads_arg(a[1], "dyk", true, dt, dev);
    const bool keys = dyk.defined();
    const at::Tensor &gq = tensor(a[6], "gamma_q", true), &gk = tensor(a[7], "gamma_k", true);
    const bool norm = gq.defined();
    const at::Tensor &q = heads_arg(a[2], "q", !norm, dt, dev),
                     &k = heads_arg(a[3], "k", !norm || !keys, dt, dev);
    const Heads hdq(dyq, "dyq");
    Heads hdk, hq, hk;
    if (keys) {
      hdk = Heads(dyk, "dyk");
      check_keys(dyq, dyk, "dyk");
    }
    if (q.defined()) {
      check_like(q, "q", dt, dyq.sizes(), dev);
      hq = Heads(q, "q");
    }
    if (k.defined()) {
      if (!keys) fail("k is given without dyk");
      check_like(k, "k", dt, dyk.sizes(), dev);
      hk = Heads(k, "k");
    }
    const Rotation rot(a[4], a[5], a[10], dyq, dev);
    check(gq, "gamma_q", dt, {hdq.D}, dev);
    check(gk, "gamma_k", dt, {hdq.D}, dev);
    const float eps = static_cast<float>(number(a[8]));
    const norm_mode_t mode = static_cast<norm_mode_t>(code_of(a[9]));
    const bool inter = truth(a[11]);
    const bool beta = norm && mode == NORM_LAYER && truth(a[18]);
    const StreamArg stream(a[20]);
    HeadsOut dq(a[12], "dq", dyq, dev), dk(keys ? a[13] : Py_None, "dk", keys ? dyk : dyq, dev);
    Output dgq(a[14], "dgamma_q", f32, {hdq.D}, dev, norm);
    Output dgk(a[15], "dgamma_k", f32, {hdq.D}, dev, norm && keys);
    Output dbq(a[16], "dbeta_q", f32, {hdq.D}, dev, beta);
    Output dbk(a[17], "dbeta_k", f32, {hdq.D}, dev, beta && keys);
    Workspace ws(a[19], dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      const Heads oq = dq.make();
      const Heads ok = keys ? dk.make() : Heads();
      for (Output *o : {&dgq, &dgk, &dbq, &dbk}) o->make();
      st = ws.make([&](size_t *b) {
        return norm_rope_bwd_workspace_bytes(hdq.T, hdq.H, hdk.H, hdq.D, norm, mode, b);
      });
      if (st == NORM_OK)
        st = norm_rope_bwd(&hdq.v, &hdk.v, &hq.v, &hk.v, hdq.T, hdq.H, hdk.H, hdq.D, rot.rd,
                           rot.pos, rot.pos_bits, rot.pos_stride, rot.inv_freq, rot.axis, rot.axes,
                           inter, ptr(gq), ptr(gk), eps, mode, code, &oq.v, &ok.v,
                           static_cast<float *>(ptr(dgq.t)), static_cast<float *>(ptr(dgk.t)),
                           static_cast<float *>(ptr(dbq.t)), static_cast<float *>(ptr(dbk.t)),
                           ptr(ws.t), ws.bytes, on.s);
    }
    return result(st, {dq.t, dk.t, dgq.t, dgk.t, dbq.t, dbk.t});
  });
}

// A tensor of rows [..., C], contiguous in the last dimension, whose leading
// dimensions are evenly strided rows.
struct RowsView {
  void *p = nullptr;
  int64_t ld = 0, M = 0, C = 0;

  RowsView() = default;
  RowsView(const at::Tensor &t, const char *name) {
    if (!t.defined()) return;
    const int64_t n = t.dim();
    if (n < 1) fail(std::string(name) + " must have at least one dimension");
    C = t.size(n - 1);
    if (C > 1 && t.stride(n - 1) != 1)
      fail(std::string(name) + " must be contiguous in its last dimension");
    M = 1;
    ld = C;
    bool any = false;
    for (int64_t i = n - 2; i >= 0; --i) {
      if (t.size(i) == 1) continue;
      if (!any)
        ld = t.stride(i);
      else if (t.stride(i) != ld * M)
        fail(std::string(name) + " must have evenly strided rows in its leading dimensions");
      any = true;
      M *= t.size(i);
    }
    p = t.numel() ? t.data_ptr() : nullptr;
  }
};

// An output of rows: the given tensor (any strides that RowsView takes) or a new
// contiguous one.
struct RowsOut {
  at::Tensor t;
  at::ScalarType dt;
  c10::DimVector shape;
  const char *name;
  bool wanted;

  RowsOut(PyObject *o, const char *what, at::ScalarType type, c10::IntArrayRef sizes,
          c10::Device dev, bool want = true)
      : dt(type), shape(sizes.begin(), sizes.end()), name(what), wanted(want) {
    if (o == Py_None) return;
    t = tensor(o, name);
    check_like(t, name, dt, sizes, dev);
    RowsView checked(t, name);
  }
  RowsView make() {
    if (!t.defined() && wanted) {
      const int64_t bytes =
          static_cast<int64_t>(c10::elementSize(dt)) * c10::multiply_integers(shape);
      t = device_tensor((bytes + 511) & ~int64_t(511), dt, shape);
    }
    return RowsView(t, name);
  }
};

norm_dtype_t half_code(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() == at::kBFloat16) return NORM_BF16;
  if (t.scalar_type() == at::kHalf) return NORM_FP16;
  fail(std::string(name) + " must be bfloat16 or float16, got " + c10::toString(t.scalar_type()));
}

c10::DimVector with_last(const at::Tensor &t, int64_t last) {
  c10::DimVector d(t.sizes().begin(), t.sizes().end());
  d.back() = last;
  return d;
}

// The operands of a forward call.
struct LinearIn {
  const at::Tensor &x, &w;
  RowsView vx, vw;
  LinearIn(PyObject *ox, PyObject *ow) : x(tensor(ox, "x")), w(tensor(ow, "w")) {
    half_code(x, "x");
    if (w.dim() != 2) fail("w must be [N, K]");
    vx = RowsView(x, "x");
    check_like(w, "w", x.scalar_type(), {w.size(0), vx.C}, x.device());
    vw = RowsView(w, "w");
  }
};

// (x, w, bias, r, act, want_z, y, z, workspace, stream) -> (y, z)
PyObject *linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<10>(n, [&]() -> PyObject * {
    const LinearIn in(a[0], a[1]);
    const norm_dtype_t code = half_code(in.x, "x");
    const c10::Device dev = in.x.device();
    const at::ScalarType dt = in.x.scalar_type();
    const int64_t N = in.w.size(0);
    const c10::DimVector shape = with_last(in.x, N);
    const at::Tensor &bias = tensor(a[2], "bias", true), &r = tensor(a[3], "r", true);
    check(bias, "bias", dt, {N}, dev);
    if (r.defined()) check_like(r, "r", dt, shape, dev);
    const RowsView vr(r, "r");
    const norm_act_t act = static_cast<norm_act_t>(code_of(a[4]));
    const StreamArg stream(a[9]);
    RowsOut y(a[6], "y", dt, shape, dev), z(a[7], "z", dt, shape, dev, truth(a[5]));
    Workspace ws(a[8], dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      const RowsView vy = y.make(), vz = z.make();
      st = ws.make([&](size_t *b) {
        return norm_linear_fwd_workspace_bytes(in.vx.p, in.vx.ld, in.vw.p, in.vw.ld, in.vx.M,
                                               in.vx.C, N, b);
      });
      if (st == NORM_OK)
        st = norm_linear_fwd(in.vx.p, in.vx.ld, in.vw.p, in.vw.ld, ptr(bias), vr.p, vr.ld, in.vx.M,
                             in.vx.C, N, act, code, vy.p, vy.ld, vz.p, vz.ld, ptr(ws.t), ws.bytes,
                             on.s);
    }
    return result(st, {y.t, z.t});
  });
}

// What a backward call reads, and which outputs it wants.
struct LinearGrad {
  const at::Tensor &dy, &x, &w, &z;
  RowsView vdy, vx, vw, vz;
  int64_t M, K, N;
  norm_act_t act;
  bool dx, dw, dbias;
  c10::DimVector xshape;

  // (dy, x, w, z, act, want_dx, want_dw, want_dbias)
  explicit LinearGrad(PyObject *const *a)
      : dy(tensor(a[0], "dy")), x(tensor(a[1], "x", true)), w(tensor(a[2], "w", true)),
        z(tensor(a[3], "z", true)), act(static_cast<norm_act_t>(code_of(a[4]))), dx(truth(a[5])),
        dw(truth(a[6])), dbias(truth(a[7])) {
    half_code(dy, "dy");
    const c10::Device dev = dy.device();
    const at::ScalarType dt = dy.scalar_type();
    vdy = RowsView(dy, "dy");
    M = vdy.M;
    N = vdy.C;
    if (!x.defined() && dw) fail("x must be given for dw");
    if (!w.defined() && dx) fail("w must be given for dx");
    if (w.defined() && (w.dim() != 2 || w.size(0) != N))
      fail("w has shape " + show(w.sizes()) + ", expected " + std::to_string(N) + " rows");
    K = w.defined() ? w.size(1) : x.defined() ? x.size(-1) : 1;
    xshape = with_last(dy, K);
    if (w.defined()) check_like(w, "w", dt, {N, K}, dev);
    if (x.defined()) check_like(x, "x", dt, xshape, dev);
    if (z.defined()) check_like(z, "z", dt, dy.sizes(), dev);
    vx = RowsView(x, "x");
    vw = RowsView(w, "w");
    vz = RowsView(z, "z");
  }
  norm_status_t bytes(size_t *b) const {
    return norm_linear_bwd_workspace_bytes(vdy.p, vdy.ld, vx.p, vx.ld, vw.p, vw.ld, vz.p, vz.ld, M,
                                           K, N, act, dx, dw, dbias, b);
  }
};

// (dy, x, w, z, act, want_dx, want_dw, want_dbias, dx, dw, dbias, workspace,
// stream) -> (dx, dw, dbias)
PyObject *linear_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<13>(n, [&]() -> PyObject * {
    const LinearGrad in(a);
    const norm_dtype_t code = half_code(in.dy, "dy");
    const c10::Device dev = in.dy.device();
    const at::ScalarType dt = in.dy.scalar_type();
    const StreamArg stream(a[12]);
    RowsOut dx(in.dx ? a[8] : Py_None, "dx", dt, in.xshape, dev, in.dx);
    RowsOut dw(in.dw ? a[9] : Py_None, "dw", dt, {in.N, in.K}, dev, in.dw);
    Output db(in.dbias ? a[10] : Py_None, "dbias", at::kFloat, {in.N}, dev, in.dbias);
    Workspace ws(a[11], dev);
    norm_status_t st;
    {
      const Unlocked unlocked;
      const StreamScope on(stream, dev);
      const RowsView vdx = dx.make(), vdw = dw.make();
      db.make();
      st = ws.make([&](size_t *b) { return in.bytes(b); });
      if (st == NORM_OK)
        st = norm_linear_bwd(in.vdy.p, in.vdy.ld, in.vx.p, in.vx.ld, in.vw.p, in.vw.ld, in.vz.p,
                             in.vz.ld, in.M, in.K, in.N, in.act, code, vdx.p, vdx.ld, vdw.p, vdw.ld,
                             static_cast<float *>(ptr(db.t)), ptr(ws.t), ws.bytes, on.s);
    }
    return result(st, {dx.t, dw.t, db.t});
  });
}

// Workspace bytes, or minus the status.
PyObject *linear_fwd_workspace(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<2>(n, [&]() -> PyObject * {
    const LinearIn in(a[0], a[1]);
    size_t b = 0;
    const norm_status_t st = norm_linear_fwd_workspace_bytes(
        in.vx.p, in.vx.ld, in.vw.p, in.vw.ld, in.vx.M, in.vx.C, in.w.size(0), &b);
    return PyLong_FromLongLong(st == NORM_OK ? static_cast<long long>(b) : -st);
  });
}

PyObject *linear_bwd_workspace(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<8>(n, [&]() -> PyObject * {
    const LinearGrad in(a);
    const c10::cuda::CUDAGuard on(in.dy.device());
    size_t b = 0;
    const norm_status_t st = in.bytes(&b);
    return PyLong_FromLongLong(st == NORM_OK ? static_cast<long long>(b) : -st);
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
    {"linear_fwd", as_method(linear_fwd), METH_FASTCALL, nullptr},
    {"linear_bwd", as_method(linear_bwd), METH_FASTCALL, nullptr},
    {"linear_fwd_workspace", as_method(linear_fwd_workspace), METH_FASTCALL, nullptr},
    {"linear_bwd_workspace", as_method(linear_bwd_workspace), METH_FASTCALL, nullptr},
    {"rope_fwd", as_method(rope_fwd), METH_FASTCALL, nullptr},
    {"rope_bwd", as_method(rope_bwd), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gbnorm_torch", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gbnorm_torch() { return PyModule_Create(&module); }
