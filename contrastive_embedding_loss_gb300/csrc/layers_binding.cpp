// layers_binding.cpp -- the Python side of include/uf_layers.h: checks of the tensor arguments,
// outputs and scratch from torch's allocator, and one C call on the current stream.
//
// A call of a few microseconds on the GPU is bound by the host's way to it; in Python that way
// took 15 us, here it takes a third.  layers.py documents the functions and passes their
// arguments on in order; the C entry points are bound by address (bind), so this module does not
// link the CUDA library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <limits>
#include <optional>
#include <string>
#include <type_traits>
#include <vector>

#include "../../include/uf_layers.h"

namespace {

using at::Tensor;

// The C entry points.
struct Api {
  decltype(&uf_rmsnorm_fwd) rmsnorm_fwd;
  decltype(&uf_rmsnorm_bwd_workspace) rmsnorm_bwd_workspace;
  decltype(&uf_rmsnorm_bwd) rmsnorm_bwd;
  decltype(&uf_linear_fwd_workspace) linear_fwd_workspace;
  decltype(&uf_linear_fwd) linear_fwd;
  decltype(&uf_linear_bwd_workspace) linear_bwd_workspace;
  decltype(&uf_linear_bwd) linear_bwd;
  decltype(&uf_gated_fwd_workspace) gated_fwd_workspace;
  decltype(&uf_gated_fwd) gated_fwd;
  decltype(&uf_gated_bwd_workspace) gated_bwd_workspace;
  decltype(&uf_gated_bwd) gated_bwd;
  decltype(&uf_adamw_step) adamw_step;
} api;
PyObject* uf_error = nullptr;  // binding.UfError(status, what)

// A Python exception that is already set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised{};
}

const char* name_of(at::ScalarType t) {
  return t == at::kBFloat16 ? "bfloat16" : t == at::kFloat ? "float32" : t == at::kFloat8_e4m3fn ? "float8_e4m3fn" : "uint8";
}
int type_of(at::ScalarType t) { return t == at::kBFloat16 ? UF_BF16 : t == at::kFloat ? UF_F32 : UF_E4M3; }

struct Types {
  at::ScalarType a, b;  // b == a: one type
  bool has(at::ScalarType t) const { return t == a || t == b; }
  std::string names() const { return a == b ? name_of(a) : std::string(name_of(a)) + " or " + name_of(b); }
};
constexpr Types kBf16{at::kBFloat16, at::kBFloat16}, kF32{at::kFloat, at::kFloat}, kFloats{at::kBFloat16, at::kFloat},
    kOperands{at::kBFloat16, at::kFloat8_e4m3fn};

const Tensor& tensor(const char* name, PyObject* o, Types types) {
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    if (types.has(t.scalar_type()) && t.is_cuda()) return t;
  }
  raise(PyExc_TypeError, "%s must be a CUDA tensor of %s", name, types.names().c_str());
}

// A 2-D CUDA tensor with contiguous rows; rows, cols: -1 for any.
const Tensor& matrix(const char* name, PyObject* o, Types types, const c10::Device* dev = nullptr, int64_t rows = -1,
                     int64_t cols = -1) {
  const Tensor& t = tensor(name, o, types);
  if (dev && t.device() != *dev) raise(PyExc_ValueError, "%s must be on %s, not %s", name, dev->str().c_str(), t.device().str().c_str());
  if (t.dim() != 2) raise(PyExc_ValueError, "%s must be 2-D, not %d-D", name, static_cast<int>(t.dim()));
  if ((rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols))
    raise(PyExc_ValueError, "%s must be (%s, %lld), not (%lld, %lld)", name, rows < 0 ? "any" : std::to_string(rows).c_str(),
          static_cast<long long>(cols < 0 ? t.size(1) : cols), static_cast<long long>(t.size(0)),
          static_cast<long long>(t.size(1)));
  if (t.stride(1) != 1 && t.size(1) > 1 && t.size(0) > 0)
    raise(PyExc_ValueError, "%s's rows must be contiguous (a stride of 1 within a row)", name);
  return t;
}
const Tensor& vector(const char* name, PyObject* o, Types types, const c10::Device& dev, int64_t n) {
  const Tensor& t = tensor(name, o, types);
  if (t.device() != dev || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    raise(PyExc_ValueError, "%s must be a contiguous vector of %lld on %s", name, static_cast<long long>(n), dev.str().c_str());
  return t;
}

// A matrix's width, an int in the C entry points.
int width_of(const char* name, int64_t n) {
  if (n > std::numeric_limits<int>::max())
    raise(PyExc_ValueError, "%s may be at most %d, not %lld", name, std::numeric_limits<int>::max(), static_cast<long long>(n));
  return static_cast<int>(n);
}

// Row stride in elements (a single row has none of its own).
int64_t ld(const Tensor& t) { return t.size(0) != 1 ? t.stride(0) : t.size(1); }

bool given(PyObject* o) { return o != Py_None; }

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// (past the dispatcher: three outputs of a norm cost a microsecond more through it)
Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const c10::Device& dev) {
  return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}

// The caller's scratch or one of the needed size, and the caller's status word.
struct Scratch {
  Tensor own;
  void* ptr = nullptr;
  size_t bytes = 0;
  int* status = nullptr;
  Scratch(size_t need, const c10::Device& dev, PyObject* workspace, PyObject* device_status) {
    if (given(workspace)) {
      if (!THPVariable_Check(workspace)) raise(PyExc_TypeError, "workspace must be a contiguous uint8 tensor on the inputs' device");
      const Tensor& w = THPVariable_Unpack(workspace);
      if (w.scalar_type() != at::kByte || w.device() != dev || !w.is_contiguous())
        raise(PyExc_TypeError, "workspace must be a contiguous uint8 tensor on the inputs' device");
      ptr = w.data_ptr();
      bytes = static_cast<size_t>(w.numel());
    } else if (need) {
      own = empty({static_cast<int64_t>(need)}, at::kByte, dev);
      ptr = own.data_ptr();
      bytes = need;
    }
    if (given(device_status)) {
      const bool ok = THPVariable_Check(device_status) && THPVariable_Unpack(device_status).scalar_type() == at::kInt &&
                      THPVariable_Unpack(device_status).device() == dev && THPVariable_Unpack(device_status).numel() >= 1;
      if (!ok) raise(PyExc_TypeError, "device_status must be an int32 tensor (one element) on the inputs' device");
      status = static_cast<int*>(THPVariable_Unpack(device_status).data_ptr());
    }
  }
};

// The tensors' device made current for a call, and the stream to call on: the caller's (a
// torch.cuda.Stream), made current too, so that outputs and scratch are allocated on the stream
// that uses them and scratch that is freed on return goes back to it; or the current one.  What the
// caller hands to a call on another stream than its own is marked as used there (uses), so that
// memory that the caller frees after the call is not given away before the kernels have run.
struct On {
  c10::cuda::OptionalCUDAStreamGuard stream_guard;
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  std::optional<c10::cuda::CUDAStream> other;  // the stream, if it is not the current one
  On(const c10::Device& dev, PyObject* s) {
    if (given(s)) {
      const auto part = [&](const char* name) {
        PyObject* o = PyObject_GetAttrString(s, name);
        if (!o) throw Raised{};
        const int64_t v = PyLong_AsLongLong(o);
        Py_DECREF(o);
        if (v == -1 && PyErr_Occurred()) throw Raised{};
        return v;
      };
      const auto cs = c10::cuda::CUDAStream::unpack3(part("stream_id"), static_cast<c10::DeviceIndex>(part("device_index")),
                                                     static_cast<c10::DeviceType>(part("device_type")));
      if (cs.device() != dev) raise(PyExc_ValueError, "stream must be on %s, not %s", dev.str().c_str(), cs.device().str().c_str());
      if (cs != c10::cuda::getCurrentCUDAStream(dev.index())) other = cs;
      stream_guard.reset_stream(cs);
      stream = cs.stream();
      return;
    }
    if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
    stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  }
  // The tensors among a call's arguments, and those of its lists.
  void uses(PyObject* const* args, int n) const {
    if (!other) return;
    for (int i = 0; i < n; ++i) {
      if (THPVariable_Check(args[i])) {
        const Tensor& t = THPVariable_Unpack(args[i]);
        if (t.is_cuda()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *other);
      } else if (PyList_Check(args[i])) {
        for (Py_ssize_t k = 0; k < PyList_GET_SIZE(args[i]); ++k) {
          PyObject* item = PyList_GET_ITEM(args[i], k);
          uses(&item, 1);
        }
      } else if (PyTuple_Check(args[i])) {
        for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(args[i]); ++k) {
          PyObject* item = PyTuple_GET_ITEM(args[i], k);
          uses(&item, 1);
        }
      }
    }
  }
};

void check(uf_status_t st, const char* what) {
  if (st == UF_OK) return;
  PyObject* e = PyObject_CallFunction(uf_error, "is", static_cast<int>(st), what);
  if (e) {
    PyErr_SetObject(uf_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

struct Result {
  PyObject* dict = PyDict_New();
  void put(const char* key, const Tensor& t) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o || PyDict_SetItemString(dict, key, o) != 0) {
      Py_XDECREF(o);
      Py_DECREF(dict);
      throw Raised{};
    }
    Py_DECREF(o);
  }
};

void* opt(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// ------------------------------------------------------------------------------ functions
// Arguments come by position, as layers.py lists them.

// x, weight, residual, eps, e4m3, stream
PyObject* rmsnorm_fwd(PyObject* const* a) {
  const bool res = given(a[2]), e4m3 = truth(a[4]);
  const Tensor& x = matrix("x", a[0], res ? kBf16 : kFloats);
  const int64_t rows = x.size(0);
  const int width = width_of("x's width", x.size(1));
  const c10::Device dev = x.device();
  const Tensor& w = vector("weight", a[1], kFloats, dev, width);
  const Tensor none;
  const Tensor& r = res ? matrix("residual", a[2], kFloats, &dev, rows, width) : none;
  const On on(dev, a[5]);
  const Tensor y = empty({rows, width}, e4m3 ? at::kFloat8_e4m3fn : at::kBFloat16, dev);
  const Tensor rstd = empty({rows}, at::kFloat, dev);
  Tensor s, scale;
  if (res) s = empty({rows, width}, r.scalar_type(), dev);
  if (e4m3) scale = empty({rows}, at::kFloat, dev);
  check(api.rmsnorm_fwd(x.data_ptr(), ld(x), type_of(x.scalar_type()), opt(r), res ? ld(r) : 0,
                        res ? type_of(r.scalar_type()) : 0, w.data_ptr(), type_of(w.scalar_type()), rows,
                        width, static_cast<float>(number(a[3])), y.data_ptr(), width,
                        e4m3 ? UF_E4M3 : UF_BF16, static_cast<float*>(opt(scale)), opt(s), width,
                        static_cast<float*>(rstd.data_ptr()), on.stream),
        "uf_rmsnorm_fwd");
  on.uses(a, 6);
  Result out;
  out.put("y", y);
  out.put("rstd", rstd);
  if (res) out.put("stream", s);
  if (e4m3) out.put("scale", scale);
  return out.dict;
}

// dy, s, weight, rstd, d_stream, weight_grad, workspace, stream
PyObject* rmsnorm_bwd(PyObject* const* a) {
  const Tensor& s = matrix("s", a[1], kFloats);
  const int64_t rows = s.size(0);
  const int width = width_of("s's width", s.size(1));
  const c10::Device dev = s.device();
  const Tensor& dy = matrix("dy", a[0], kFloats, &dev, rows, width);
  const Tensor& w = vector("weight", a[2], kFloats, dev, width);
  const Tensor& rstd = vector("rstd", a[3], kF32, dev, rows);
  const bool carry = given(a[4]), grad = truth(a[5]);
  const Tensor none;
  const Tensor& ds = carry ? matrix("d_stream", a[4], Types{s.scalar_type(), s.scalar_type()}, &dev, rows, width) : none;
  const On on(dev, a[7]);
  const Tensor dx = empty({rows, width}, s.scalar_type(), dev);
  Tensor dw;
  if (grad) dw = empty({width}, at::kFloat, dev);
  const Scratch ws(grad ? api.rmsnorm_bwd_workspace(rows, width) : 0, dev, a[6], Py_None);
  check(api.rmsnorm_bwd(dy.data_ptr(), ld(dy), type_of(dy.scalar_type()), s.data_ptr(), ld(s), type_of(s.scalar_type()),
                        w.data_ptr(), type_of(w.scalar_type()), static_cast<const float*>(rstd.data_ptr()), opt(ds),
                        carry ? ld(ds) : 0, rows, width, dx.data_ptr(), width, static_cast<float*>(opt(dw)),
                        ws.ptr, ws.bytes, on.stream),
        "uf_rmsnorm_bwd");
  on.uses(a, 8);
  Result out;
  out.put("dx", dx);
  if (grad) out.put("dweight", dw);
  return out.dict;
}

// A linear weight: outer x inner of x's type.
const Tensor& weight_of(PyObject* o, const Tensor& x) {
  const c10::Device dev = x.device();
  const Tensor& w = matrix("W", o, Types{x.scalar_type(), x.scalar_type()}, &dev);
  if (w.size(1) != x.size(1))
    raise(PyExc_ValueError, "W must be outer x %lld, not (%lld, %lld)", static_cast<long long>(x.size(1)),
          static_cast<long long>(w.size(0)), static_cast<long long>(w.size(1)));
  return w;
}

// x, W, bias, act, residual, x_scale, w_scale, keep_pre, workspace, device_status, stream
PyObject* linear_fwd(PyObject* const* a) {
  const Tensor& x = matrix("x", a[0], kOperands);
  const int64_t rows = x.size(0);
  const int inner = width_of("x's width", x.size(1));
  const c10::Device dev = x.device();
  const Tensor& w = weight_of(a[1], x);
  const int outer = width_of("W's rows", w.size(0));
  const bool e4m3 = x.scalar_type() == at::kFloat8_e4m3fn;
  if (e4m3 && (!given(a[5]) || !given(a[6]))) raise(PyExc_ValueError, "e4m3 operands need x_scale and w_scale");
  if (!e4m3 && (given(a[5]) || given(a[6]))) raise(PyExc_ValueError, "x_scale and w_scale go with e4m3 operands");
  const Tensor none;
  const Tensor& xs = e4m3 ? vector("x_scale", a[5], kF32, dev, rows) : none;
  const Tensor& wsc = e4m3 ? vector("w_scale", a[6], kF32, dev, outer) : none;
  const Tensor& b = given(a[2]) ? vector("bias", a[2], kFloats, dev, outer) : none;
  const Tensor& r = given(a[4]) ? matrix("residual", a[4], kBf16, &dev, rows, outer) : none;
  const int type = type_of(x.scalar_type());
  const On on(dev, a[10]);
  const Tensor y = empty({rows, outer}, at::kBFloat16, dev);
  Tensor pre;
  if (truth(a[7])) pre = empty({rows, outer}, at::kBFloat16, dev);
  const Scratch ws(api.linear_fwd_workspace(rows, inner, outer, type), dev, a[8], a[9]);
  check(api.linear_fwd(x.data_ptr(), ld(x), w.data_ptr(), ld(w), type, static_cast<const float*>(opt(xs)),
                       static_cast<const float*>(opt(wsc)), opt(b), b.defined() ? type_of(b.scalar_type()) : 0, opt(r),
                       r.defined() ? ld(r) : 0, static_cast<int>(integer(a[3])), rows, inner,
                       outer, y.data_ptr(), outer, opt(pre), outer, ws.ptr, ws.bytes, ws.status, on.stream),
        "uf_linear_fwd");
  on.uses(a, 11);
  Result out;
  out.put("y", y);
  if (pre.defined()) out.put("pre", pre);
  return out.dict;
}

// dy, x, W, pre, act, dx, dW, dbias, workspace, device_status, stream
PyObject* linear_bwd(PyObject* const* a) {
  const Tensor& x = matrix("x", a[1], kBf16);
  const int64_t rows = x.size(0);
  const int inner = width_of("x's width", x.size(1));
  const c10::Device dev = x.device();
  const Tensor& w = weight_of(a[2], x);
  const int outer = width_of("W's rows", w.size(0));
  const Tensor& dy = matrix("dy", a[0], kFloats, &dev, rows, outer);
  const int act = static_cast<int>(integer(a[4]));
  const Tensor none;
  if (act && !given(a[3])) raise(PyExc_ValueError, "an activation's backward needs pre");
  const Tensor& pre = act ? matrix("pre", a[3], kBf16, &dev, rows, outer) : none;
  const On on(dev, a[10]);
  Tensor dx, dw, db;
  if (truth(a[5])) dx = empty({rows, inner}, at::kBFloat16, dev);
  if (truth(a[6])) dw = empty({outer, inner}, at::kBFloat16, dev);
  if (truth(a[7])) db = empty({outer}, at::kFloat, dev);
  const Scratch ws(api.linear_bwd_workspace(rows, inner, outer), dev, a[8], a[9]);
  check(api.linear_bwd(dy.data_ptr(), ld(dy), type_of(dy.scalar_type()), x.data_ptr(), ld(x), w.data_ptr(), ld(w), opt(pre),
                       act ? ld(pre) : 0, act, rows, inner, outer, opt(dx), inner,
                       opt(dw), inner, static_cast<float*>(opt(db)), ws.ptr, ws.bytes, ws.status, on.stream),
        "uf_linear_bwd");
  on.uses(a, 11);
  Result out;
  if (dx.defined()) out.put("dx", dx);
  if (dw.defined()) out.put("dW", dw);
  if (db.defined()) out.put("dbias", db);
  return out.dict;
}

const Tensor& gated_weight(PyObject* o, const Tensor& x) {
  const c10::Device dev = x.device();
  const Tensor& w = matrix("W", o, kBf16, &dev);
  if (w.size(1) != x.size(1) || w.size(0) % 2)
    raise(PyExc_ValueError, "W must be (2 outer) x %lld (the gate's rows, then the up projection's), not (%lld, %lld)",
          static_cast<long long>(x.size(1)), static_cast<long long>(w.size(0)), static_cast<long long>(w.size(1)));
  return w;
}

// x, W, act, keep_pre, workspace, device_status, stream
PyObject* gated_fwd(PyObject* const* a) {
  const Tensor& x = matrix("x", a[0], kBf16);
  const int64_t rows = x.size(0);
  const int inner = width_of("x's width", x.size(1));
  const c10::Device dev = x.device();
  const Tensor& w = gated_weight(a[1], x);
  const int outer = width_of("W's rows", w.size(0)) / 2;
  const On on(dev, a[6]);
  const Tensor h = empty({rows, outer}, at::kBFloat16, dev);
  Tensor pre;
  if (truth(a[3])) pre = empty({rows, 2 * outer}, at::kBFloat16, dev);
  const Scratch ws(api.gated_fwd_workspace(rows, inner, outer), dev, a[4], a[5]);
  check(api.gated_fwd(x.data_ptr(), ld(x), w.data_ptr(), ld(w), static_cast<int>(integer(a[2])), rows,
                      inner, outer, h.data_ptr(), outer, opt(pre), 2 * outer, ws.ptr,
                      ws.bytes, ws.status, on.stream),
        "uf_gated_fwd");
  on.uses(a, 7);
  Result out;
  out.put("h", h);
  if (pre.defined()) out.put("pre", pre);
  return out.dict;
}

// dh, x, W, pre, act, dx, dW, workspace, device_status, stream
PyObject* gated_bwd(PyObject* const* a) {
  const Tensor& x = matrix("x", a[1], kBf16);
  const int64_t rows = x.size(0);
  const int inner = width_of("x's width", x.size(1));
  const c10::Device dev = x.device();
  const Tensor& w = gated_weight(a[2], x);
  const int outer = width_of("W's rows", w.size(0)) / 2;
  const Tensor& dh = matrix("dh", a[0], kBf16, &dev, rows, outer);
  const Tensor& pre = matrix("pre", a[3], kBf16, &dev, rows, 2 * outer);
  const On on(dev, a[9]);
  Tensor dx, dw;
  if (truth(a[5])) dx = empty({rows, inner}, at::kBFloat16, dev);
  if (truth(a[6])) dw = empty({2 * outer, inner}, at::kBFloat16, dev);
  const Scratch ws(api.gated_bwd_workspace(rows, inner, outer), dev, a[7], a[8]);
  check(api.gated_bwd(dh.data_ptr(), ld(dh), x.data_ptr(), ld(x), w.data_ptr(), ld(w), pre.data_ptr(), ld(pre),
                      static_cast<int>(integer(a[4])), rows, inner, outer, opt(dx),
                      inner, opt(dw), inner, ws.ptr, ws.bytes, ws.status, on.stream),
        "uf_gated_bwd");
  on.uses(a, 10);
  Result out;
  if (dx.defined()) out.put("dx", dx);
  if (dw.defined()) out.put("dW", dw);
  return out.dict;
}

// The optimizer's tensors as a step finds them.  Nothing of them is kept between steps: the storage
// under a tensor may be replaced at any time (p.data = ..., set_, resize_, a state moved to the
// host and back), and so may an entry of the lists.
struct AdamTensors {
  std::vector<void*> p, m, v, copy;
  std::vector<float*> ms, vs;
  std::vector<const void*> g;
  std::vector<int64_t> sizes;
  std::vector<c10::TensorImpl*> written;  // of the lists, which hold them
  c10::Device dev{c10::kCPU};
  at::ScalarType ptype = at::kFloat, stype = at::kFloat, gtype = at::kFloat;
};
constexpr int64_t kStateBlock = 256;  // elements that share a scale in 8-bit states

// Calls f(i, tensor) for a list of contiguous CUDA tensors of one type on dev.
template <typename F>
void each(const c10::Device& dev, const char* name, PyObject* list, Types types, int64_t n, const std::vector<int64_t>* numels,
          at::ScalarType* type, F&& f) {
  PyObject* seq = PySequence_Fast(list, name);
  if (!seq) throw Raised{};
  try {
    if (PySequence_Fast_GET_SIZE(seq) != n)
      raise(PyExc_ValueError, "%s must hold %lld tensors, not %lld", name, static_cast<long long>(n),
            static_cast<long long>(PySequence_Fast_GET_SIZE(seq)));
    PyObject** items = PySequence_Fast_ITEMS(seq);
    for (int64_t i = 0; i < n; ++i) {
      const bool ok = THPVariable_Check(items[i]);
      if (i == 0 && ok && types.has(THPVariable_Unpack(items[0]).scalar_type())) *type = THPVariable_Unpack(items[0]).scalar_type();
      const Types want = i == 0 ? types : Types{*type, *type};
      if (!ok || !want.has(THPVariable_Unpack(items[i]).scalar_type()) || !THPVariable_Unpack(items[i]).is_cuda())
        raise(PyExc_TypeError, "%s[%lld] must be a CUDA tensor of %s", name, static_cast<long long>(i), want.names().c_str());
      const Tensor& t = THPVariable_Unpack(items[i]);
      if (t.device() != dev || !t.is_contiguous() || (numels && t.numel() != (*numels)[i])) {
        if (numels)
          raise(PyExc_ValueError, "%s[%lld] must be contiguous, on %s and have %lld elements", name, static_cast<long long>(i),
                dev.str().c_str(), static_cast<long long>((*numels)[i]));
        raise(PyExc_ValueError, "%s[%lld] must be contiguous and on %s", name, static_cast<long long>(i), dev.str().c_str());
      }
      f(i, t);
    }
  } catch (...) {
    Py_DECREF(seq);
    throw;
  }
  Py_DECREF(seq);
}

// params, m, v, m_scale, v_scale, copies
AdamTensors adam_tensors(PyObject* const* a) {
  AdamTensors q;
  const Py_ssize_t n = PySequence_Size(a[0]);
  if (n < 0) throw Raised{};
  if (n > 0) {
    PyObject* first = PySequence_GetItem(a[0], 0);
    if (first && THPVariable_Check(first)) q.dev = THPVariable_Unpack(first).device();
    Py_XDECREF(first);
  }
  auto keep = [&](auto& to) {
    to.reserve(static_cast<size_t>(n));
    return [&](int64_t, const Tensor& t) {
      q.written.push_back(t.unsafeGetTensorImpl());
      to.push_back(static_cast<typename std::decay_t<decltype(to)>::value_type>(t.data_ptr()));
    };
  };
  q.p.reserve(static_cast<size_t>(n));
  q.sizes.reserve(static_cast<size_t>(n));
  q.written.reserve(static_cast<size_t>(n) * 6);
  each(q.dev, "params", a[0], kFloats, n, nullptr, &q.ptype, [&](int64_t, const Tensor& t) {
    q.written.push_back(t.unsafeGetTensorImpl());
    q.p.push_back(t.data_ptr());
    q.sizes.push_back(t.numel());
  });
  const Types states{at::kFloat, at::kFloat8_e4m3fn};
  each(q.dev, "m", a[1], states, n, &q.sizes, &q.stype, keep(q.m));
  at::ScalarType v_type = q.stype;
  each(q.dev, "v", a[2], Types{q.stype, q.stype}, n, &q.sizes, &v_type, keep(q.v));
  const bool e8 = n > 0 && q.stype == at::kFloat8_e4m3fn;
  if (e8 != given(a[3]) || e8 != given(a[4])) raise(PyExc_ValueError, "m_scale and v_scale go with 8-bit states");
  if (e8) {
    std::vector<int64_t> blocks;
    blocks.reserve(static_cast<size_t>(n));
    for (int64_t s : q.sizes) blocks.push_back((s + kStateBlock - 1) / kStateBlock);
    at::ScalarType f = at::kFloat;
    each(q.dev, "m_scale", a[3], kF32, n, &blocks, &f, keep(q.ms));
    each(q.dev, "v_scale", a[4], kF32, n, &blocks, &f, keep(q.vs));
  }
  if (given(a[5])) {
    if (q.ptype != at::kFloat) raise(PyExc_ValueError, "copies go with fp32 parameters");
    at::ScalarType b = at::kBFloat16;
    each(q.dev, "copies", a[5], kBf16, n, &q.sizes, &b, keep(q.copy));
  }
  return q;
}

// params, m, v, m_scale, v_scale, copies: checks them
PyObject* adamw_check(PyObject* const* a) {
  adam_tensors(a);
  Py_RETURN_NONE;
}

// params, m, v, m_scale, v_scale, copies, grads, lr (float or tensor), betas[0], betas[1], eps, weight_decay,
// step, step_dev, seed, grad_scale, stream
PyObject* adamw_step(PyObject* const* a) {
  PyObject* const* lists = a;
  a += 6;
  // (numbers first: none of them may run code once addresses are taken)
  const bool lr_tensor = THPVariable_Check(a[1]);
  const float lr = lr_tensor ? 0.f : static_cast<float>(number(a[1]));
  const double beta1 = number(a[2]), beta2 = number(a[3]);
  const float eps = static_cast<float>(number(a[4])), decay = static_cast<float>(number(a[5]));
  const int64_t step = integer(a[6]);
  const uint32_t seed = static_cast<uint32_t>(integer(a[8]));
  AdamTensors q = adam_tensors(lists);
  const int64_t n = static_cast<int64_t>(q.sizes.size());
  q.g.reserve(static_cast<size_t>(n));
  each(q.dev, "grads", a[0], kFloats, n, &q.sizes, &q.gtype, [&](int64_t, const Tensor& t) { q.g.push_back(t.data_ptr()); });
  if (n == 0) Py_RETURN_NONE;
  auto scalar = [&](const char* name, PyObject* o, at::ScalarType t) -> void* {
    if (!given(o)) return nullptr;
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).scalar_type() != t || THPVariable_Unpack(o).device() != q.dev ||
        THPVariable_Unpack(o).numel() != 1)
      raise(PyExc_TypeError, "%s must be a one-element %s tensor on %s", name, t == at::kFloat ? "float32" : "int64",
            q.dev.str().c_str());
    return THPVariable_Unpack(o).data_ptr();
  };
  const auto* lr_dev = static_cast<const float*>(lr_tensor ? scalar("lr", a[1], at::kFloat) : nullptr);
  const auto* step_dev = static_cast<const int64_t*>(scalar("step_dev", a[7], at::kLong));
  const auto* gs = static_cast<const float*>(scalar("grad_scale", a[9], at::kFloat));
  const On on(q.dev, a[10]);
  check(api.adamw_step(static_cast<int>(n), q.p.data(), q.g.data(), q.m.data(), q.v.data(),
                       q.ms.empty() ? nullptr : q.ms.data(), q.vs.empty() ? nullptr : q.vs.data(),
                       q.copy.empty() ? nullptr : q.copy.data(), q.sizes.data(), type_of(q.ptype), type_of(q.gtype),
                       type_of(q.stype), lr, lr_dev, beta1, beta2, eps, decay, step, step_dev, seed, gs, on.stream),
        "uf_adamw_step");
  on.uses(lists, 17);
  // as torch's in-place operations do: a backward that saved one of them raises
  for (c10::TensorImpl* t : q.written)
    if (!t->is_inference()) t->bump_version();
  Py_RETURN_NONE;
}

// UfError, {name: address of a C entry point}
PyObject* bind(PyObject* const* a) {
  auto get = [&](const char* name) -> void* {
    PyObject* o = PyDict_GetItemString(a[1], name);
    if (!o) raise(PyExc_KeyError, "%s", name);
    void* p = PyLong_AsVoidPtr(o);
    if (!p) raise(PyExc_ValueError, "%s has no address", name);
    return p;
  };
#define UF_BIND(f) api.f = reinterpret_cast<decltype(api.f)>(get("uf_" #f))
  UF_BIND(rmsnorm_fwd);
  UF_BIND(rmsnorm_bwd_workspace);
  UF_BIND(rmsnorm_bwd);
  UF_BIND(linear_fwd_workspace);
  UF_BIND(linear_fwd);
  UF_BIND(linear_bwd_workspace);
  UF_BIND(linear_bwd);
  UF_BIND(gated_fwd_workspace);
  UF_BIND(gated_fwd);
  UF_BIND(gated_bwd_workspace);
  UF_BIND(gated_bwd);
  UF_BIND(adamw_step);
#undef UF_BIND
  Py_INCREF(a[0]);
  Py_XDECREF(uf_error);
  uf_error = a[0];
  Py_RETURN_NONE;
}

// A function of N positional arguments; no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), int N, bool BOUND>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "takes %d arguments, not %zd", N, n);
  if (BOUND && !uf_error) return PyErr_Format(PyExc_RuntimeError, "the library's entry points are not bound");
  HANDLE_TH_ERRORS  // torch's own errors (its allocator's among them) under their own types
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N, bool BOUND = true>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F, N, BOUND>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 2, false>("bind"),
                         method<rmsnorm_fwd, 6>("rmsnorm_fwd"),
                         method<rmsnorm_bwd, 8>("rmsnorm_bwd"),
                         method<linear_fwd, 11>("linear_fwd"),
                         method<linear_bwd, 11>("linear_bwd"),
                         method<gated_fwd, 7>("gated_fwd"),
                         method<gated_bwd, 10>("gated_bwd"),
                         method<adamw_check, 6>("adamw_check"),
                         method<adamw_step, 17>("adamw_step"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_native(void) { return PyModule_Create(&module); }
