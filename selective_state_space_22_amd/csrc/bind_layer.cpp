// bind_layer.cpp -- the marshalling of layer.py's calls, as a CPython module over torch's C++ tensors.
//
// A call on one token is as long as its checks and allocations: formed in Python, those of the backward of the
// norms took 25 us beside 7 us of launches.  Every function checks its tensors (GPU, device, contiguity, type,
// shape), allocates the outputs that were not given, and calls the entry point of the same name of the C ABI,
// whose address it takes from the library that ctypes has loaded.  Nothing else of the library is known here.
#include <Python.h>

#include <dlfcn.h>

#include <initializer_list>
#include <string>

#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mamba_mi355x_layer.h"

namespace {

struct Api {
  decltype(&mamba_conv_fwd) conv_fwd;
  decltype(&mamba_conv_bwd_workspace_size) conv_bwd_ws;
  decltype(&mamba_conv_bwd) conv_bwd;
  decltype(&mamba_conv_update) conv_update;
  decltype(&mamba_conv_ssm_update_workspace_size) conv_ssm_ws;
  decltype(&mamba_conv_ssm_update) conv_ssm;
  decltype(&mamba_residual_norm_fwd) norm_fwd;
  decltype(&mamba_residual_norm_bwd_workspace_size) norm_bwd_ws;
  decltype(&mamba_residual_norm_bwd) norm_bwd;
  decltype(&mamba_draft_verify_workspace_size) verify_ws;
  decltype(&mamba_draft_verify) verify;
} api;

PyObject* g_error = nullptr;   // MambaError(func, status)
PyObject* g_stream = nullptr;  // device index -> raw stream

// Thrown where a Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    case at::kBool: return "torch.bool";
    default: return std::string("torch.") + at::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument, null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor* t = tensor(o, name);
  if (!t) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  if (dims >= 0 && t->dim() != dims)
    raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dims) + " dimensions, has " +
                                std::to_string(t->dim()));
  return *t;
}

int io_type(at::ScalarType t) {
  if (t == at::kFloat) return MAMBA_IO_F32;
  if (t == at::kBFloat16) return MAMBA_IO_BF16;
  raise(PyExc_TypeError, "I/O tensors must be float32 or bfloat16, got " + type_name(t));
}

// What a call's tensors have in common.
struct Call {
  at::Device dev;
  c10::OptionalDeviceGuard guard;  // kernels go to the tensors' device, whichever is current
  explicit Call(const at::Tensor& x, const char* name) : dev(x.device()) {
    if (!x.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a GPU tensor");
    guard.reset_device(dev);
  }
  void* stream() const {
    PyObject* index = PyLong_FromLong(dev.index());
    PyObject* s = index ? PyObject_CallOneArg(g_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!s) throw Raised{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  }
  // Address of a contiguous tensor of that type and shape on the call's device; null for None and for no elements.
  void* at(const at::Tensor* t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (!t) return nullptr;
    if (t->device() != dev || !t->is_contiguous() || t->scalar_type() != type || t->sizes() != shape)
      refuse(*t, name, type, shape);
    return t->numel() > 0 ? t->data_ptr() : nullptr;
  }
  void* at(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    return at(tensor(o, name), name, type, shape);
  }
  const float* f32(PyObject* o, const char* name, at::IntArrayRef shape) const {
    return static_cast<const float*>(at(o, name, at::kFloat, shape));
  }
  const uint8_t* bytes(PyObject* o, const char* name, at::IntArrayRef shape) const {
    const at::Tensor* t = tensor(o, name);
    if (!t) return nullptr;
    if (t->scalar_type() != at::kBool && t->scalar_type() != at::kByte)
      raise(PyExc_TypeError, std::string(name) + " must be bool or uint8, got " + type_name(t->scalar_type()));
    return static_cast<const uint8_t*>(at(t, name, t->scalar_type(), shape));
  }
  [[noreturn]] void refuse(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    const std::string n(name);
    if (!t.is_cuda()) raise(PyExc_ValueError, n + " must be a GPU tensor");
    if (t.device() != dev) raise(PyExc_ValueError, n + " is on " + t.device().str() + ", expected " + dev.str());
    if (!t.is_contiguous()) raise(PyExc_ValueError, n + " must be contiguous");
    if (t.scalar_type() != type)
      raise(PyExc_TypeError, n + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    raise(PyExc_ValueError, n + " has shape " + shape_name(t.sizes()) + ", expected " + shape_name(shape));
  }
  at::Tensor make(at::ScalarType type, at::IntArrayRef shape) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  }
};

// An output: the caller's tensor, or a new one where `wanted`.
struct Out {
  at::Tensor made;
  PyObject* given = Py_None;
  void* p = nullptr;
  Out(const Call& c, PyObject* o, bool wanted, const char* name, at::ScalarType type, at::IntArrayRef shape) : given(o) {
    if (o != Py_None) {
      p = c.at(o, name, type, shape);
    } else if (wanted) {
      made = c.make(type, shape);
      p = made.numel() > 0 ? made.data_ptr() : nullptr;
    }
  }
  // A new reference to it, or to None.
  PyObject* object() const {
    if (!made.defined()) return Py_NewRef(given);
    PyObject* r = THPVariable_Wrap(made);
    if (!r) throw Raised{};
    return r;
  }
  float* f32() const { return static_cast<float*>(p); }
};

// The caller's workspace, or a new one where need > 0.
struct Workspace {
  at::Tensor made;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(const Call& c, PyObject* o, size_t need) {
    const at::Tensor* t = tensor(o, "workspace");
    if (!t) {
      if (need == 0) return;
      made = c.make(at::kByte, {(int64_t)need});
      t = &made;
    }
    p = c.at(t, "workspace", t->scalar_type(), t->sizes());
    bytes = t->nbytes();
  }
};

void check(const char* func, int status) {
  if (status == MAMBA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", func, status);
  if (e) {
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw Raised{};
}

PyObject* tuple_of(std::initializer_list<const Out*> outs) {
  PyObject* t = PyTuple_New((Py_ssize_t)outs.size());
  if (!t) throw Raised{};
  Py_ssize_t i = 0;
  for (const Out* o : outs) {
    PyObject* v;
    try {
      v = o->object();
    } catch (...) {
      Py_DECREF(t);
      throw;
    }
    PyTuple_SET_ITEM(t, i++, v);
  }
  return t;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

// Calls F(args) with C++ exceptions turned into Python's.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
  try {
    return F(a);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, weight, bias, window, reset, lengths, silu, out, last_window, return_last_window
PyObject* conv_fwd(PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x", 3);
  const at::Tensor& w = needed(a[1], "weight", 2);
  const Call c(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int io = io_type(t);
  const int64_t B = x.size(0), L = x.size(1), D = x.size(2), W = w.size(1);
  const void* px = c.at(&x, "x", t, {B, L, D});
  const float* pw = static_cast<const float*>(c.at(&w, "weight", at::kFloat, {D, W}));
  const float* pb = c.f32(a[2], "bias", {D});
  const int64_t H = W > 0 ? W - 1 : 0;
  const void* win = c.at(a[3], "window", t, {B, H, D});
  const uint8_t* reset = c.bytes(a[4], "reset", {B, L});
  const void* len = c.at(a[5], "lengths", at::kInt, {B});
  const Out out(c, a[7], true, "out", t, {B, L, D});
  const Out last(c, a[8], truth(a[9]), "last_window", t, {B, H, D});
  check("mamba_conv_fwd", api.conv_fwd(B, L, D, W, io, px, pw, pb, win, reset, static_cast<const int32_t*>(len),
                                       truth(a[6]), out.p, last.p, c.stream()));
  return tuple_of({&out, &last});
}

// x, weight, dout, bias, window, reset, silu, dlast_window, dx, dweight, dbias, dwindow, want_dbias, want_dwindow, workspace
PyObject* conv_bwd(PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x", 3);
  const at::Tensor& w = needed(a[1], "weight", 2);
  const Call c(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int io = io_type(t);
  const int64_t B = x.size(0), L = x.size(1), D = x.size(2), W = w.size(1), H = W > 0 ? W - 1 : 0;
  const void* px = c.at(&x, "x", t, {B, L, D});
  const float* pw = static_cast<const float*>(c.at(&w, "weight", at::kFloat, {D, W}));
  const void* dout = c.at(&needed(a[2], "dout", -1), "dout", t, {B, L, D});
  const float* pb = c.f32(a[3], "bias", {D});
  const void* win = c.at(a[4], "window", t, {B, H, D});
  const uint8_t* reset = c.bytes(a[5], "reset", {B, L});
  const void* dlast = c.at(a[7], "dlast_window", t, {B, H, D});
  const Out dx(c, a[8], true, "dx", t, {B, L, D});
  const Out dw(c, a[9], true, "dweight", at::kFloat, {D, W});
  const Out db(c, a[10], truth(a[12]), "dbias", at::kFloat, {D});
  const Out dwin(c, a[11], truth(a[13]), "dwindow", t, {B, H, D});
  const Workspace ws(c, a[14], api.conv_bwd_ws(B, L, D, W, io));
  check("mamba_conv_bwd", api.conv_bwd(B, L, D, W, io, px, pw, pb, win, reset, truth(a[6]), dout, dlast, dx.p, dw.f32(),
                                       db.f32(), dwin.p, ws.p, ws.bytes, c.stream()));
  return tuple_of({&dx, &dw, &db, &dwin});
}

// window, x, weight, bias, slots, silu, out
PyObject* conv_update(PyObject* const* a) {
  const at::Tensor& win = needed(a[0], "window", 3);
  const at::Tensor& x = needed(a[1], "x", 2);
  const at::Tensor& w = needed(a[2], "weight", 2);
  const Call c(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int io = io_type(t);
  const int64_t B = x.size(0), D = x.size(1), S = win.size(0), W = w.size(1), H = W > 0 ? W - 1 : 0;
  void* pwin = c.at(&win, "window", t, {S, H, D});
  const void* px = c.at(&x, "x", t, {B, D});
  const float* pw = static_cast<const float*>(c.at(&w, "weight", at::kFloat, {D, W}));
  const float* pb = c.f32(a[3], "bias", {D});
  const void* slots = c.at(a[4], "slots", at::kInt, {B});
  const Out out(c, a[6], true, "out", t, {B, D});
  check("mamba_conv_update", api.conv_update(B, D, W, io, S, pwin, px, pw, pb, static_cast<const int32_t*>(slots),
                                             truth(a[5]), out.p, c.stream()));
  return out.object();
}

// state, window, x, conv_weight, W_x, W_dt, A, conv_bias, z, dt_bias, Dskip, slots, out, workspace
PyObject* conv_ssm_update(PyObject* const* a) {
  const at::Tensor& state = needed(a[0], "state", 3);
  const at::Tensor& x = needed(a[2], "x", 2);
  const at::Tensor& cw = needed(a[3], "conv_weight", 2);
  const at::Tensor& wdt = needed(a[5], "W_dt", 2);
  const at::Tensor& A = needed(a[6], "A", 2);
  const Call c(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int io = io_type(t);
  const int64_t B = x.size(0), D = x.size(1), S = state.size(0), W = cw.size(1), N = A.size(1), R = wdt.size(1);
  float* ps = static_cast<float*>(c.at(&state, "state", at::kFloat, {S, D, N}));
  void* win = c.at(&needed(a[1], "window", 3), "window", t, {S, W > 0 ? W - 1 : 0, D});
  const void* px = c.at(&x, "x", t, {B, D});
  const float* pcw = static_cast<const float*>(c.at(&cw, "conv_weight", at::kFloat, {D, W}));
  const void* wx = c.at(&needed(a[4], "W_x", 2), "W_x", t, {R + 2 * N, D});
  const void* pwdt = c.at(&wdt, "W_dt", t, {D, R});
  const float* pA = static_cast<const float*>(c.at(&A, "A", at::kFloat, {D, N}));
  const float* cb = c.f32(a[7], "conv_bias", {D});
  const void* z = c.at(a[8], "z", t, {B, D});
  const float* dtb = c.f32(a[9], "dt_bias", {D});
  const float* ds = c.f32(a[10], "Dskip", {D});
  const void* slots = c.at(a[11], "slots", at::kInt, {B});
  const Out out(c, a[12], true, "out", t, {B, D});
  const Workspace ws(c, a[13], api.conv_ssm_ws(B, D, N, R, io));
  check("mamba_conv_ssm_update",
        api.conv_ssm(B, D, N, R, W, io, S, ps, win, px, pcw, cb, wx, pwdt, dtb, pA, ds, z,
                     static_cast<const int32_t*>(slots), out.p, ws.p, ws.bytes, c.stream()));
  return out.object();
}

// The residual stream's type: that of the first tensor given, else float32 (code 0), bfloat16 (1) or x's (-1).
at::ScalarType residual_type(std::initializer_list<const at::Tensor*> given, PyObject* code, at::ScalarType x) {
  at::ScalarType r = x;
  bool found = false;
  for (const at::Tensor* t : given)
    if (t && !found) {
      r = t->scalar_type();
      found = true;
    }
  if (!found) {
    const long v = PyLong_AsLong(code);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    r = v < 0 ? x : (v == 0 ? at::kFloat : at::kBFloat16);
  }
  if (r != x && r != at::kFloat)
    raise(PyExc_TypeError, "residual must be " + type_name(x) + " or torch.float32, got " + type_name(r));
  return r;
}

// x, pre_weight, gate, post_weight, scale, residual, alpha, eps, gate_first, out, residual_out, res_code, return_residual
PyObject* norm_fwd(PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x", -1);
  if (x.dim() == 0) raise(PyExc_ValueError, "x must have a dimension");
  const Call c(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int io = io_type(t);
  const at::IntArrayRef shape = x.sizes();
  const int64_t D = shape.back(), rows = D ? x.numel() / D : 0;
  const at::ScalarType rt = residual_type({tensor(a[5], "residual"), tensor(a[10], "residual_out")}, a[11], t);
  const void* px = c.at(&x, "x", t, shape);
  const float* pre = c.f32(a[1], "pre_weight", {D});
  const void* gate = c.at(a[2], "gate", t, shape);
  const float* post = c.f32(a[3], "post_weight", {D});
  const float* scale = c.f32(a[4], "scale", {D});
  const void* res = c.at(a[5], "residual", rt, shape);
  const bool normed = a[1] != Py_None;
  const Out out(c, normed ? a[9] : Py_None, normed, "out", t, shape);
  const Out rout(c, a[10], truth(a[12]), "residual_out", rt, shape);
  check("mamba_residual_norm_fwd",
        api.norm_fwd(rows, D, io, io_type(rt), px, gate, truth(a[8]), post, scale, res, pre, number(a[6]), number(a[7]),
                     rout.p, out.p, c.stream()));
  return tuple_of({&out, &rout});
}

// x, pre_weight, dout, dresidual_out, gate, post_weight, scale, residual, alpha, eps, gate_first, res_code, then dx,
// dgate, dresidual, dpost_weight, dscale, dpre_weight, then whether the last five are wanted, then workspace
PyObject* norm_bwd(PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x", -1);
  if (x.dim() == 0) raise(PyExc_ValueError, "x must have a dimension");
  const Call c(x, "x");
  const at::ScalarType t = x.scalar_type();
  const int io = io_type(t);
  const at::IntArrayRef shape = x.sizes();
  const int64_t D = shape.back(), rows = D ? x.numel() / D : 0;
  if ((a[1] == Py_None) != (a[2] == Py_None)) raise(PyExc_ValueError, "dout and pre_weight go together");
  const at::ScalarType rt = residual_type({tensor(a[7], "residual"), tensor(a[3], "dresidual_out")}, a[11], t);
  const void* px = c.at(&x, "x", t, shape);
  const float* pre = c.f32(a[1], "pre_weight", {D});
  const void* dout = c.at(a[2], "dout", t, shape);
  const void* dres = c.at(a[3], "dresidual_out", rt, shape);
  const void* gate = c.at(a[4], "gate", t, shape);
  const float* post = c.f32(a[5], "post_weight", {D});
  const float* scale = c.f32(a[6], "scale", {D});
  const void* res = c.at(a[7], "residual", rt, shape);
  const Out dx(c, a[12], true, "dx", t, shape);
  const Out dgate(c, a[13], truth(a[18]), "dgate", t, shape);
  const Out dresidual(c, a[14], truth(a[19]), "dresidual", rt, shape);
  const Out dpost(c, a[15], truth(a[20]), "dpost_weight", at::kFloat, {D});
  const Out dscale(c, a[16], truth(a[21]), "dscale", at::kFloat, {D});
  const Out dpre(c, a[17], truth(a[22]), "dpre_weight", at::kFloat, {D});
  const Workspace ws(c, a[23], api.norm_bwd_ws(rows, D, io));
  check("mamba_residual_norm_bwd",
        api.norm_bwd(rows, D, io, io_type(rt), px, gate, truth(a[10]), post, scale, res, pre, number(a[8]), number(a[9]),
                     dout, dres, dx.p, dgate.p, dresidual.p, dpost.f32(), dscale.f32(), dpre.f32(), ws.p, ws.bytes,
                     c.stream()));
  return tuple_of({&dx, &dgate, &dresidual, &dpost, &dscale, &dpre});
}

// target, draft, drafted, uniform, noise, counts, tokens, accepted, workspace
PyObject* draft_verify(PyObject* const* a) {
  const at::Tensor& p = needed(a[0], "target", 3);
  const at::Tensor& q = needed(a[1], "draft", 3);
  const Call c(p, "target");
  const at::ScalarType t = p.scalar_type();
  const int io = io_type(t);
  const int64_t rows = q.size(0), K = q.size(1), V = q.size(2);
  const void* pp = c.at(&p, "target", t, {rows, K + 1, V});
  const void* pq = c.at(&q, "draft", t, {rows, K, V});
  const void* ids = c.at(&needed(a[2], "drafted", -1), "drafted", at::kLong, {rows, K});
  const void* u = c.at(&needed(a[3], "uniform", -1), "uniform", at::kFloat, {rows, K});
  const void* noise = c.at(&needed(a[4], "noise", -1), "noise", at::kFloat, {rows, V});
  const void* counts = c.at(a[5], "counts", at::kInt, {rows});
  const Out tokens(c, a[6], true, "tokens", at::kLong, {rows, K + 1});
  const Out accepted(c, a[7], true, "accepted", at::kInt, {rows});
  const Workspace ws(c, a[8], api.verify_ws(rows, K, V, io));
  check("mamba_draft_verify",
        api.verify(rows, K, V, io, pp, pq, static_cast<const int64_t*>(ids), static_cast<const float*>(u),
                   static_cast<const float*>(noise), static_cast<const int32_t*>(counts), static_cast<int64_t*>(tokens.p),
                   static_cast<int32_t*>(accepted.p), ws.p, ws.bytes, c.stream()));
  return tuple_of({&tokens, &accepted});
}

// use(handle, MambaError, stream of a device): the library that dlopen's handle names.
PyObject* use(PyObject*, PyObject* args) {
  PyObject *handle, *error, *stream;
  if (!PyArg_ParseTuple(args, "OOO", &handle, &error, &stream)) return nullptr;
  void* lib = PyLong_AsVoidPtr(handle);
  if (!lib) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no library");
  bool all = true;
  auto take = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
    if (!f && all) {
      PyErr_Format(PyExc_ImportError, "the library has no %s: build it again", name);
      all = false;
    }
  };
  take(api.conv_fwd, "mamba_conv_fwd");
  take(api.conv_bwd_ws, "mamba_conv_bwd_workspace_size");
  take(api.conv_bwd, "mamba_conv_bwd");
  take(api.conv_update, "mamba_conv_update");
  take(api.conv_ssm_ws, "mamba_conv_ssm_update_workspace_size");
  take(api.conv_ssm, "mamba_conv_ssm_update");
  take(api.norm_fwd, "mamba_residual_norm_fwd");
  take(api.norm_bwd_ws, "mamba_residual_norm_bwd_workspace_size");
  take(api.norm_bwd, "mamba_residual_norm_bwd");
  take(api.verify_ws, "mamba_draft_verify_workspace_size");
  take(api.verify, "mamba_draft_verify");
  if (!all) return nullptr;
  Py_XSETREF(g_error, Py_NewRef(error));
  Py_XSETREF(g_stream, Py_NewRef(stream));
  Py_RETURN_NONE;
}

#define S6_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"use", use, METH_VARARGS, nullptr}, S6_ENTRY(conv_fwd, 10), S6_ENTRY(conv_bwd, 15),
                         S6_ENTRY(conv_update, 7), S6_ENTRY(conv_ssm_update, 14), S6_ENTRY(norm_fwd, 13),
                         S6_ENTRY(norm_bwd, 24), S6_ENTRY(draft_verify, 9), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__layer() { return PyModule_Create(&module); }
