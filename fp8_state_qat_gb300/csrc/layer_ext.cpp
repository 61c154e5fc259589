// layer_ext.cpp -- the Python side of the layer operators: argument checks, allocations on the current
// stream, and the call of the C ABI (include/gdnqat.h), whose entry points are handed over as addresses.
//
// The small calls take 3 to 5 us on the GPU; checks and allocations in Python take 8 to 20 us a call, here 1 to 3.
// Python keeps the signatures, the documentation and the case of another stream or device (layer.py).
#include <Python.h>

#include <cstdarg>
#include <initializer_list>
#include <optional>
#include <string>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdnqat.h"

namespace {

using at::Tensor;

// ---- the library's entry points, and the Python function that raises its errors ----
#define ENTRIES(X)                                                                                                 \
  X(la_chunk_fwd) X(la_chunk_fwd_workspace_size) X(la_chunk_bwd) X(la_chunk_bwd_workspace_size) X(la_decode_step) \
  X(gdn_upload_i32) X(gated_norm_fwd) X(gated_norm_bwd) X(gated_norm_bwd_workspace_size) X(residual_norm_fwd)     \
  X(residual_norm_bwd) X(residual_norm_bwd_workspace_size)
#define DECLARE(f) decltype(&::f) p_##f = nullptr;
ENTRIES(DECLARE)
#undef DECLARE
PyObject* raise_status = nullptr;

struct Bad {};   // a Python exception is set

[[noreturn]] void bad(PyObject* type, const char* format, ...) {
  va_list a;
  va_start(a, format);
  PyErr_FormatV(type, format, a);
  va_end(a);
  throw Bad();
}

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}
const char* text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
// A tensor, or an undefined one for None.
Tensor optional(PyObject* o, const char* name) { return o == Py_None ? Tensor() : tensor(o, name); }

// The address of a contiguous tensor of this type and shape on this device (null for an undefined one).
void* is(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, int device, const char* name) {
  if (!t.defined()) return nullptr;
  if (t.scalar_type() != type) bad(PyExc_ValueError, "%s must be %s, got %s", name, text(type), text(t.scalar_type()));
  if (t.sizes() != shape)
    bad(PyExc_ValueError, "%s must have shape %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
  if (!t.is_cuda() || t.get_device() != device)
    bad(PyExc_ValueError, "%s must be a CUDA tensor on device %d, got one on %s", name, device, t.device().str().c_str());
  if (!t.is_contiguous()) bad(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}
int32_t code(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return GDN_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return GDN_DTYPE_F32;
  bad(PyExc_ValueError, "%s must be torch.bfloat16 or torch.float32, got %s", name, text(t.scalar_type()));
}

Tensor make(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
}
// The workspace that was given, or one of the size that is needed.
struct Room {
  Tensor t;
  void* p;
  size_t n;
};
Room room(PyObject* given, size_t need, int device) {
  Tensor t = optional(given, "workspace");
  if (!t.defined()) t = make({(int64_t)(need > 256 ? need : 256)}, at::kByte, device);
  return {t, is(t, at::kByte, t.sizes(), device, "workspace"), (size_t)t.numel()};
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Bad();
  return x;
}
gdn_stream_t stream(int device) {
  return reinterpret_cast<gdn_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
}
void done(const char* fn, gdn_status s) {
  if (s == GDN_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "si", fn, (int)s);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
  throw Bad();
}
// The device of the call: the first tensor's; -1 where it is not the current one (layer.py then makes it so).
int here(const Tensor& t) {
  const int d = t.is_cuda() ? (int)t.get_device() : -1;
  return d >= 0 && d == (int)c10::cuda::current_device() ? d : -1;
}
PyObject* elsewhere() { Py_RETURN_NOTIMPLEMENTED; }

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* pack(std::initializer_list<PyObject*> items) {   // steals the references
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (r) PyTuple_SET_ITEM(r, i++, o);
    else Py_XDECREF(o);
  }
  return r;
}

// ---- linear attention ----
struct LaCall {
  la_chunk_args a{};
  Tensor q, k, v, g, h0, cu_dev;   // what the arguments point into
  std::vector<int32_t> cu_host;
  int device;
};
// Other Python threads run in its scope.
struct NoGil {
  PyThreadState* const state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// The offsets of packed sequences, read once: the host's validation and sizes and the kernels go by the same values,
// whatever becomes of the tensor after the call.
void offsets(LaCall& c, const Tensor& cu) {
  if (cu.dim() != 1 || cu.numel() < 1) bad(PyExc_ValueError, "cu_seqlens must be [N + 1]");
  if (!at::isIntegralType(cu.scalar_type(), false))
    bad(PyExc_ValueError, "cu_seqlens must hold whole numbers, got %s", text(cu.scalar_type()));
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cu.is_cuda() && cudaStreamIsCapturing((cudaStream_t)stream(c.device), &capture) == cudaSuccess &&
      capture != cudaStreamCaptureStatusNone)
    bad(PyExc_ValueError, "cu_seqlens on the device cannot be read while a graph is captured: pass a CPU tensor");
  Tensor host;
  {
    // From a CUDA tensor this waits for the stream, whose work may itself wait for another thread. A CPU tensor's values
    // are there: to give the lock away for them could cost the time that a busy thread keeps it, milliseconds.
    std::optional<NoGil> others;
    if (cu.is_cuda()) others.emplace();
    host = cu.detach().to(at::kCPU, at::kLong).contiguous();
  }
  const int64_t* x = static_cast<const int64_t*>(host.data_ptr());
  c.cu_host.resize((size_t)host.numel());
  for (size_t i = 0; i < c.cu_host.size(); ++i) {
    if (x[i] != (int32_t)x[i]) bad(PyExc_ValueError, "cu_seqlens[%zu] does not fit in 32 bits", i);
    c.cu_host[i] = (int32_t)x[i];
  }
  c.cu_dev = make({host.numel()}, at::kInt, c.device);
  int32_t* const device = static_cast<int32_t*>(c.cu_dev.data_ptr());
  done("gdn_upload_i32", p_gdn_upload_i32(c.cu_host.data(), device, host.numel(), stream(c.device)));
  c.a.cu_seqlens = device;
  c.a.cu_seqlens_host = c.cu_host.data();
}
void la_args(LaCall& c, PyObject* const* o, double scale) {   // q, k, v, g, h0, cu_seqlens
  c.k = tensor(o[1], "k");
  c.v = tensor(o[2], "v");
  c.g = tensor(o[3], "g");
  c.h0 = optional(o[4], "h0");
  const Tensor cu = optional(o[5], "cu_seqlens");
  if (c.q.dim() != 4 || c.v.dim() != 4) bad(PyExc_ValueError, "q, k, v must be [B, T, H, D]");
  const int64_t B = c.q.size(0), T = c.q.size(1), Hqk = c.q.size(2), dk = c.q.size(3), Hv = c.v.size(2), dv = c.v.size(3);
  int64_t N = B;
  if (cu.defined()) {
    offsets(c, cu);
    N = (int64_t)c.cu_host.size() - 1;
  }
  const bool head = c.g.dim() == 1;
  c.a.q = is(c.q, at::kBFloat16, c.q.sizes(), c.device, "q");
  c.a.k = is(c.k, at::kBFloat16, c.q.sizes(), c.device, "k");
  c.a.v = is(c.v, at::kBFloat16, {B, T, Hv, dv}, c.device, "v");
  c.a.g = static_cast<const float*>(head ? is(c.g, at::kFloat, {Hv}, c.device, "g") : is(c.g, at::kFloat, {B, T, Hv}, c.device, "g"));
  c.a.h0 = static_cast<const float*>(is(c.h0, at::kFloat, {N, Hv, dk, dv}, c.device, "h0"));
  for (int64_t x : {B, T, N, Hqk, Hv, dk, dv})
    if (x > INT32_MAX) bad(PyExc_ValueError, "a dimension is too large");
  c.a.B = (int32_t)B;
  c.a.T = (int32_t)T;
  c.a.N = (int32_t)N;
  c.a.Hqk = (int32_t)Hqk;
  c.a.Hv = (int32_t)Hv;
  c.a.dk = (int32_t)dk;
  c.a.dv = (int32_t)dv;
  c.a.scale = (float)scale;
  c.a.flags = head ? LA_FLAG_HEAD_DECAY : 0;
}

// q, k, v, g, h0, cu_seqlens, scale, o, hT, output_final_state, workspace
PyObject* la_chunk_fwd_(PyObject* const* o) {
  LaCall c;
  c.q = tensor(o[0], "q");
  if ((c.device = here(c.q)) < 0) return elsewhere();
  la_args(c, o, number(o[6]));
  Tensor out = optional(o[7], "o"), hT = optional(o[8], "hT");
  const int64_t state[4] = {c.a.N, c.a.Hv, c.a.dk, c.a.dv};
  if (!out.defined()) out = make(c.v.sizes(), at::kBFloat16, c.device);
  if (!hT.defined() && PyObject_IsTrue(o[9])) hT = make(state, at::kFloat, c.device);
  c.a.o = is(out, at::kBFloat16, c.v.sizes(), c.device, "o");
  c.a.hT = static_cast<float*>(is(hT, at::kFloat, state, c.device, "hT"));
  const Room ws = room(o[10], p_la_chunk_fwd_workspace_size(&c.a), c.device);
  done("la_chunk_fwd", p_la_chunk_fwd(&c.a, ws.p, ws.n, stream(c.device)));
  return pack({wrap(out), wrap(hT)});
}

// q, k, v, g, h0, cu_seqlens, dout, dhT, scale, want_dh0, workspace
PyObject* la_chunk_bwd_(PyObject* const* o) {
  LaCall c;
  c.q = tensor(o[0], "q");
  if ((c.device = here(c.q)) < 0) return elsewhere();
  if (o[6] == Py_None) bad(PyExc_ValueError, "dout is required");
  la_args(c, o, number(o[8]));
  const Tensor dout = tensor(o[6], "dout"), dhT = optional(o[7], "dhT");
  const int64_t state[4] = {c.a.N, c.a.Hv, c.a.dk, c.a.dv};
  la_chunk_grads gr{};
  gr.dout = is(dout, at::kBFloat16, c.v.sizes(), c.device, "dout");
  gr.dhT = static_cast<const float*>(is(dhT, at::kFloat, state, c.device, "dhT"));
  const Tensor dq = make(c.q.sizes(), at::kBFloat16, c.device), dk = make(c.q.sizes(), at::kBFloat16, c.device);
  const Tensor dv = make(c.v.sizes(), at::kBFloat16, c.device), dg = make(c.g.sizes(), at::kFloat, c.device);
  const Tensor dh0 = PyObject_IsTrue(o[9]) ? make(state, at::kFloat, c.device) : Tensor();
  gr.dq = dq.data_ptr();
  gr.dk = dk.data_ptr();
  gr.dv = dv.data_ptr();
  gr.dg = static_cast<float*>(dg.data_ptr());
  gr.dh0 = dh0.defined() ? static_cast<float*>(dh0.data_ptr()) : nullptr;
  const Room ws = room(o[10], p_la_chunk_bwd_workspace_size(&c.a), c.device);
  done("la_chunk_bwd", p_la_chunk_bwd(&c.a, &gr, ws.p, ws.n, stream(c.device)));
  return pack({wrap(dq), wrap(dk), wrap(dv), wrap(dg), wrap(dh0)});
}

// q, k, v, g, state, state_out, flags, scale, o
PyObject* la_decode_step_(PyObject* const* o) {
  const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &v = tensor(o[2], "v"), &g = tensor(o[3], "g"),
               &state = tensor(o[4], "state");
  const int d = here(q);
  if (d < 0) return elsewhere();
  if (q.dim() != 3 || v.dim() != 3) bad(PyExc_ValueError, "q, k, v must be [N, H, D]");
  const int64_t N = q.size(0), Hqk = q.size(1), dk = q.size(2), Hv = v.size(1), dv = v.size(2);
  const int64_t full[4] = {N, Hv, dk, dv};
  Tensor state_out = optional(o[5], "state_out"), out = optional(o[8], "o");
  const unsigned long flags = PyLong_AsUnsignedLong(o[6]);
  if (PyErr_Occurred()) throw Bad();
  if (!out.defined()) out = make(v.sizes(), at::kBFloat16, d);
  for (int64_t x : full)
    if (x > INT32_MAX) bad(PyExc_ValueError, "a dimension is too large");
  float* const in = static_cast<float*>(is(state, at::kFloat, full, d, "state"));
  float* const to = state_out.defined() ? static_cast<float*>(is(state_out, at::kFloat, full, d, "state_out")) : in;
  done("la_decode_step",
       p_la_decode_step(is(q, at::kBFloat16, q.sizes(), d, "q"), is(k, at::kBFloat16, q.sizes(), d, "k"),
                        is(v, at::kBFloat16, {N, Hv, dv}, d, "v"),
                        static_cast<const float*>(is(g, at::kFloat, {N, Hv}, d, "g")), in, to,
                        is(out, at::kBFloat16, v.sizes(), d, "o"), (int32_t)N, (int32_t)Hqk, (int32_t)Hv, (int32_t)dk,
                        (int32_t)dv, (float)number(o[7]), (uint32_t)flags, stream(d)));
  return wrap(out);
}

// ---- norms ----
struct Rows {
  int64_t rows;
  int32_t D;
};
Rows rows_of(const Tensor& x) {
  if (x.dim() == 0) bad(PyExc_ValueError, "the normalised tensor needs a last dimension");
  const int64_t D = x.size(-1);
  if (D > INT32_MAX) bad(PyExc_ValueError, "a dimension is too large");
  return {D ? x.numel() / D : 0, (int32_t)D};
}

// x, z, w, eps, y
PyObject* gated_norm_fwd_(PyObject* const* o) {
  const Tensor &x = tensor(o[0], "x"), &z = tensor(o[1], "z"), &w = tensor(o[2], "w");
  const int d = here(x);
  if (d < 0) return elsewhere();
  const int32_t tx = code(x, "x"), tw = code(w, "w");
  const Rows r = rows_of(x);
  const void* px = is(x, x.scalar_type(), x.sizes(), d, "x");
  const void* pz = is(z, at::kBFloat16, x.sizes(), d, "z");
  const void* pw = is(w, w.scalar_type(), {r.D}, d, "w");
  Tensor y = optional(o[4], "y");
  if (!y.defined()) y = make(x.sizes(), at::kBFloat16, d);
  done("gated_norm_fwd", p_gated_norm_fwd(px, tx, pz, pw, tw, is(y, at::kBFloat16, x.sizes(), d, "y"), r.rows, r.D,
                                          (float)number(o[3]), stream(d)));
  return wrap(y);
}

// dy, x, z, w, eps, workspace
PyObject* gated_norm_bwd_(PyObject* const* o) {
  const Tensor &dy = tensor(o[0], "dy"), &x = tensor(o[1], "x"), &z = tensor(o[2], "z"), &w = tensor(o[3], "w");
  const int d = here(x);
  if (d < 0) return elsewhere();
  const int32_t tx = code(x, "x"), tw = code(w, "w");
  const Rows r = rows_of(x);
  const void* pd = is(dy, at::kBFloat16, x.sizes(), d, "dy");
  const void* px = is(x, x.scalar_type(), x.sizes(), d, "x");
  const void* pz = is(z, at::kBFloat16, x.sizes(), d, "z");
  const void* pw = is(w, w.scalar_type(), {r.D}, d, "w");
  const Tensor dx = make(x.sizes(), x.scalar_type(), d), dz = make(x.sizes(), at::kBFloat16, d), dw = make({r.D}, at::kFloat, d);
  const Room ws = room(o[5], p_gated_norm_bwd_workspace_size(r.rows, r.D), d);
  done("gated_norm_bwd",
       p_gated_norm_bwd(pd, px, tx, pz, pw, tw, dx.data_ptr(), dz.data_ptr(), static_cast<float*>(dw.data_ptr()), r.rows,
                        r.D, (float)number(o[4]), ws.p, ws.n, stream(d)));
  return pack({wrap(dx), wrap(dz), wrap(dw)});
}

struct Residual {
  int device;
  int32_t th, tw;
  Rows r;
  const void *y, *h, *w1, *w2;
};
// y, h, w_pre, w_post
bool residual(Residual& a, PyObject* const* o) {
  const Tensor &y = tensor(o[0], "y"), &h = tensor(o[1], "h"), &w1 = tensor(o[2], "w_pre");
  const Tensor w2 = optional(o[3], "w_post");
  if ((a.device = here(h)) < 0) return false;
  a.th = code(h, "h");
  a.tw = code(w1, "w_pre");
  a.r = rows_of(h);
  a.y = is(y, at::kBFloat16, h.sizes(), a.device, "y");
  a.h = is(h, h.scalar_type(), h.sizes(), a.device, "h");
  a.w1 = is(w1, w1.scalar_type(), {a.r.D}, a.device, "w_pre");
  a.w2 = is(w2, w1.scalar_type(), {a.r.D}, a.device, "w_post (as w_pre)");
  return true;
}

// y, h, w_pre, w_post, alpha, eps, h_out, x
PyObject* residual_norm_fwd_(PyObject* const* o) {
  Residual a;
  if (!residual(a, o)) return elsewhere();
  const Tensor& h = tensor(o[1], "h");
  Tensor h_out = optional(o[6], "h_out"), x = optional(o[7], "x");
  if (!h_out.defined()) h_out = make(h.sizes(), h.scalar_type(), a.device);
  if (!x.defined()) x = make(h.sizes(), at::kBFloat16, a.device);
  done("residual_norm_fwd",
       p_residual_norm_fwd(a.y, a.h, a.th, a.w2, a.w1, a.tw, is(h_out, h.scalar_type(), h.sizes(), a.device, "h_out"),
                           is(x, at::kBFloat16, h.sizes(), a.device, "x"), a.r.rows, a.r.D, (float)number(o[4]),
                           (float)number(o[5]), stream(a.device)));
  return pack({wrap(h_out), wrap(x)});
}

// y, h, w_pre, w_post, alpha, eps, dx, dh_out, workspace
PyObject* residual_norm_bwd_(PyObject* const* o) {
  Residual a;
  if (!residual(a, o)) return elsewhere();
  const Tensor& h = tensor(o[1], "h");
  const int d = a.device;
  const Tensor dx = tensor(o[6], "dx"), dh_out = optional(o[7], "dh_out");
  const void* pdx = is(dx, at::kBFloat16, h.sizes(), d, "dx");
  const void* pdh = is(dh_out, h.scalar_type(), h.sizes(), d, "dh_out");
  const Tensor dy = make(h.sizes(), at::kBFloat16, d), dh = make(h.sizes(), h.scalar_type(), d);
  const Tensor dw1 = make({a.r.D}, at::kFloat, d), dw2 = a.w2 ? make({a.r.D}, at::kFloat, d) : Tensor();
  const Room ws = room(o[8], p_residual_norm_bwd_workspace_size(a.r.rows, a.r.D), d);
  done("residual_norm_bwd",
       p_residual_norm_bwd(pdx, pdh, a.y, a.h, a.th, a.w2, a.w1, a.tw, dy.data_ptr(), dh.data_ptr(),
                           dw2.defined() ? static_cast<float*>(dw2.data_ptr()) : nullptr,
                           static_cast<float*>(dw1.data_ptr()), a.r.rows, a.r.D, (float)number(o[4]),
                           (float)number(o[5]), ws.p, ws.n, stream(d)));
  return pack({wrap(dy), wrap(dh), wrap(dw1), wrap(dw2)});
}

// ---- the module ----
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Bad&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind({name: address}, raise_status)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyDict_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "bind(addresses, raise_status)");
    return nullptr;
  }
#define SET(f)                                                                    \
  {                                                                               \
    PyObject* a = PyDict_GetItemString(args[0], #f);                              \
    if (!a) return PyErr_Format(PyExc_KeyError, "no address of %s", #f);          \
    p_##f = reinterpret_cast<decltype(p_##f)>(PyLong_AsVoidPtr(a));               \
    if (PyErr_Occurred()) return nullptr;                                         \
  }
  ENTRIES(SET)
#undef SET
  Py_INCREF(args[1]);
  Py_XDECREF(raise_status);
  raise_status = args[1];
  Py_RETURN_NONE;
}

#define METHOD(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<name##_, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    METHOD(la_chunk_fwd, 11),
    METHOD(la_chunk_bwd, 11),
    METHOD(la_decode_step, 9),
    METHOD(gated_norm_fwd, 5),
    METHOD(gated_norm_bwd, 6),
    METHOD(residual_norm_fwd, 8),
    METHOD(residual_norm_bwd, 9),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdnqat_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdnqat_layer(void) { return PyModule_Create(&module); }
