// p24_torch.cpp -- the binding's marshalling of torch tensors for the calls of which a program makes many on little
// data: pointers, sizes, strides and types are taken from the tensors here instead of in Python, where each of a
// tensor's attributes costs 0.1 us (a norm of one row 6.6 us a call there; the norm over 48 gradients 34 us, clipping
// 144 into other tensors 134). It checks arguments, allocates outputs and scratch that are not given, as memory of the
// current stream, and calls the C entry points of include/prune24.h; there is no arithmetic in it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/Allocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <torch/csrc/Exceptions.h>

#include <algorithm>
#include <string>
#include <vector>

#include "prune24.h"

namespace {

// What a call refuses: thrown here, raised in Python.
struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse_value(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }
[[noreturn]] void refuse_type(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }

std::string device_name(int i) { return i < 0 ? "the CPU" : "cuda:" + std::to_string(i); }
std::string shape_name(int64_t T, int64_t d) {
  return d < 0 ? "(" + std::to_string(T) + ",)" : "(" + std::to_string(T) + ", " + std::to_string(d) + ")";
}

// A call launches on the current device: its tensors have to be there.
void require_device(int tensors, int current) {
  if (tensors != current)
    refuse_value("the tensors are on " + device_name(tensors) + ", the current device is " + device_name(current));
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
int cuda_index(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

int32_t code_of(const at::Tensor& t, const char* name, bool codes = false) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return P24_BF16;
    case at::kFloat: return P24_F32;
    case at::kFloat8_e4m3fn:
      if (codes) return P24_E4M3;
      [[fallthrough]];
    default: refuse_type(std::string(name) + " must be torch.bfloat16 or torch.float32" + (codes ? " or torch.float8_e4m3fn" : "") +
                         ", got " + c10::toString(t.scalar_type()));
  }
}

// What all matrices of a call have in common.
struct Shape {
  int64_t T, d;
  int device;
};
struct Rows {
  const void* p = nullptr;
  int64_t ld = 0;
  int32_t code = P24_F32;
  int64_t T = 0, d = 0;
  int device = -1;
};

// A [T, d] matrix with any row stride; `want`: of that shape and device.
Rows rows(const at::Tensor& t, const char* name, const Shape* want = nullptr, bool codes = false) {
  Rows r;
  r.code = code_of(t, name, codes);
  r.device = cuda_index(t);
  if (t.dim() != 2) refuse_value(std::string(name) + " must be 2-D");
  if (r.device < 0) refuse_value(std::string(name) + " must be a CUDA tensor (libprune24 has no CPU path)");
  r.T = t.size(0), r.d = t.size(1);
  if (want && (r.T != want->T || r.d != want->d || r.device != want->device))
    refuse_value(std::string(name) + " must be a " + shape_name(want->T, want->d) + " tensor on " + device_name(want->device));
  if (r.d > 1 && r.T > 0 && t.stride(1) != 1) refuse_value(std::string(name) + " must be contiguous along its last dimension");
  // a matrix of one row, or of none, may have any row stride in torch
  r.ld = r.T > 1 ? t.stride(0) : std::max(r.d, t.stride(0));
  r.p = t.const_data_ptr();
  return r;
}
// One that is written to: memory that it shares with a lazy copy becomes its own.
void* written(const at::Tensor& t) { return t.mutable_data_ptr(); }
// A contiguous vector of n elements.
const void* vector(const at::Tensor& t, const char* name, int64_t n, at::ScalarType type, int device) {
  if (t.scalar_type() != type) refuse_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.dim() != 1 || t.size(0) != n || cuda_index(t) != device || !t.is_contiguous())
    refuse_value(std::string(name) + " must be a contiguous " + shape_name(n, -1) + " tensor on " + device_name(device));
  return t.const_data_ptr();
}

// An output: the tensor given, or a new one.
at::Tensor output(PyObject* given, const char* name, at::IntArrayRef sizes, const at::Tensor& like, at::ScalarType type) {
  return given == Py_None ? at::empty(sizes, like.options().dtype(type).layout(at::kStrided)) : tensor(given, name);
}
// The caller's object for an output, or one for the new tensor.
PyObject* result(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}

struct Scratch {
  c10::DataPtr own;
  void* p = nullptr;
  size_t bytes = 0;
};
// A call's scratch: the caller's, or one from torch's allocator (without a tensor around it, 0.9 us a call), which is the
// current stream's memory again when it is dropped.
Scratch scratch(PyObject* given, size_t need, const at::Tensor& like) {
  Scratch s;
  if (given == Py_None) {
    static c10::Allocator* const memory = c10::GetAllocator(c10::DeviceType::CUDA);
    s.bytes = std::max<size_t>(need, 16);
    s.own = memory->allocate(s.bytes);
    s.p = s.own.get();
  } else {
    const at::Tensor& t = tensor(given, "workspace");
    if (cuda_index(t) != cuda_index(like) || !t.is_contiguous())
      refuse_value("the workspace must be a contiguous tensor on " + device_name(cuda_index(like)));
    s.p = t.data_ptr(), s.bytes = t.nbytes();
  }
  return s;
}

void* stream_on(int device) {
  require_device(device, c10::cuda::current_device());
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}

int64_t whole(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type(std::string(name) + " must be a whole number");
  }
  return v;
}
float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type(std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse_type(std::string(name) + " must be true or false");
  }
  return v == 1;
}
int32_t group_of(int64_t g) { return g < 0 || g > 256 ? -1 : static_cast<int32_t>(g); }  // the library refuses what is left
int64_t groups_of(int64_t d, int64_t group) { return group > 0 ? (d + group - 1) / group : 1; }

// A function of `n` arguments, with what it throws raised in Python.
template <typename F>
PyObject* call(const char* name, Py_ssize_t given, Py_ssize_t n, F&& f) {
  if (given != n) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, n, given);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (...) {  // torch's own, memory that is not there among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

PyObject* built(int rc, std::initializer_list<PyObject*> results) {
  PyObject* t = PyTuple_New(1 + static_cast<Py_ssize_t>(results.size()));
  Py_ssize_t i = 0;
  if (t) PyTuple_SET_ITEM(t, i++, PyLong_FromLong(rc));
  for (PyObject* r : results) {
    if (t) PyTuple_SET_ITEM(t, i++, r);
    else Py_XDECREF(r);
  }
  return t;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// (x, weight, residual, eps, group, y, h, scale, rstd) -> (status, y, h, scale, rstd)
PyObject* py_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("rmsnorm", n, 9, [&] {
    const at::Tensor& x = tensor(a[0], "x");
    const Rows rx = rows(x, "x");
    const Shape s{rx.T, rx.d, rx.device};
    void* stream = stream_on(s.device);
    const bool quant = a[4] != Py_None;
    const int64_t group = quant ? whole(a[4], "group") : 0;
    p24_rmsnorm_args g{};
    g.T = s.T, g.d = s.d, g.x_dtype = rx.code, g.x = rx.p, g.ldx = rx.ld;
    g.eps = number(a[3], "eps"), g.group = group_of(group);
    if (a[1] != Py_None) {
      const at::Tensor& w = tensor(a[1], "weight");
      g.w_dtype = code_of(w, "weight");
      g.w = vector(w, "weight", s.d, w.scalar_type(), s.device);
    } else {
      g.w_dtype = P24_F32;
    }
    const at::Tensor y = output(a[5], "y", {s.T, s.d}, x, quant ? at::kFloat8_e4m3fn : x.scalar_type());
    const Rows ry = rows(y, "y", &s, true);
    if (quant != (ry.code == P24_E4M3)) refuse_type("y is 8 bits with a group, and is not without one");
    g.y_dtype = ry.code, g.y = written(y), g.ldy = ry.ld;
    at::Tensor h, scale;
    g.r_dtype = rx.code;
    if (a[2] != Py_None) {
      const at::Tensor& r = tensor(a[2], "residual");
      const Rows rr = rows(r, "residual", &s);
      h = output(a[6], "h", {s.T, s.d}, r, r.scalar_type());
      const Rows rh = rows(h, "h", &s);
      if (rh.code != rr.code) refuse_type("h must have the residual's type");
      g.r_dtype = rr.code, g.r = rr.p, g.ldr = rr.ld, g.h = written(h), g.ldh = rh.ld;
    }
    if (quant) {
      const Shape ss{s.T, groups_of(s.d, group), s.device};
      scale = output(a[7], "scale", {ss.T, ss.d}, x, at::kFloat);
      const Rows rs = rows(scale, "scale", &ss);
      if (rs.code != P24_F32) refuse_type("scale must be torch.float32");
      g.scale = static_cast<float*>(written(scale)), g.lds = rs.ld;
    }
    const at::Tensor rstd = output(a[8], "rstd", {s.T}, x, at::kFloat);
    vector(rstd, "rstd", s.T, at::kFloat, s.device);
    g.rstd = static_cast<float*>(written(rstd));
    const int rc = p24_rmsnorm(&g, stream);
    return built(rc, {result(a[5], y), h.defined() ? result(a[6], h) : none(), scale.defined() ? result(a[7], scale) : none(),
                      result(a[8], rstd)});
  });
}

// (dy, h, weight, rstd, dres, dx, dweight or False, workspace) -> (status, dx, dweight)
PyObject* py_rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("rmsnorm_bwd", n, 8, [&] {
    const at::Tensor& h = tensor(a[1], "h");
    const Rows rh = rows(h, "h");
    const Shape s{rh.T, rh.d, rh.device};
    void* stream = stream_on(s.device);
    const Rows rd = rows(tensor(a[0], "dy"), "dy", &s);
    p24_rmsnorm_bwd_args g{};
    g.T = s.T, g.d = s.d, g.h_dtype = rh.code, g.h = rh.p, g.ldh = rh.ld, g.dy_dtype = rd.code, g.dy = rd.p, g.lddy = rd.ld;
    g.w_dtype = P24_F32;
    if (a[2] != Py_None) {
      const at::Tensor& w = tensor(a[2], "weight");
      g.w_dtype = code_of(w, "weight");
      g.w = vector(w, "weight", s.d, w.scalar_type(), s.device);
    }
    g.rstd = static_cast<const float*>(vector(tensor(a[3], "rstd"), "rstd", s.T, at::kFloat, s.device));
    const at::Tensor dx = output(a[5], "dx", {s.T, s.d}, h, h.scalar_type());
    const Rows rx = rows(dx, "dx", &s);
    g.r_dtype = g.dx_dtype = rx.code, g.dx = written(dx), g.lddx = rx.ld;
    if (a[4] != Py_None) {
      const Rows rr = rows(tensor(a[4], "dres"), "dres", &s);
      g.r_dtype = rr.code, g.dres = rr.p, g.ldres = rr.ld;
    }
    at::Tensor dw;
    Scratch ws;
    if (a[6] != Py_False) {
      dw = output(a[6], "dweight", {s.d}, h, at::kFloat);
      vector(dw, "dweight", s.d, at::kFloat, s.device);
      g.dw = static_cast<float*>(written(dw));
      ws = scratch(a[7], p24_rmsnorm_bwd_workspace_size(s.T, s.d), h);
    }
    const int rc = p24_rmsnorm_bwd(&g, ws.p, ws.bytes, stream);
    return built(rc, {result(a[5], dx), dw.defined() ? result(a[6], dw) : none()});
  });
}

// (q, scale, group, out) -> (status, out)
PyObject* py_dequant8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("dequant8", n, 4, [&] {
    const at::Tensor& q = tensor(a[0], "q");
    const Rows rq = rows(q, "q", nullptr, true);
    if (rq.code != P24_E4M3) refuse_type("q must be torch.float8_e4m3fn");
    const Shape s{rq.T, rq.d, rq.device};
    void* stream = stream_on(s.device);
    const int64_t group = whole(a[2], "group");
    const at::Tensor y = output(a[3], "out", {s.T, s.d}, q, at::kBFloat16);
    const Rows ry = rows(y, "out", &s);
    const Shape ss{s.T, groups_of(s.d, group), s.device};
    const Rows rs = rows(tensor(a[1], "scale"), "scale", &ss);
    if (rs.code != P24_F32) refuse_type("scale must be torch.float32");
    const p24_dequant8_args g{s.T, s.d, ry.code, group_of(group), rq.p, rq.ld, static_cast<const float*>(rs.p), rs.ld,
                              written(y), ry.ld};
    const int rc = p24_dequant8(&g, stream);
    return built(rc, {result(a[3], y)});
  });
}

// (tokens, W, scale, out) -> (status, out)
PyObject* py_embed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("embed", n, 4, [&] {
    const at::Tensor &tok = tensor(a[0], "tokens"), &W = tensor(a[1], "W");
    const Rows rw = rows(W, "W");
    if (tok.dim() != 1) refuse_value("tokens must be 1-D");
    const Shape s{tok.size(0), rw.d, rw.device};
    void* stream = stream_on(s.device);
    const void* t = vector(tok, "tokens", s.T, at::kInt, s.device);
    const at::Tensor y = output(a[3], "out", {s.T, s.d}, W, W.scalar_type());
    const Rows ry = rows(y, "out", &s);
    const p24_embed_args g{s.T, rw.T, s.d, rw.code, ry.code, number(a[2], "scale"), static_cast<const int32_t*>(t), rw.p, rw.ld,
                           written(y), ry.ld};
    const int rc = p24_embed(&g, stream);
    return built(rc, {result(a[3], y)});
  });
}

// (dY, tokens, V, scale, dW, accumulate, workspace) -> (status, dW)
PyObject* py_embed_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("embed_bwd", n, 7, [&] {
    const bool accumulate = truth(a[5], "accumulate");
    const at::Tensor& dY = tensor(a[0], "dY");
    const Rows ry = rows(dY, "dY");
    void* stream = stream_on(ry.device);
    const void* t = vector(tensor(a[1], "tokens"), "tokens", ry.T, at::kInt, ry.device);
    const int64_t V = whole(a[2], "V");
    if (accumulate && a[4] == Py_None) refuse_value("accumulate needs the dW to add to");
    const Shape sw{V, ry.d, ry.device};
    const at::Tensor dW = a[4] == Py_None && V < 1 ? dY : output(a[4], "dW", {V, ry.d}, dY, dY.scalar_type());
    const Rows rw = V < 1 ? Rows{} : rows(dW, "dW", &sw);
    const Scratch ws = scratch(a[6], p24_embed_bwd_workspace_size(ry.T, ry.d), dY);
    const p24_embed_bwd_args g{ry.T, V, ry.d, ry.code, rw.code, number(a[3], "scale"), accumulate ? 1 : 0,
                               static_cast<const int32_t*>(t), ry.p, ry.ld, V < 1 ? nullptr : written(dW), rw.ld};
    const int rc = p24_embed_bwd(&g, ws.p, ws.bytes, stream);
    return built(rc, {result(a[4], dW)});
  });
}

// A sequence of tensors as p24_tensor[]; holds a reference to it meanwhile. Elements are taken in the order of memory, so
// any tensor without holes will do.
struct List {
  PyObject* seq;
  std::vector<p24_tensor> v;
  int device = -1;
  at::Tensor first;
  List(PyObject* o, const char* name, bool write) : seq(PySequence_Fast(o, "")) {
    if (!seq) {
      PyErr_Clear();
      refuse_type(std::string(name) + " must be a list of tensors");
    }
    try {
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
      v.reserve(static_cast<size_t>(n));
      for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(seq, i), name);
        const int32_t code = code_of(t, name);
        if (i == 0) {
          first = t;
          device = cuda_index(t);
          if (device < 0) refuse_value(std::string(name) + " must be CUDA tensors (libprune24 has no CPU path)");
        }
        if (cuda_index(t) != device || !t.is_non_overlapping_and_dense())
          refuse_value(std::string(name) + " must be dense tensors on " + device_name(device));
        v.push_back(p24_tensor{write ? written(t) : const_cast<void*>(t.const_data_ptr()), t.numel(), code});
      }
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
  ~List() { Py_DECREF(seq); }
  List(const List&) = delete;
  const at::Tensor& at(size_t i) const { return THPVariable_Unpack(PySequence_Fast_GET_ITEM(seq, static_cast<Py_ssize_t>(i))); }
};

// Tensors that are scaled overlap no others: one that is listed twice would be scaled twice, or while it is read.
void require_apart(const std::vector<p24_tensor>& g, const std::vector<p24_tensor>& to) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Range> all;
  all.reserve(2 * g.size());
  auto add = [&](const p24_tensor& t, bool written) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(t.p);
    if (t.n > 0) all.push_back(Range{p, p + static_cast<uintptr_t>(t.n) * (t.dtype == P24_BF16 ? 2 : 4), written});
  };
  for (size_t i = 0; i < g.size(); ++i) {
    add(to[i], true);
    if (to[i].p != g[i].p) add(g[i], false);
  }
  auto before = [](const Range& a, const Range& b) { return a.begin < b.begin; };
  if (!std::is_sorted(all.begin(), all.end(), before)) std::sort(all.begin(), all.end(), before);
  uintptr_t written = 0, any = 0;
  for (const Range& r : all) {
    if (r.begin < (r.written ? any : written)) refuse_value("tensors that are scaled must not overlap others, nor be listed twice");
    any = std::max(any, r.end);
    if (r.written) written = std::max(written, r.end);
  }
}

// (gradients, out or None, max_norm or None for the norm alone, norm, workspace) -> (status, norm)
PyObject* py_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("grads", n, 5, [&] {
    const List g(a[0], "gradients", a[2] != Py_None && a[1] == Py_None);
    if (g.v.empty()) refuse_value("an empty list has no device to run on");
    void* stream = stream_on(g.device);
    const at::Tensor norm = output(a[3], "norm", {1}, g.first, at::kFloat);
    vector(norm, "norm", 1, at::kFloat, g.device);
    float* pn = static_cast<float*>(written(norm));
    const int64_t count = static_cast<int64_t>(g.v.size());
    const Scratch ws = scratch(a[4], p24_grad_norm_workspace_size(count), g.first);
    int rc;
    if (a[2] == Py_None) {
      rc = p24_grad_norm(g.v.data(), count, pn, ws.p, ws.bytes, stream);
    } else if (a[1] == Py_None) {
      require_apart(g.v, g.v);
      rc = p24_clip_grads(g.v.data(), nullptr, count, number(a[2], "max_norm"), pn, ws.p, ws.bytes, stream);
    } else {
      const List out(a[1], "out", true);
      if (out.v.size() != g.v.size())
        refuse_value(std::to_string(count) + " gradients, and " + std::to_string(out.v.size()) + " tensors to write to");
      if (out.device != g.device) refuse_value("out must be dense tensors on " + device_name(g.device));
      for (size_t i = 0; i < g.v.size(); ++i)
        if (out.v[i].n == g.v[i].n && !(out.at(i).is_contiguous() && g.at(i).is_contiguous()) &&
            (out.at(i).sizes() != g.at(i).sizes() || out.at(i).strides() != g.at(i).strides()))
          refuse_value("out must have the gradients' strides");
      require_apart(g.v, out.v);
      rc = p24_clip_grads(g.v.data(), out.v.data(), count, number(a[2], "max_norm"), pn, ws.p, ws.bytes, stream);
    }
    return built(rc, {result(a[3], norm)});
  });
}

PyObject* py_require_device(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("require_device", n, 2, [&] {
    require_device(static_cast<int>(whole(a[0], "tensors")), static_cast<int>(whole(a[1], "current")));
    return none();
  });
}

#define P24_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {P24_METHOD(rmsnorm), P24_METHOD(rmsnorm_bwd), P24_METHOD(dequant8), P24_METHOD(embed),
                         P24_METHOD(embed_bwd), P24_METHOD(grads), P24_METHOD(require_device), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_p24_torch", "Marshalling of torch tensors for libprune24.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__p24_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", P24_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
