// The plain case of the decoder-side and clipping calls of api.py, marshalled in C++: tensors are looked at, outputs allocated by torch's CUDA
// allocator and the C entry point called on the current stream, without the interpreter between.
//
// For a token or a small model the host is what such a call takes: cross attention of one row is 5 us on the device, and took 17
// from Python through ctypes (2 of checks, 4 of allocations, 4 of ctypes, 2 of the launch, the rest the interpreter).
// Nothing is decided here that api.py does not decide: a call with anything out of the ordinary (a stream, a tensor of another
// device, type or layout, a refusal by the library) returns None before anything was launched, and api.py goes the long way,
// with its own checks and messages.  A failure that may come from behind a call's first launch raises what it raises on the long way
// (the package's WbError, torch's exceptions): a call made twice would scale gradients twice.
// Built beside libwb.so where torch's and Python's headers are; without it every call goes the long way.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

#include "../../include/wb.h"

namespace {

// Entry points of the libwb.so that the package has loaded, in the order of bind()'s arguments.
decltype(&wb_cross_attention) p_cross = nullptr;
decltype(&wb_cross_attention_backward) p_cross_backward = nullptr;
decltype(&wb_cross_attention_backward_workspace_bytes) p_cross_workspace = nullptr;
decltype(&wb_clip_grad_norm) p_clip = nullptr;
decltype(&wb_clip_grad_norm_workspace_bytes) p_clip_workspace = nullptr;
decltype(&wb_policy_loss) p_policy = nullptr;
decltype(&wb_policy_loss_workspace_bytes) p_policy_workspace = nullptr;
decltype(&wb_policy_loss_backward) p_policy_backward = nullptr;

PyObject* wb_error = nullptr;            // the package's exception

struct LongWay {};                       // not the plain case
struct Raised {};                        // with Python's exception set

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) throw LongWay();       // a tensor or a parameter; subclasses may be anything
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) throw LongWay();
  return t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw LongWay();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw LongWay();
  return v != 0;
}
// The current device, which all tensors of a call are on.
struct Here {
  c10::DeviceIndex index = c10::cuda::current_device();
  const at::Tensor& on(const at::Tensor& t) const {
    if (t.get_device() != index) throw LongWay();
    return t;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(index).stream(); }
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, index), std::nullopt));
  }
  at::Tensor workspace(size_t bytes) const { return empty({static_cast<int64_t>(std::max<size_t>(bytes, 256))}, at::kByte); }
};
// A contiguous tensor of this type and shape.
const at::Tensor& need(const Here& here, PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = here.on(tensor(o));
  if (t.scalar_type() != type || !t.is_contiguous() || t.sizes() != shape) throw LongWay();
  return t;
}

struct Rows {
  const void* p;
  int64_t batch, T, d, s0, s1;
};
Rows rows(const Here& here, PyObject* o) {
  const at::Tensor& t = here.on(tensor(o));
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3) throw LongWay();
  const Rows r{t.const_data_ptr(), t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
  if (r.d <= 0 || r.d % 64 || r.d > 65536 || t.stride(2) != 1 || r.T > (1 << 24) || r.batch > (1 << 30)) throw LongWay();
  return r;
}
const int32_t* lengths(const Here& here, PyObject* o, int64_t batch) {
  return o == Py_None ? nullptr : need(here, o, at::kInt, {batch}).const_data_ptr<int32_t>();
}

PyObject* wrap(std::initializer_list<const at::Tensor*> list) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(list.size()));
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* x : list) {
    PyObject* o = Py_None;
    if (x->defined()) o = THPVariable_Wrap(*x);
    else Py_INCREF(o);
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// Makes a call of the library, and goes on if it launched all it should.
template <typename F>
void call(bool& launched, const char* name, F f) {
  launched = true;
  const wb_status status = f();
  if (status == WB_OK) return;
  if (status == WB_EINVAL || status == WB_EUNSUPPORTED || status == WB_EWORKSPACE) throw LongWay();      // refusals: nothing was launched
  PyObject* e = PyObject_CallFunction(wb_error, "si", name, static_cast<int>(status));
  if (e) PyErr_SetObject(wb_error, e);
  Py_XDECREF(e);
  throw Raised();
}

// Every entry: None for LongWay and for exceptions before the call of the library (no device, an allocation that failed); null with Python's
// exception set for those behind it.
template <typename F>
PyObject* plain(F f) {
  HANDLE_TH_ERRORS
  bool launched = false;
  try {
    return f(launched);
  } catch (const LongWay&) {
    return none();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception&) {
    if (launched) throw;
    return none();
  }
  END_HANDLE_TH_ERRORS
}

PyObject* cross_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !p_cross) return none();
  return plain([&](bool& launched) -> PyObject* {
    const Here here;
    const Rows q = rows(here, a[0]), k = rows(here, a[1]), v = rows(here, a[2]);
    if (k.batch != q.batch || v.batch != q.batch || v.T != k.T || v.d != k.d || q.d % k.d) throw LongWay();
    const float scale = static_cast<float>(number(a[3]));
    const int32_t *ql = lengths(here, a[4], q.batch), *kl = lengths(here, a[5], q.batch);
    const at::Tensor out = here.empty({q.batch, q.T, q.d}, at::kBFloat16), lse = here.empty({q.batch, q.d / 64, q.T}, at::kFloat);
    call(launched, "wb_cross_attention", [&] {
      return p_cross(q.p, q.s0, q.s1, k.p, k.s0, k.s1, v.p, v.s0, v.s1, ql, kl, static_cast<int>(q.batch), static_cast<int>(q.T),
                     static_cast<int>(k.T), static_cast<int>(q.d / 64), static_cast<int>(k.d / 64), scale, out.mutable_data_ptr(),
                     lse.mutable_data_ptr<float>(), here.stream());
    });
    return wrap({&out, &lse});
  });
}

PyObject* cross_attention_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11 || !p_cross_backward) return none();
  return plain([&](bool& launched) -> PyObject* {
    const Here here;
    const Rows g = rows(here, a[0]), q = rows(here, a[1]), k = rows(here, a[2]), v = rows(here, a[3]);
    if (k.batch != q.batch || v.batch != q.batch || v.T != k.T || v.d != k.d || q.d % k.d || g.batch != q.batch || g.T != q.T || g.d != q.d)
      throw LongWay();
    const at::Tensor& out = need(here, a[4], at::kBFloat16, {q.batch, q.T, q.d});
    const at::Tensor& lse = need(here, a[5], at::kFloat, {q.batch, q.d / 64, q.T});
    const float scale = static_cast<float>(number(a[6]));
    const int32_t *ql = lengths(here, a[7], q.batch), *kl = lengths(here, a[8], q.batch);
    const int H = static_cast<int>(q.d / 64);
    at::Tensor dq, dk, dv;
    if (truth(a[9])) dq = here.empty({q.batch, q.T, q.d}, at::kBFloat16);
    if (truth(a[10])) {
      dk = here.empty({k.batch, k.T, k.d}, at::kBFloat16);
      dv = here.empty({k.batch, k.T, k.d}, at::kBFloat16);
    }
    const at::Tensor ws = here.workspace(p_cross_workspace(static_cast<int>(q.batch), static_cast<int>(q.T), H));
    auto at_ = [](const at::Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; };
    call(launched, "wb_cross_attention_backward", [&] {
      return p_cross_backward(g.p, g.s0, g.s1, q.p, q.s0, q.s1, k.p, k.s0, k.s1, v.p, v.s0, v.s1, out.const_data_ptr(),
                              lse.const_data_ptr<float>(), ql, kl, static_cast<int>(q.batch), static_cast<int>(q.T), static_cast<int>(k.T), H,
                              static_cast<int>(k.d / 64), scale, at_(dq), at_(dk), at_(dv), ws.mutable_data_ptr(),
                              static_cast<size_t>(ws.numel()), here.stream());
    });
    return wrap({&dq, &dk, &dv});
  });
}

int32_t element_type(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return WB_BF16;
    case at::kHalf: return WB_F16;
    case at::kFloat: return WB_F32;
    default: throw LongWay();
  }
}

// (grads, max_norm, out): out None: the norm alone; grads itself: in place
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3 || !p_clip || !PyList_CheckExact(a[0]) || (a[2] != Py_None && !PyList_CheckExact(a[2]))) return none();
  return plain([&](bool& launched) -> PyObject* {
    const Here here;
    const Py_ssize_t count = PyList_GET_SIZE(a[0]);
    const bool write = a[2] != Py_None;
    if (count < 1 || count > WB_CLIP_MAX_TENSORS || (write && PyList_GET_SIZE(a[2]) != count)) throw LongWay();
    std::vector<const void*> grads(count);
    std::vector<void*> outs(write ? count : 0);
    std::vector<int64_t> numel(count);
    std::vector<int32_t> types(count), out_types(write ? count : 0);
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& t = here.on(tensor(PyList_GET_ITEM(a[0], i)));
      if (!t.is_contiguous()) throw LongWay();
      grads[i] = t.const_data_ptr();
      numel[i] = t.numel();
      types[i] = element_type(t);
      if (!write) continue;
      const at::Tensor& o = a[2] == a[0] ? t : here.on(tensor(PyList_GET_ITEM(a[2], i)));
      if (!o.is_contiguous() || o.sizes() != t.sizes()) throw LongWay();
      outs[i] = o.mutable_data_ptr();
      out_types[i] = element_type(o);
      if (out_types[i] != types[i] && out_types[i] != WB_F32) throw LongWay();
    }
    const at::Tensor norm = here.empty({}, at::kFloat), ws = here.workspace(p_clip_workspace(static_cast<int>(count)));
    call(launched, "wb_clip_grad_norm", [&] {
      return p_clip(grads.data(), write ? outs.data() : nullptr, numel.data(), types.data(), write ? out_types.data() : nullptr,
                    static_cast<int>(count), static_cast<float>(number(a[1])), norm.mutable_data_ptr<float>(), ws.mutable_data_ptr(),
                    static_cast<size_t>(ws.numel()), here.stream());
    });
    return THPVariable_Wrap(norm);
  });
}

struct Policy {
  const float *nll, *old_nll, *ref, *adv;
  const int64_t* labels;
  int64_t S, T;
  int per_token;
};
Policy policy(const Here& here, PyObject* nll, PyObject* old_nll, PyObject* adv, PyObject* labels, PyObject* ref) {
  const at::Tensor& t = here.on(tensor(nll));
  if (t.dim() != 2) throw LongWay();
  const int64_t S = t.size(0), T = t.size(1);
  Policy p;
  p.S = S;
  p.T = T;
  p.nll = need(here, nll, at::kFloat, {S, T}).const_data_ptr<float>();
  p.old_nll = need(here, old_nll, at::kFloat, {S, T}).const_data_ptr<float>();
  p.labels = need(here, labels, at::kLong, {S, T}).const_data_ptr<int64_t>();
  p.ref = ref == Py_None ? nullptr : need(here, ref, at::kFloat, {S, T}).const_data_ptr<float>();
  p.per_token = tensor(adv).dim() == 2;
  p.adv = (p.per_token ? need(here, adv, at::kFloat, {S, T}) : need(here, adv, at::kFloat, {S})).const_data_ptr<float>();
  return p;
}

// (nll, old_nll, advantage, labels, ref_nll, clip_low, clip_high, kl_weight, per_sequence)
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9 || !p_policy) return none();
  return plain([&](bool& launched) -> PyObject* {
    const Here here;
    const Policy p = policy(here, a[0], a[1], a[2], a[3], a[4]);
    const int per_sequence = truth(a[8]);
    const at::Tensor stats = here.empty({3}, at::kFloat), weight = here.empty({p.S}, at::kFloat);
    const size_t bytes = p_policy_workspace(p.S, p.T);
    at::Tensor ws;
    if (bytes) ws = here.workspace(bytes);
    call(launched, "wb_policy_loss", [&] {
      return p_policy(p.nll, p.old_nll, p.ref, p.adv, p.per_token, p.labels, p.S, p.T, number(a[5]), number(a[6]),
                      static_cast<float>(number(a[7])), per_sequence, stats.mutable_data_ptr<float>(), weight.mutable_data_ptr<float>(),
                      bytes ? ws.mutable_data_ptr() : nullptr, bytes ? static_cast<size_t>(ws.numel()) : 0, here.stream());
    });
    return wrap({&stats, &weight});
  });
}

// (dloss, nll, old_nll, advantage, labels, weight, ref_nll, clip_low, clip_high, kl_weight)
PyObject* policy_loss_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10 || !p_policy_backward) return none();
  return plain([&](bool& launched) -> PyObject* {
    const Here here;
    const Policy p = policy(here, a[1], a[2], a[3], a[4], a[6]);
    const at::Tensor& dloss = here.on(tensor(a[0]));
    if (dloss.scalar_type() != at::kFloat || dloss.numel() != 1) throw LongWay();
    const at::Tensor& weight = need(here, a[5], at::kFloat, {p.S});
    const at::Tensor dnll = here.empty({p.S, p.T}, at::kFloat);
    call(launched, "wb_policy_loss_backward", [&] {
      return p_policy_backward(dloss.const_data_ptr<float>(), p.nll, p.old_nll, p.ref, p.adv, p.per_token, p.labels,
                               weight.const_data_ptr<float>(), p.S, p.T, number(a[7]), number(a[8]), static_cast<float>(number(a[9])),
                               dnll.mutable_data_ptr<float>(), here.stream());
    });
    return THPVariable_Wrap(dnll);
  });
}

// The package's exception, and addresses of the entry points, as integers.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[8];
  if (n != 9 || !PyType_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "bind: an exception and eight addresses expected");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XDECREF(wb_error);
  wb_error = a[0];
  p_cross = reinterpret_cast<decltype(p_cross)>(p[0]);
  p_cross_backward = reinterpret_cast<decltype(p_cross_backward)>(p[1]);
  p_cross_workspace = reinterpret_cast<decltype(p_cross_workspace)>(p[2]);
  p_clip = reinterpret_cast<decltype(p_clip)>(p[3]);
  p_clip_workspace = reinterpret_cast<decltype(p_clip_workspace)>(p[4]);
  p_policy = reinterpret_cast<decltype(p_policy)>(p[5]);
  p_policy_workspace = reinterpret_cast<decltype(p_policy_workspace)>(p[6]);
  p_policy_backward = reinterpret_cast<decltype(p_policy_backward)>(p[7]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(cross_attention), FAST(cross_attention_backward), FAST(clip_grad_norm), FAST(policy_loss),
                         FAST(policy_loss_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "wb_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_wb_host(void) { return PyModule_Create(&module); }
