// The short way from Python to the calls around the linear.  These kernels take two to
// twenty microseconds, and a call through ctypes spends ten on the host: its checks in
// Python, its output tensors, its arguments one by one.  Here the same checks run on the
// tensors themselves (norm of one token 10.1 -> 5 us a call).
//
// A function here serves the usual call alone: contiguous tensors of the right types and
// sizes on the current device, its current stream, outputs of its own.  For anything else
// it returns None and does nothing: the Python functions then say what is wrong, or take
// the call.  An int is a status of the library that is not MACAQ_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "macaq.h"

namespace {

using at::Tensor;

// An argument that is a tensor, or absent (None).
struct Arg {
  const Tensor* t = nullptr;
  bool ok = true;
  explicit Arg(PyObject* o) {
    if (o == Py_None) return;
    if (THPVariable_Check(o)) t = &THPVariable_Unpack(o);
    else ok = false;
  }
  // present, of this type, contiguous, on device dev
  bool is(at::ScalarType type, int dev) const {
    return t != nullptr && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->is_contiguous();
  }
  bool is(at::ScalarType type, int dev, at::IntArrayRef shape) const { return is(type, dev) && t->sizes() == shape; }
  bool absent_or(at::ScalarType type, int dev, at::IntArrayRef shape) const {
    return ok && (t == nullptr || is(type, dev, shape));
  }
  template <typename T>
  T* ptr() const {
    return t != nullptr ? static_cast<T*>(t->data_ptr()) : nullptr;
  }
};

// The device of the call, its first tensor's, if that is the current one; else -1.
int device_of(const Arg& a) {
  if (a.t == nullptr || !a.t->is_cuda()) return -1;
  const int dev = a.t->get_device();
  return dev == c10::cuda::current_device() ? dev : -1;
}
Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// bf16 or fp32: its code in the library, else -1.
int element_type(const Arg& a) {
  if (a.t == nullptr) return -1;
  if (a.t->scalar_type() == at::kBFloat16) return MACAQ_BF16;
  return a.t->scalar_type() == at::kFloat ? MACAQ_FP32 : -1;
}
bool integer(PyObject* o, int64_t& v) {
  if (!PyLong_CheckExact(o)) return false;
  v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred() != nullptr) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool number(PyObject* o, float& v) {
  if (!PyFloat_CheckExact(o)) return false;
  v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}
PyObject* wrapped(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// block_norm(h, y, w_post, gate, rows_per_gate, w_pre, scale, eps, weight_offset) -> (h', n)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) Py_RETURN_NONE;
  const Arg h(a[0]), y(a[1]), w_post(a[2]), gate(a[3]), w_pre(a[5]);
  const int dev = device_of(h);
  if (dev < 0) Py_RETURN_NONE;
  const int h_type = element_type(h);
  float scale, eps, offset;
  if (h_type < 0 || !h.is(h.t->scalar_type(), dev) || h.t->dim() != 2 || !number(a[6], scale) || !number(a[7], eps) ||
      !number(a[8], offset))
    Py_RETURN_NONE;
  const int64_t M = h.t->size(0), C = h.t->size(1);
  if (!y.is(at::kBFloat16, dev, h.t->sizes()) || !w_post.absent_or(at::kFloat, dev, {C}) ||
      !w_pre.absent_or(at::kFloat, dev, {C}) || !gate.ok)
    Py_RETURN_NONE;
  int gate_type = MACAQ_BF16;
  int64_t per = 1;
  if (gate.t != nullptr) {
    gate_type = element_type(gate);
    if (gate_type < 0 || gate.t->dim() != 2 || (a[4] != Py_None && !integer(a[4], per)) || per < 1 ||
        !gate.is(gate.t->scalar_type(), dev, {M > 0 ? (M - 1) / per + 1 : 0, C}))
      Py_RETURN_NONE;
  }
  Tensor out_h = empty(h.t->sizes(), h.t->scalar_type(), dev), out_n;
  if (w_pre.t != nullptr) out_n = empty(h.t->sizes(), at::kBFloat16, dev);
  const int st = macaq_block_norm(h.ptr<void>(), h_type, y.ptr<uint16_t>(), w_post.ptr<float>(), gate.ptr<void>(),
                                  gate_type, per, w_pre.ptr<float>(), scale, eps, offset, out_h.data_ptr(),
                                  out_n.defined() ? static_cast<uint16_t*>(out_n.data_ptr()) : nullptr, M, C,
                                  stream_of(dev));
  if (st != MACAQ_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrapped(std::move(out_h)));
  if (out_n.defined()) {
    PyTuple_SET_ITEM(r, 1, wrapped(std::move(out_n)));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 1, Py_None);
  }
  return r;
}

// moe_route(logits, k, score, renorm, scale) -> (ids, weights, counts, order)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) Py_RETURN_NONE;
  const Arg logits(a[0]);
  const int dev = device_of(logits);
  if (dev < 0) Py_RETURN_NONE;
  const int type = element_type(logits);
  int64_t k, score;
  float scale;
  const int renorm = PyObject_IsTrue(a[3]);
  if (renorm < 0) return nullptr;
  if (type < 0 || !logits.is(logits.t->scalar_type(), dev) || logits.t->dim() != 2 || !integer(a[1], k) ||
      !integer(a[2], score) || score < 0 || score > 1 || !number(a[4], scale))
    Py_RETURN_NONE;
  const int64_t T = logits.t->size(0), E = logits.t->size(1);
  if (T < 1 || k < 1 || k > E || k > 32) Py_RETURN_NONE;
  Tensor ids = empty({T, k}, at::kInt, dev), weights = empty({T, k}, at::kFloat, dev), counts = empty({E}, at::kLong, dev),
         order = empty({T * k}, at::kInt, dev), ws;
  const size_t need = macaq_route_workspace_bytes(T, E);
  if (need > 0) ws = empty({static_cast<int64_t>(need)}, at::kByte, dev);
  const int st = macaq_moe_route(logits.ptr<void>(), type, T, E, k, static_cast<int>(score), renorm, scale,
                                 static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(weights.data_ptr()),
                                 static_cast<int64_t*>(counts.data_ptr()), static_cast<int32_t*>(order.data_ptr()),
                                 need > 0 ? ws.data_ptr() : nullptr, need, stream_of(dev));
  if (st != MACAQ_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(4);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrapped(std::move(ids)));
  PyTuple_SET_ITEM(r, 1, wrapped(std::move(weights)));
  PyTuple_SET_ITEM(r, 2, wrapped(std::move(counts)));
  PyTuple_SET_ITEM(r, 3, wrapped(std::move(order)));
  return r;
}

// moe_mm(x, logits, D_up, Wq_up, Ws_up, D_down, Wq_down, Ws_down, inner, k, score, renorm, scale, act_type) -> y
PyObject* moe_mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  const Arg x(a[0]), logits(a[1]), d_up(a[2]), q_up(a[3]), s_up(a[4]), d_down(a[5]), q_down(a[6]), s_down(a[7]);
  const int dev = device_of(x);
  if (dev < 0) Py_RETURN_NONE;
  const int type = element_type(logits);
  int64_t inner, k, score, act;
  float scale;
  const int renorm = PyObject_IsTrue(a[11]);
  if (renorm < 0) return nullptr;
  if (type < 0 || !x.is(at::kBFloat16, dev) || x.t->dim() != 2 || !integer(a[8], inner) || !integer(a[9], k) ||
      !integer(a[10], score) || score < 0 || score > 1 || !number(a[12], scale) || !integer(a[13], act) || act < 0 || act > 5)
    Py_RETURN_NONE;
  const int64_t T = x.t->size(0), H = x.t->size(1);
  if (logits.t->dim() != 2 || logits.t->size(0) != T || !logits.is(logits.t->scalar_type(), dev)) Py_RETURN_NONE;
  const int64_t E = logits.t->size(1);
  auto image = [&](const Arg& w, size_t bytes) {
    return bytes > 0 && w.is(at::kByte, dev) && static_cast<size_t>(w.t->numel()) >= bytes;
  };
  const size_t need = macaq_moe_workspace_bytes(T, k, inner);
  if (need == 0 || !d_up.is(at::kFloat, dev, {E, H}) || !d_down.is(at::kFloat, dev, {E, inner}) ||
      !image(q_up, macaq_weight_code_bytes(E, 2 * inner, H)) || !image(s_up, macaq_weight_scale_bytes(E, 2 * inner, H)) ||
      !image(q_down, macaq_weight_code_bytes(E, H, inner)) || !image(s_down, macaq_weight_scale_bytes(E, H, inner)))
    Py_RETURN_NONE;
  Tensor y = empty({T, H}, at::kBFloat16, dev), ws = empty({static_cast<int64_t>(need)}, at::kByte, dev);
  const int st = macaq_moe_mm(x.ptr<uint16_t>(), logits.ptr<void>(), type, d_up.ptr<float>(), q_up.ptr<uint8_t>(),
                              s_up.ptr<uint8_t>(), d_down.ptr<float>(), q_down.ptr<uint8_t>(), s_down.ptr<uint8_t>(), T, E,
                              k, H, inner, static_cast<int>(score), renorm, scale, static_cast<int>(act),
                              static_cast<uint16_t*>(y.data_ptr()), ws.data_ptr(), need, nullptr, stream_of(dev));
  if (st != MACAQ_OK) return PyLong_FromLong(st);
  return wrapped(std::move(y));
}

// C++ exceptions (an allocation that fails) become the Python ones torch's own calls raise.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<block_norm>("block_norm"), method<moe_route>("moe_route"), method<moe_mm>("moe_mm"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
