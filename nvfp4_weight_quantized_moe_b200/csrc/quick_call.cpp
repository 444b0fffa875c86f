// The short way of the Python binding for the operators around the forward.
//
// A decode step makes these calls on tensors whose kernels take 2 to 5 us; looking
// at five tensors from Python and going through ctypes takes 3 us on top of the
// launch's 2.4.  Each function here looks at the same things in C++ and calls the
// library's entry point (the address that _binding.py hands over).  It returns
// the entry point's status, or -1 without a call where something is not as usual:
// a strided view, another device than the current one, a wrong type or shape.
// _binding.py then takes the long way, which knows strides and devices and says
// what is wrong.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/nvfp4_moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

decltype(&nvfp4_moe_route_topk) g_route = nullptr;
decltype(&nvfp4_moe_add_rms_norm) g_norm = nullptr;
decltype(&nvfp4_moe_int8_matmul) g_int8 = nullptr;

// Thrown and caught here only: not the usual call.
struct Unusual {};

const Tensor* optional(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Unusual{};
  return &THPVariable_Unpack(o);
}

const Tensor& required(PyObject* o) {
  const Tensor* t = optional(o);
  if (t == nullptr) throw Unusual{};
  return *t;
}

// A contiguous tensor on the device.
void* on(const Tensor& t, int dev) {
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) throw Unusual{};
  return t.data_ptr();
}

void* vector(const Tensor& t, int64_t n, ScalarType type, int dev) {
  if (t.dim() != 1 || t.size(0) != n || t.scalar_type() != type) throw Unusual{};
  return on(t, dev);
}

void* matrix(const Tensor& t, int64_t m, int64_t n, ScalarType type, int dev) {
  if (t.dim() != 2 || t.size(0) != m || t.size(1) != n || t.scalar_type() != type) throw Unusual{};
  return on(t, dev);
}

int32_t float_type(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return NVFP4_MOE_BF16;
  if (t.scalar_type() == at::kFloat) return NVFP4_MOE_F32;
  throw Unusual{};
}

// The current device, which has to be the leading tensor's.
int device_of(const Tensor& t) {
  if (!t.is_cuda() || t.dim() != 2) throw Unusual{};
  const int dev = t.get_device();
  if (c10::cuda::current_device() != dev) throw Unusual{};
  return dev;
}

uint32_t u32(int64_t v) {
  if (v < 0 || v > 0xffffffffll) throw Unusual{};
  return (uint32_t)v;
}

uint32_t u32(PyObject* o) {
  const unsigned long v = PyLong_AsUnsignedLong(o);
  if (PyErr_Occurred()) throw Unusual{};
  return u32((int64_t)v);
}

int32_t truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Unusual{};
  return v;
}

float f32(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw Unusual{};
  return (float)v;
}

template <typename F, typename Args>
int launch(F entry, const Args& args, int dev) {
  cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = entry(&args, stream);
  Py_END_ALLOW_THREADS;
  return status;
}

// Runs `call` and turns whatever it throws into -1.
template <typename Call>
PyObject* answer(Py_ssize_t n, Py_ssize_t wanted, Call call) {
  long status = -1;
  if (n == wanted) {
    try {
      status = call();
    } catch (...) {
      PyErr_Clear();
    }
  }
  return PyLong_FromLong(status);
}

// (logits, topk_ids, topk_weights, bias, score, num_groups, topk_groups, group_top,
// renormalize, scale)
PyObject* route_topk(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return answer(n, 10, [&] {
    const Tensor &logits = required(v[0]), &ids = required(v[1]);
    const int dev = device_of(logits);
    nvfp4_moe_route_args a{};
    const int64_t m = logits.size(0), e = logits.size(1), k = ids.dim() == 2 ? ids.size(1) : -1;
    a.logits_type = float_type(logits);
    a.logits = on(logits, dev);
    a.topk_ids = static_cast<int32_t*>(matrix(ids, m, k, at::kInt, dev));
    a.topk_weights = static_cast<float*>(matrix(required(v[2]), m, k, at::kFloat, dev));
    if (const Tensor* bias = optional(v[3])) a.bias = static_cast<float*>(vector(*bias, e, at::kFloat, dev));
    a.ld = (uint64_t)e;
    a.num_tokens = u32(m);
    a.num_experts = u32(e);
    a.topk = u32(k);
    a.score = (int32_t)u32(v[4]);
    a.num_groups = u32(v[5]);
    a.topk_groups = u32(v[6]);
    a.group_top = u32(v[7]);
    a.renormalize = truth(v[8]);
    a.scale = f32(v[9]);
    return launch(g_route, a, dev);
  });
}

// (x, weight, eps, out, residual, residual_out, q, q_scale)
PyObject* add_rms_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return answer(n, 8, [&] {
    const Tensor &x = required(v[0]), &weight = required(v[1]);
    const int dev = device_of(x);
    nvfp4_moe_norm_args a{};
    const int64_t m = x.size(0), h = x.size(1);
    a.x_type = float_type(x);
    a.x = on(x, dev);
    a.weight_type = float_type(weight);
    a.weight = vector(weight, h, weight.scalar_type(), dev);
    a.eps = f32(v[2]);
    if (const Tensor* out = optional(v[3])) a.out = static_cast<uint16_t*>(matrix(*out, m, h, at::kBFloat16, dev));
    const Tensor* residual = optional(v[4]);
    if (residual != nullptr) {
      a.residual_type = float_type(*residual);
      a.residual = matrix(*residual, m, h, residual->scalar_type(), dev);
    }
    if (const Tensor* out = optional(v[5])) {
      if (residual == nullptr) throw Unusual{};
      a.residual_out = matrix(*out, m, h, residual->scalar_type(), dev);
    }
    const Tensor *q = optional(v[6]), *scale = optional(v[7]);
    if ((q == nullptr) != (scale == nullptr)) throw Unusual{};
    if (q != nullptr) {
      const ScalarType type = q->scalar_type();
      if (type != at::kChar && type != at::kFloat8_e4m3fn) throw Unusual{};
      a.q_type = type == at::kChar ? NVFP4_MOE_INT8 : NVFP4_MOE_E4M3;
      a.q = matrix(*q, m, h, type, dev);
      a.q_scale = static_cast<float*>(vector(*scale, m, at::kFloat, dev));
    }
    a.ldx = a.ldr = (uint64_t)h;
    a.num_rows = u32(m);
    a.hidden = u32(h);
    return launch(g_norm, a, dev);
  });
}

// (x_q, x_scale, w_q, w_scale, out, bias)
PyObject* int8_matmul(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return answer(n, 6, [&] {
    const Tensor &x = required(v[0]), &w = required(v[2]), &out = required(v[4]);
    const int dev = device_of(x);
    if (w.dim() != 2) throw Unusual{};
    nvfp4_moe_int8_args a{};
    const int64_t m = x.size(0), k = x.size(1), c = w.size(0);
    a.x = static_cast<int8_t*>(matrix(x, m, k, at::kChar, dev));
    a.x_scale = static_cast<float*>(vector(required(v[1]), m, at::kFloat, dev));
    a.w = static_cast<int8_t*>(matrix(w, c, k, at::kChar, dev));
    a.w_scale = static_cast<float*>(vector(required(v[3]), c, at::kFloat, dev));
    a.out_type = float_type(out);
    a.out = matrix(out, m, c, out.scalar_type(), dev);
    if (const Tensor* bias = optional(v[5])) a.bias = static_cast<float*>(vector(*bias, c, at::kFloat, dev));
    a.ldx = (uint64_t)k;
    a.ldo = (uint64_t)c;
    a.num_tokens = u32(m);
    a.n = u32(c);
    a.k = u32(k);
    return launch(g_int8, a, dev);
  });
}

// (route_topk, add_rms_norm, int8_matmul): the entry points' addresses.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long route, norm, int8;
  if (!PyArg_ParseTuple(args, "KKK", &route, &norm, &int8)) return nullptr;
  g_route = reinterpret_cast<decltype(g_route)>(route);
  g_norm = reinterpret_cast<decltype(g_norm)>(norm);
  g_int8 = reinterpret_cast<decltype(g_int8)>(int8);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"route_topk", method(route_topk), METH_FASTCALL, nullptr},
    {"add_rms_norm", method(add_rms_norm), METH_FASTCALL, nullptr},
    {"int8_matmul", method(int8_matmul), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quick_call", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__quick_call() { return PyModule_Create(&module); }
