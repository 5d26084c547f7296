// callutil.h -- what the C++ sides of the operators' Python calls share: reading
// tensors and numbers of the usual kind, without raising.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/replayssm_hybrid.h"

namespace {

using Tensor = at::Tensor;

PyObject* none() { Py_RETURN_NONE; }

// The tensor, or nullptr for anything else.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// All tensors on the current device, and none wants a gradient or has a tangent (nullptr: not given); its index, or -1.
template <int N>
int device_of(const Tensor* const (&ts)[N]) {
  const int d = c10::cuda::current_device();
  const bool grad = c10::GradMode::is_enabled();
  for (const Tensor* t : ts)
    if (t != nullptr && !(t->is_cuda() && t->get_device() == d && !(grad && t->requires_grad()) && !t->_fw_grad(0).defined())) return -1;
  return d;
}

int input_code(const Tensor& t) {
  const auto s = t.scalar_type();
  return s == at::kBFloat16 ? RSM_BF16 : s == at::kFloat ? RSM_F32 : -1;
}

// contiguous [n] of a type
bool vector(const Tensor& t, int64_t n, at::ScalarType type) {
  return t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && (n <= 1 || t.stride(0) == 1);
}

bool is(const Tensor& t, at::IntArrayRef sizes, at::ScalarType type) {
  return t.scalar_type() == type && t.sizes() == sizes && t.is_contiguous();
}

bool fits(int64_t v) { return v >= 0 && v <= 0x7FFFFFFF; }

// a Python integer of 32 bits
bool int32(PyObject* o, int32_t* v) {
  const long long n = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *v = static_cast<int32_t>(n);
  return *v == n;
}

void* ptr(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

Tensor like(const Tensor& x) { return at::empty(x.sizes(), x.options()); }

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {  // the Python side meets the same, and says so
    PyErr_Clear();
    return none();
  }
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}

}  // namespace
