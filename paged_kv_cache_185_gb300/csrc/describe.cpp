// describe.cpp -- torch tensors to wllm_tensor descriptors for the Python
// binding, as one small CPython module (_describe.so).
//
// describe((t0, t1, ...)) returns (owner, device, p0, p1, ...): the addresses
// of the tensors' descriptors, which live in the bytes object `owner`, and the
// index of the tensors' common CUDA device.  None stands for a tensor that is
// not given and stays None.  Filling a descriptor from Python takes about a
// microsecond a tensor, as long as a short kernel for a call of four; here it
// takes a few nanoseconds.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "wllm.h"

namespace {

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return WLLM_F32;
    case at::kHalf: return WLLM_F16;
    case at::kBFloat16: return WLLM_BF16;
    case at::kInt: return WLLM_I32;
    case at::kLong: return WLLM_I64;
    case at::kFloat8_e4m3fn: return WLLM_FP8_E4M3;
    case at::kByte: return WLLM_FP8_E4M3;  // raw E4M3 codes
    default: return -1;
  }
}

// One descriptor; `device` is the tensors' common device so far.  False with a
// Python error set when the tensor cannot be described.
bool fill(PyObject* o, const at::Tensor& t, wllm_tensor* d, int* device) {
  if (!t.is_cuda()) {
    PyErr_SetString(PyExc_ValueError, "all tensors must be CUDA tensors (the library has no CPU path)");
    return false;
  }
  if (*device >= 0 && t.get_device() != *device) {
    PyErr_SetString(PyExc_ValueError, "all tensors must be on one device");
    return false;
  }
  *device = static_cast<int>(t.get_device());
  if (t.dim() > WLLM_MAX_DIMS) {
    PyErr_SetString(PyExc_ValueError, "at most 4 dims");
    return false;
  }
  const int code = dtype_code(t.scalar_type());
  if (code < 0) {
    PyObject* dtype = PyObject_GetAttrString(o, "dtype");
    if (dtype != nullptr) {
      PyErr_SetObject(PyExc_KeyError, dtype);
      Py_DECREF(dtype);
    }
    return false;
  }
  d->data = t.numel() > 0 ? t.data_ptr() : nullptr;
  d->dtype = code;
  d->ndim = static_cast<int32_t>(t.dim());
  for (int k = 0; k < WLLM_MAX_DIMS; ++k) {
    d->shape[k] = k < t.dim() ? t.size(k) : 0;
    d->stride[k] = k < t.dim() ? t.stride(k) : 0;
  }
  return true;
}

PyObject* describe(PyObject*, PyObject* tensors) {
  if (!PyTuple_Check(tensors)) {
    PyErr_SetString(PyExc_TypeError, "describe takes a tuple of tensors");
    return nullptr;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(tensors);
  PyObject* owner = PyBytes_FromStringAndSize(nullptr, n * static_cast<Py_ssize_t>(sizeof(wllm_tensor)) + 8);
  if (owner == nullptr) return nullptr;
  PyObject* out = PyTuple_New(n + 2);
  if (out == nullptr) {
    Py_DECREF(owner);
    return nullptr;
  }
  PyTuple_SET_ITEM(out, 0, owner);
  const uintptr_t base = (reinterpret_cast<uintptr_t>(PyBytes_AS_STRING(owner)) + 7) & ~uintptr_t(7);
  wllm_tensor* d = reinterpret_cast<wllm_tensor*>(base);
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i, ++d) {
    PyObject* o = PyTuple_GET_ITEM(tensors, i);
    if (o == Py_None) {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out, i + 2, Py_None);
      continue;
    }
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
      break;
    }
    try {  // no C++ exception may leave a C function
      if (!fill(o, THPVariable_Unpack(o), d, &device)) break;
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
      break;
    }
    PyObject* address = PyLong_FromVoidPtr(d);
    if (address == nullptr) break;
    PyTuple_SET_ITEM(out, i + 2, address);
  }
  if (!PyErr_Occurred()) {
    PyObject* index = PyLong_FromLong(device);
    if (index != nullptr) {
      PyTuple_SET_ITEM(out, 1, index);
      return out;
    }
  }
  Py_DECREF(out);
  return nullptr;
}

PyMethodDef methods[] = {
    {"describe", describe, METH_O, "describe((t0, t1, ...)) -> (owner, device, address of t0's descriptor, ...)"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_describe", "wllm_tensor descriptors of torch tensors", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__describe() { return PyModule_Create(&module); }
