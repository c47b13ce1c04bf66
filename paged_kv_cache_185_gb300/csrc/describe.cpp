// describe.cpp -- the Python binding's calls of entry points that take tensors,
// as one small CPython module (_describe.so).
//
// bind(name, address) returns a capsule for the entry point of that name, whose
// type is the header's.  call(entry, (t0, t1, ...), scalars...) fills the
// tensors' wllm_tensor descriptors (None: a null pointer), calls the entry on
// the current stream of the tensors' device with the interpreter's lock
// released, and returns the status.  Filling a descriptor from Python takes
// about a microsecond a tensor, as long as a short kernel for a call of four.
// One call from Python, by ctypes on addresses of descriptors filled here and by
// call(): 5 tensors 4.2 and 3.0 us, 7 tensors 5.6 and 3.9, 11 tensors 6.1 and
// 4.3, of which the launch itself is 2.1.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <exception>
#include <tuple>
#include <type_traits>
#include <utility>

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

constexpr int kMostTensors = 16;

// The arguments of one call, taken in the order of the entry's parameters.
struct Arguments {
  const wllm_tensor* tensors[kMostTensors];
  PyObject* const* scalars;
  wllm_stream stream;
  int tensor = 0, scalar = 0;

  template <typename A>
  A next();
};

template <>
const wllm_tensor* Arguments::next<const wllm_tensor*>() {
  return tensors[tensor++];
}
template <>
int Arguments::next<int>() {
  const long x = PyLong_AsLong(scalars[scalar++]);
  if (!PyErr_Occurred() && (x < INT_MIN || x > INT_MAX)) PyErr_SetString(PyExc_OverflowError, "an int argument out of range");
  return static_cast<int>(x);
}
template <>
float Arguments::next<float>() {
  return static_cast<float>(PyFloat_AsDouble(scalars[scalar++]));
}
template <>
const wllm_rotary* Arguments::next<const wllm_rotary*>() {
  return static_cast<const wllm_rotary*>(PyLong_AsVoidPtr(scalars[scalar++]));
}
template <>
wllm_stream Arguments::next<wllm_stream>() {
  return stream;
}

template <typename F>
struct Entry;
template <typename... A>
struct Entry<int(A...)> {
  static constexpr int kTensors = (0 + ... + (std::is_same<A, const wllm_tensor*>::value ? 1 : 0));
  static constexpr int kScalars = static_cast<int>(sizeof...(A)) - kTensors - 1;
  static_assert(kTensors <= kMostTensors, "room for the descriptors");
  // False with a Python error set: nothing was called.
  static bool run(void* address, Arguments& arguments, int* status) {
    const std::tuple<A...> values{arguments.next<A>()...};  // braces: from left to right
    if (PyErr_Occurred()) return false;
    Py_BEGIN_ALLOW_THREADS;
    *status = std::apply(reinterpret_cast<int (*)(A...)>(address), values);
    Py_END_ALLOW_THREADS;
    return true;
  }
};

struct Kind {
  const char* name;
  int tensors, scalars;
  bool (*run)(void*, Arguments&, int*);
};

#define WLLM_ENTRY(name) \
  Kind { #name, Entry<decltype(name)>::kTensors, Entry<decltype(name)>::kScalars, &Entry<decltype(name)>::run }
const Kind kinds[] = {
    WLLM_ENTRY(wllm_reshape_and_cache),
    WLLM_ENTRY(wllm_paged_attention_decode),
    WLLM_ENTRY(wllm_decode_step),
    WLLM_ENTRY(wllm_reshape_and_cache_fp8),
    WLLM_ENTRY(wllm_paged_attention_decode_fp8),
    WLLM_ENTRY(wllm_decode_step_fp8),
    WLLM_ENTRY(wllm_paged_attention_prefill),
    WLLM_ENTRY(wllm_paged_attention_prefill_fp8),
    WLLM_ENTRY(wllm_paged_attention_decode_noalloc),
    WLLM_ENTRY(wllm_rotate_and_cache),
    WLLM_ENTRY(wllm_rotate_and_cache_fp8),
    WLLM_ENTRY(wllm_update_key_bounds),
    WLLM_ENTRY(wllm_select_blocks),
    WLLM_ENTRY(wllm_paged_attention_decode_sparse),
    WLLM_ENTRY(wllm_paged_attention_decode_sparse_fp8),
    WLLM_ENTRY(wllm_assign_slots),
    WLLM_ENTRY(wllm_reshape_and_cache_block_scaled),
    WLLM_ENTRY(wllm_paged_attention_decode_block_scaled),
    WLLM_ENTRY(wllm_paged_attention_prefill_block_scaled),
};
#undef WLLM_ENTRY

struct Bound {
  const Kind* kind;
  void* address;
};
constexpr const char* kCapsule = "wllm entry";

PyObject* bind(PyObject*, PyObject* args) {
  const char* name;
  PyObject* address;
  if (!PyArg_ParseTuple(args, "sO", &name, &address)) return nullptr;
  void* at = PyLong_AsVoidPtr(address);
  if (PyErr_Occurred()) return nullptr;
  for (const Kind& k : kinds)
    if (at != nullptr && std::strcmp(k.name, name) == 0)
      return PyCapsule_New(new Bound{&k, at}, kCapsule, [](PyObject* capsule) {
        delete static_cast<Bound*>(PyCapsule_GetPointer(capsule, kCapsule));
      });
  PyErr_Format(PyExc_KeyError, "%s is no entry point that takes tensors first", name);
  return nullptr;
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 2 || !PyTuple_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "call takes an entry, a tuple of tensors and scalars");
    return nullptr;
  }
  const Bound* entry = static_cast<const Bound*>(PyCapsule_GetPointer(args[0], kCapsule));
  if (entry == nullptr) return nullptr;
  const Kind& kind = *entry->kind;
  if (PyTuple_GET_SIZE(args[1]) != kind.tensors || n - 2 != kind.scalars) {
    PyErr_Format(PyExc_TypeError, "%s takes %d tensors and %d scalars", kind.name, kind.tensors, kind.scalars);
    return nullptr;
  }
  wllm_tensor descriptors[kMostTensors];
  Arguments arguments;
  arguments.scalars = args + 2;
  int device = -1, status = 0;
  try {  // no C++ exception may leave a C function
    for (int i = 0; i < kind.tensors; ++i) {
      PyObject* o = PyTuple_GET_ITEM(args[1], i);
      arguments.tensors[i] = o == Py_None ? nullptr : &descriptors[i];
      if (o == Py_None) continue;
      if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
        return nullptr;
      }
      if (!fill(o, THPVariable_Unpack(o), &descriptors[i], &device)) return nullptr;
    }
    if (device < 0) {
      PyErr_SetString(PyExc_TypeError, "a call needs a tensor");
      return nullptr;
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    arguments.stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    if (!kind.run(entry->address, arguments, &status)) return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  return PyLong_FromLong(status);
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(name, address) -> entry"},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(entry, (t0, t1, ...), scalars...) -> status"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_describe", "calls of libwllm.so's entry points with torch tensors", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__describe() { return PyModule_Create(&module); }
