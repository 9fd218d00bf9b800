// What the CPython modules _ffn and _train have in common: the checks of a
// call's torch tensors and the call into libmoe.so.
#pragma once

#include <Python.h>

#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>

#include "moe.h"

namespace moe_py {

inline PyObject* g_error = nullptr;  // moe.MoEError(code, what)

enum Types : unsigned { kFp8 = 1, kBf16 = 2, kF32 = 4, kFloat = 8, kI32 = 16 };

inline const char* type_names(unsigned types) {
  switch (types) {
    case kFp8: return "torch.float8_e4m3fn or torch.uint8";
    case kBf16: return "torch.bfloat16 or torch.int16";
    case kF32: return "torch.float32";
    case kFloat: return "torch.bfloat16 or torch.float32";
    default: return "torch.int32";
  }
}

inline bool is_one_of(at::ScalarType t, unsigned types) {
  switch (t) {
    case at::ScalarType::Float8_e4m3fn: return types == kFp8;
    case at::ScalarType::Byte: return types == kFp8;
    case at::ScalarType::Short: return types == kBf16;  // bf16 bits, as the dispatch and combine calls take them
    case at::ScalarType::BFloat16: return types == kBf16 || types == kFloat;
    case at::ScalarType::Float: return types == kF32 || types == kFloat;
    case at::ScalarType::Int: return types == kI32;
    default: return false;
  }
}

inline PyObject* fail(int code, const char* format, ...) {
  char what[256];
  va_list args;
  va_start(args, format);
  std::vsnprintf(what, sizeof what, format, args);
  va_end(args);
  PyObject* error = PyObject_CallFunction(g_error, "is", code, what);
  if (error) {
    PyErr_SetObject(g_error, error);
    Py_DECREF(error);
  }
  return nullptr;
}

inline const at::Tensor* tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) {
    fail(MOE_EINVAL, "%s must be a tensor", name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// The call's device: that of the first tensor, which must be current; -1 if not.
inline int device_of(const char* name, const at::Tensor& t) {
  int current = -1;
  if (!t.is_cuda() || cudaGetDevice(&current) != cudaSuccess || t.get_device() != current) {
    fail(MOE_EINVAL, "%s must be on the current CUDA device", name);
    return -1;
  }
  return current;
}

// Whether `o` is a contiguous tensor of this type and shape on this device; its address.
inline bool arg(const char* name, PyObject* o, unsigned types, int ndim, const int64_t* shape, int device, void** address) {
  const at::Tensor* t = tensor(name, o);
  if (!t) return false;
  if (!is_one_of(t->scalar_type(), types)) {
    fail(MOE_EINVAL, "%s must be of type %s", name, type_names(types));
    return false;
  }
  bool same = t->dim() == ndim;
  for (int i = 0; same && i < ndim; ++i) same = t->size(i) == shape[i];
  if (!same) {
    char want[96] = "", *at = want;
    for (int i = 0; i < ndim; ++i)
      at += std::snprintf(at, want + sizeof want - at, "%s%lld", i ? ", " : "", static_cast<long long>(shape[i]));
    fail(MOE_EINVAL, "%s must have the shape [%s]", name, want);
    return false;
  }
  if (!t->is_contiguous()) {
    fail(MOE_EINVAL, "%s must be contiguous", name);
    return false;
  }
  if (!t->is_cuda() || t->get_device() != device) {
    fail(MOE_EINVAL, "%s must be on cuda:%d", name, device);
    return false;
  }
  *address = t->data_ptr();
  return true;
}

inline bool arg1(const char* name, PyObject* o, unsigned types, int64_t n, int device, void** address) {
  return arg(name, o, types, 1, &n, device, address);
}
inline bool arg2(const char* name, PyObject* o, unsigned types, int64_t n0, int64_t n1, int device, void** address) {
  const int64_t shape[2] = {n0, n1};
  return arg(name, o, types, 2, shape, device, address);
}

inline bool stream_of(PyObject* o, void** stream) {
  *stream = PyLong_AsVoidPtr(o);
  return *stream || !PyErr_Occurred();
}

// A call into libmoe.so, without the interpreter lock: a launch waits while the
// launch queue is full, and what empties it may need the lock (a host function
// in the stream, another thread).
template <class F>
PyObject* call(const char* what, F&& f) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = f();  // a C entry point: nothing is thrown
  PyEval_RestoreThread(state);
  if (rc != MOE_OK) return fail(rc, "%s", what);
  Py_RETURN_NONE;
}

inline bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
  return false;
}

// A size that the C interface takes as int32.
inline bool fits(const char* name, int64_t v) {
  if (v <= INT32_MAX) return true;
  fail(MOE_EINVAL, "%s is too large", name);
  return false;
}

inline PyObject* init(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

// C++ exceptions of the tensor library do not leave a call.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

}  // namespace moe_py
