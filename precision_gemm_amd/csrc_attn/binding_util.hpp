// What the CPython bindings share: argument checks on torch tensors, output allocation, and the
// translation of C++ exceptions into Python's.  Included by each binding's one source file.
#pragma once
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <initializer_list>
#include <limits>
#include <stdexcept>
#include <string>

#include "../../include/lora_lowp.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error { using std::runtime_error::runtime_error; };

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& req(PyObject* o, const char* name) {
  const Tensor* t = opt(o, name);
  if (!t) throw Refused(std::string(name) + " must be a tensor");
  return *t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) { PyErr_Clear(); throw Refused("sizes must be integers"); }
  return v;
}
int32_t int32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused("sizes must fit 32 bits");
  return (int32_t)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) { PyErr_Clear(); throw Refused("scale and eps must be numbers"); }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) { PyErr_Clear(); throw Refused(std::string(name) + " must be a truth value"); }
  return v == 1;
}

std::string list(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

void on_device(const Tensor& t, const char* name, const at::Device& dev) {
  if (dev.type() != at::kCUDA) throw Refused(std::string(name) + " must be a device tensor");
  if (t.device() != dev) throw Refused(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}

// Address of a dense device tensor of this type and shape.
void* need(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& dev) {
  if (t.scalar_type() != type)
    throw Refused(std::string(name) + " must have dtype " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (t.sizes() != shape) throw Refused(std::string(name) + " must have shape " + list(shape) + ", got " + list(t.sizes()));
  on_device(t, name, dev);
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return t.data_ptr();
}
void* need_or_null(const Tensor* t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& dev) {
  return t ? need(*t, name, type, shape, dev) : nullptr;
}

struct Rows { uint16_t* p; int64_t ld; };
// bf16 rows [T, width] (or [T, heads, D]) of any stride, their values dense within a row.
Rows rows(const Tensor& t, const char* name, int64_t width, int64_t T, const at::Device& dev) {
  if (t.scalar_type() != at::kBFloat16)
    throw Refused(std::string(name) + " must have dtype torch.bfloat16, got " + type_name(t.scalar_type()));
  on_device(t, name, dev);
  const int64_t d = t.dim();
  if ((d != 2 && d != 3) || t.size(0) != T || (d == 2 ? t.size(1) : t.size(1) * t.size(2)) != width)
    throw Refused(std::string(name) + " must be " + std::to_string(T) + " rows of " + std::to_string(width) + " values, got " + list(t.sizes()));
  if (T > 0 && ((t.size(d - 1) > 1 && t.stride(d - 1) != 1) || (d == 3 && t.size(1) > 1 && t.stride(1) != t.size(2))))
    throw Refused(std::string(name) + " must be dense within each row");
  return {static_cast<uint16_t*>(t.data_ptr()), T > 1 ? t.stride(0) : width};
}

// A new tensor straight from the device's allocator (at::empty finds it through the dispatcher).
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

int32_t tokens(const Tensor& t, const char* name) {
  if (t.dim() < 1 || t.size(0) > INT32_MAX) throw Refused(std::string(name) + " has no tokens' dimension");
  return (int32_t)t.size(0);
}
int32_t* status_word(PyObject* o, const at::Device& dev) {
  return static_cast<int32_t*>(need_or_null(opt(o, "status"), "status", at::kInt, {1}, dev));
}
void* stream(PyObject* o) { return PyLong_AsVoidPtr(o); }

PyObject* status(lora_status s) { return PyLong_FromLong(s); }

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  try {
    if (got != want) throw std::runtime_error("wrong number of arguments");
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    // torch's own type (a RuntimeError), which callers that free memory and try again catch
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

}  // namespace
