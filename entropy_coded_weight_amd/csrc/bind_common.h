// What the Python bindings share: argument checks, outputs from torch's allocator, errors.
#pragma once
#include <Python.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>

#include "../../include/ecw.h"

namespace {

PyObject* g_error = nullptr;  // EcwError

// thrown with a Python error set
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw Raised{};
}
[[noreturn]] void bad_type(const std::string& msg) { raise(PyExc_TypeError, msg); }
[[noreturn]] void bad_value(const std::string& msg) { raise(PyExc_ValueError, msg); }

void check(ecw_status s, const char* where) {
  if (s == ECW_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a cuda tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) bad_type(std::string(name) + " must be a cuda tensor");
  return t;
}

void same_device(const at::Tensor& t, const at::Tensor& with, const char* name, const char* what) {
  if (t.device() != with.device())
    bad_value(std::string(name) + " is on " + t.device().str() + ", the " + what + " on " + with.device().str());
}

int float_type(at::ScalarType t, const char* name, bool single = true) {
  if (t == at::kHalf) return ECW_DT_F16;
  if (t == at::kBFloat16) return ECW_DT_BF16;
  if (t == at::kFloat && single) return ECW_DT_F32;
  bad_type(std::string(name) + " must be float16" + (single ? ", bfloat16 or float32" : " or bfloat16"));
}

at::ScalarType dtype(PyObject* o, const char* name) {
  if (!THPDtype_Check(o)) bad_type(std::string(name) + " must be a torch dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int64_t whole(PyObject* o, const char* name, int64_t most) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < 0 || v > most) bad_value(std::string(name) + " must be in [0, " + std::to_string(most) + "]");
  return v;
}

// What a call writes advances its version, so that autograd notices if it holds the tensor.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A new tensor on like's device, from torch's allocator without a turn through its dispatcher.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

// the given output, or a new one
at::Tensor output(PyObject* o, const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type, const char* name) {
  if (o == Py_None) return fresh(shape, type, like);
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || !t.is_contiguous() || t.device() != like.device()) {
    std::string s;
    for (int64_t v : shape) s += (s.empty() ? "" : ", ") + std::to_string(v);
    bad_value(std::string(name) + " must be a contiguous (" + s + ") tensor on " + like.device().str());
  }
  written(t);
  return t;
}

ecw_stream stream_of(const at::Device& d) {
  return c10::hip::getCurrentHIPStream(d.index()).stream();
}

// [rows, cols] or [cols] of a tensor with a unit inner stride
struct Matrix {
  int64_t rows, cols, stride;
};
Matrix matrix(const at::Tensor& t, const char* name, const char* shape) {
  if (t.dim() != 1 && t.dim() != 2) bad_value(std::string(name) + " must be " + shape);
  const int64_t d = t.dim() - 1;
  if (t.size(d) > 1 && t.stride(d) != 1) bad_type(std::string(name) + " must have a unit inner stride");
  return {d ? t.size(0) : 1, t.size(d), d ? t.stride(0) : t.size(d)};
}

uint32_t size32(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) bad_value(std::string(name) + " too large");
  return (uint32_t)v;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) bad_type("wrong number of arguments");
}

template <class F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// The calls of libecw.so by name, from init's arguments: its path and EcwError.
struct Call {
  const char* name;
  void** to;
};
PyObject* load_calls(PyObject* args, std::initializer_list<Call> calls) {
  const char* path;
  PyObject* error;
  if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
  void* h = dlopen(path, RTLD_NOW);
  if (!h) return PyErr_Format(PyExc_ImportError, "%s", dlerror());
  for (const auto& f : calls)
    if (!(*f.to = dlsym(h, f.name))) return PyErr_Format(PyExc_ImportError, "%s has no %s", path, f.name);
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}

}  // namespace
