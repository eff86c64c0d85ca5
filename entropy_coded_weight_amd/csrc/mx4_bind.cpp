// Python binding of the 4-bit entry points: argument checks, outputs and workspaces from
// torch's allocator, the current stream of the operands' device.  A call from Python
// through ctypes took 8 to 10 us of host time, more than most of these kernels run.
#include <Python.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include <ATen/ATen.h>

#include "../../include/ecw.h"

namespace {

PyObject* g_error = nullptr;  // EcwError

struct Api {
  decltype(&mx4_quantize) quantize;
  decltype(&mx4_dequantize) dequantize;
  decltype(&mx4_gemm) gemm;
  decltype(&mx4_gemm_mx4) gemm_mx4;
  decltype(&kv4_append) append;
  decltype(&kv4_read) read;
  decltype(&kv4_attend_workspace_size) workspace;
  decltype(&kv4_attend) attend;
} api;

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

// the given output, or a new one
at::Tensor output(PyObject* o, const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type, const char* name) {
  if (o == Py_None) return at::empty(shape, like.options().dtype(type));
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

// ------------------------------------------------------------------ matrices
// quantize(x, codes or None, scales or None) -> codes, scales, cols
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 3);
    const at::Tensor& x = tensor(a[0], "x");
    const int xd = float_type(x.scalar_type(), "x");
    const Matrix m = matrix(x, "x", "[rows, cols] with at least one column");
    if (m.cols == 0) bad_value("x must be [rows, cols] with at least one column");
    const c10::DeviceGuard guard(x.device());
    const at::Tensor codes = output(a[1], x, {m.rows, (m.cols + 127) / 128 * 64}, at::kByte, "codes");
    const at::Tensor scales = output(a[2], x, {m.rows, (m.cols + 511) / 512 * 16}, at::kByte, "scales");
    check(api.quantize(stream_of(x.device()), x.data_ptr(), xd, m.stride, size32(m.rows, "rows"),
                       size32(m.cols, "cols"), codes.data_ptr(), scales.data_ptr()),
          "mx4_quantize");
    return Py_BuildValue("NNL", THPVariable_Wrap(codes), THPVariable_Wrap(scales), (long long)m.cols);
  });
}

// dequantize(codes, scales, cols, dtype, out or None) -> out
PyObject* py_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 5);
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
    const int64_t rows = codes.size(0), cols = whole(a[2], "cols", 1 << 30);
    const c10::DeviceGuard guard(codes.device());
    const at::ScalarType type = a[4] == Py_None ? dtype(a[3], "dtype") : tensor(a[4], "out").scalar_type();
    const int od = float_type(type, "out");
    const at::Tensor out = output(a[4], codes, {rows, cols}, type, "out");
    check(api.dequantize(stream_of(codes.device()), codes.data_ptr(), scales.data_ptr(), (uint32_t)rows,
                         (uint32_t)cols, out.data_ptr(), od),
          "mx4_dequantize");
    return THPVariable_Wrap(out);
  });
}

// gemm(codes, scales, cols, x, y or None, dtype) -> y
PyObject* py_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 6);
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales"), &x = tensor(a[3], "x");
    const int64_t rows = codes.size(0), cols = whole(a[2], "cols", 1 << 30);
    const Matrix m = matrix(x, "x", "[batch, cols]");
    if (m.cols != cols)
      bad_value("x has " + std::to_string(m.cols) + " columns, the tensor " + std::to_string(cols));
    same_device(x, codes, "x", "tensor");
    const int xd = float_type(x.scalar_type(), "x", false);
    const c10::DeviceGuard guard(codes.device());
    const at::ScalarType type = a[4] == Py_None ? dtype(a[5], "out_dtype") : tensor(a[4], "y").scalar_type();
    const int yd = float_type(type, "y");
    const at::Tensor y = output(a[4], codes, {m.rows, rows}, type, "y");
    check(api.gemm(stream_of(codes.device()), codes.data_ptr(), scales.data_ptr(), (uint32_t)rows, (uint32_t)cols,
                   x.data_ptr(), xd, m.stride, size32(m.rows, "batch"), y.data_ptr(), yd),
          "mx4_gemm");
    return THPVariable_Wrap(y);
  });
}

// gemm_mx4(codes, scales, cols, x codes, x scales, x cols, y or None, dtype) -> y
PyObject* py_gemm_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 8);
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
    const at::Tensor &xc = tensor(a[3], "x"), &xs = tensor(a[4], "x");
    const int64_t rows = codes.size(0), cols = whole(a[2], "cols", 1 << 30), have = whole(a[5], "cols", 1 << 30);
    if (have != cols) bad_value("x has " + std::to_string(have) + " columns, the tensor " + std::to_string(cols));
    same_device(xc, codes, "x", "tensor");
    const c10::DeviceGuard guard(codes.device());
    const at::ScalarType type = a[6] == Py_None ? dtype(a[7], "out_dtype") : tensor(a[6], "y").scalar_type();
    const int yd = float_type(type, "y");
    const at::Tensor y = output(a[6], codes, {xc.size(0), rows}, type, "y");
    check(api.gemm_mx4(stream_of(codes.device()), codes.data_ptr(), scales.data_ptr(), (uint32_t)rows, (uint32_t)cols,
                       xc.data_ptr(), xs.data_ptr(), (uint32_t)xc.size(0), y.data_ptr(), yd),
          "mx4_gemm_mx4");
    return THPVariable_Wrap(y);
  });
}

// ------------------------------------------------------------------ cache
// the first arguments of every cache call: data, pages, kv_heads, head_dim, page_tokens
constexpr Py_ssize_t kCacheArgs = 5;
struct CacheCall {
  const at::Tensor& data;
  ecw_kv4 c;
  explicit CacheCall(PyObject* const* a)
      : data(tensor(a[0], "cache")),
        c{data.data_ptr(), (uint32_t)PyLong_AsUnsignedLong(a[1]), (uint32_t)PyLong_AsUnsignedLong(a[2]),
          (uint32_t)PyLong_AsUnsignedLong(a[3]), (uint32_t)PyLong_AsUnsignedLong(a[4])} {}
};

const at::Tensor& ints(PyObject* o, const char* name, const at::Tensor& with, int64_t dim) {
  const std::string n(name);
  if (!THPVariable_Check(o)) bad_type(n + " must be an int32 tensor on " + with.device().str());
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != at::kInt || t.device() != with.device())
    bad_type(n + " must be an int32 tensor on " + with.device().str());
  if (t.dim() != dim) bad_value(n + " must have " + std::to_string(dim) + " dimensions, got " + shape_of(t));
  if (t.numel() && t.size(dim - 1) > 1 && t.stride(dim - 1) != 1) bad_type(n + " must have a unit inner stride");
  return t;
}

ecw_kv4_rows rows_of(const CacheCall& c, PyObject* table, PyObject* lens, PyObject* starts, int64_t rows) {
  const at::Tensor& t = ints(table, "page_table", c.data, 2);
  const at::Tensor& l = ints(lens, "lens", c.data, 1);
  const int64_t batch = t.size(0);
  if (l.size(0) != batch)
    bad_value("lens has shape " + shape_of(l) + ", expected (" + std::to_string(batch) + ")");
  const int32_t* first = nullptr;
  if (starts != Py_None) {
    const at::Tensor& s = ints(starts, "starts", c.data, 1);
    if (s.size(0) != batch + 1)
      bad_value("starts has shape " + shape_of(s) + ", expected (" + std::to_string(batch + 1) + ")");
    first = static_cast<const int32_t*>(s.data_ptr());
  } else if (rows && (batch == 0 || rows % batch)) {
    bad_value(std::to_string(rows) + " rows are not the same number for each of " + std::to_string(batch) +
              " sequences: pass starts");
  }
  return {static_cast<const int32_t*>(t.data_ptr()), t.stride(0), static_cast<const int32_t*>(l.data_ptr()), first,
          size32(batch, "batch"), size32(t.size(1), "page_table"), size32(rows, "rows")};
}

const at::Tensor& heads(PyObject* o, const char* name, const CacheCall& c, bool kv) {
  const at::Tensor& t = tensor(o, name);
  same_device(t, c.data, name, "cache");
  if (t.dim() != 3 || t.size(2) != c.c.head_dim || (kv && t.size(1) != c.c.kv_heads))
    bad_value(std::string(name) + " has shape " + shape_of(t) + ", expected (*, " +
              (kv ? std::to_string(c.c.kv_heads) : "*") + ", " + std::to_string(c.c.head_dim) + ")");
  if (t.stride(2) != 1) bad_type(std::string(name) + " must have a unit inner stride");
  return t;
}

// append(cache..., k, v, page_table, lens, starts)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, kCacheArgs + 5);
    const CacheCall c(a);
    a += kCacheArgs;
    const at::Tensor &k = heads(a[0], "k", c, true), &v = heads(a[1], "v", c, true);
    if (k.size(0) != v.size(0) || k.scalar_type() != v.scalar_type())
      bad_value("k and v must agree in rows and dtype");
    const int dt = float_type(k.scalar_type(), "k");
    const ecw_kv4_rows r = rows_of(c, a[2], a[3], a[4], k.size(0));
    const int64_t strides[4] = {k.stride(0), k.stride(1), v.stride(0), v.stride(1)};
    const c10::DeviceGuard guard(c.data.device());
    written(c.data);
    check(api.append(stream_of(c.data.device()), &c.c, &r, k.data_ptr(), v.data_ptr(), dt, strides), "kv4_append");
    Py_RETURN_NONE;
  });
}

// read(cache..., page_table, lens, starts, rows, dtype) -> k, v
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, kCacheArgs + 5);
    const CacheCall c(a);
    a += kCacheArgs;
    const int64_t rows = whole(a[3], "rows", 1 << 30);
    const ecw_kv4_rows r = rows_of(c, a[0], a[1], a[2], rows);
    const at::ScalarType type = dtype(a[4], "dtype");
    const int dt = float_type(type, "dtype");
    const c10::DeviceGuard guard(c.data.device());
    const int64_t shape[3] = {rows, (int64_t)c.c.kv_heads, (int64_t)c.c.head_dim};
    const at::Tensor k = at::empty(shape, c.data.options().dtype(type));
    const at::Tensor v = at::empty(shape, c.data.options().dtype(type));
    check(api.read(stream_of(c.data.device()), &c.c, &r, k.data_ptr(), v.data_ptr(), dt), "kv4_read");
    return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
  });
}

// attend(cache..., q, page_table, lens, starts, max_rows, max_len, window, sinks, scale, out) -> out
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, kCacheArgs + 10);
    const CacheCall c(a);
    a += kCacheArgs;
    const at::Tensor& q = heads(a[0], "q", c, false);
    const int dt = float_type(q.scalar_type(), "q", false);
    const int64_t rows = q.size(0), q_heads = q.size(1);
    if (q_heads == 0 || q_heads % c.c.kv_heads)
      bad_value(std::to_string(q_heads) + " query heads are no multiple of " + std::to_string(c.c.kv_heads) +
                " key/value heads");
    const ecw_kv4_rows r = rows_of(c, a[1], a[2], a[3], rows);
    constexpr int64_t kTop = 1 << 30;
    auto upto = [&](PyObject* o, const char* name) {
      return o == Py_None ? 0u : (uint32_t)std::min(whole(o, name, INT64_MAX), kTop);
    };
    ecw_kv4_attention at{size32(q_heads, "q_heads"), upto(a[4], "max_rows"), upto(a[5], "max_len"),
                         upto(a[6], "window"),       upto(a[7], "sinks"),    0.f};
    if (a[8] == Py_None) {
      at.scale = 1.f / std::sqrt((float)c.c.head_dim);
    } else {
      at.scale = (float)PyFloat_AsDouble(a[8]);
      if (PyErr_Occurred()) throw Raised{};
    }
    const c10::DeviceGuard guard(c.data.device());
    if (a[9] != Py_None && tensor(a[9], "out").scalar_type() != q.scalar_type()) bad_value("out must have q's dtype");
    const at::Tensor out = output(a[9], q, {rows, q_heads, (int64_t)c.c.head_dim}, q.scalar_type(), "out");
    size_t bytes = 0;
    check(api.workspace(&c.c, &r, &at, &bytes), "kv4_attend_workspace_size");
    at::Tensor ws;
    if (bytes) ws = at::empty({(int64_t)bytes}, c.data.options());
    check(api.attend(stream_of(c.data.device()), &c.c, &r, &at, q.data_ptr(), dt, q.stride(0), q.stride(1),
                     out.data_ptr(), bytes ? ws.data_ptr() : nullptr, bytes),
          "kv4_attend");
    return THPVariable_Wrap(out);
  });
}

// init(path of libecw.so, EcwError)
PyObject* py_init(PyObject*, PyObject* args) {
  const char* path;
  PyObject* error;
  if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
  void* h = dlopen(path, RTLD_NOW);
  if (!h) return PyErr_Format(PyExc_ImportError, "%s", dlerror());
  struct {
    const char* name;
    void** to;
  } const all[] = {{"mx4_quantize", (void**)&api.quantize},     {"mx4_dequantize", (void**)&api.dequantize},
                   {"mx4_gemm", (void**)&api.gemm},             {"mx4_gemm_mx4", (void**)&api.gemm_mx4},
                   {"kv4_append", (void**)&api.append},         {"kv4_read", (void**)&api.read},
                   {"kv4_attend", (void**)&api.attend},         {"kv4_attend_workspace_size", (void**)&api.workspace}};
  for (const auto& f : all)
    if (!(*f.to = dlsym(h, f.name))) return PyErr_Format(PyExc_ImportError, "%s has no %s", path, f.name);
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(quantize), FAST(dequantize), FAST(gemm),   FAST(gemm_mx4),
                         FAST(append),   FAST(read),       FAST(attend), {"init", py_init, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mx4", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx4() { return PyModule_Create(&module); }
