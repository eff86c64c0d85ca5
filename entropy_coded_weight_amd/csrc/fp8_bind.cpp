// Python binding of the 8-bit matrices, the root-mean-square norm and the rotary positions.
#include "bind_common.h"
#include "overlap.h"

namespace {

struct Api {
  decltype(&fp8_quantize) quantize;
  decltype(&fp8_dequantize) dequantize;
  decltype(&fp8_gemm) gemm;
  decltype(&fp8_gemm_workspace_size) workspace;
  decltype(&rms_norm) norm;
  decltype(&rotary_apply) rotary;
} api;

constexpr int64_t kMostCols = 1 << 30;

ecw::Box box(const at::Tensor& t) {
  return ecw::box_of(t.data_ptr(), t.element_size(), t.sizes().data(), t.strides().data(), t.dim());
}
// What a call writes next to what it reads must be none of its bytes, or (`same`) the same elements.
void apart(const at::Tensor& out, const at::Tensor& in, const char* out_name, const char* in_name, bool same = false) {
  if (same && out.data_ptr() == in.data_ptr() && out.scalar_type() == in.scalar_type() && out.sizes() == in.sizes() &&
      out.strides() == in.strides())
    return;
  if (ecw::boxes_meet(box(out), box(in))) bad_value(std::string(out_name) + " overlaps " + in_name);
}

struct Eight {
  at::Tensor codes, scales;
};
// [rows, width] bytes of a tensor of bytes from `offset` on, with its storage
at::Tensor bytes_of(const at::Tensor& all, int64_t offset, int64_t rows, int64_t width) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(offset);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({rows, width});
  return t;
}
// the given codes and scales of a [rows, cols] matrix, or new ones, in one piece of memory
Eight eight_bits(PyObject* codes, PyObject* scales, const at::Tensor& like, int64_t rows, int64_t cols) {
  const int64_t wide = (cols + 127) / 128 * 128, scale_wide = (cols + 2047) / 2048 * 16;
  if (codes == Py_None && scales == Py_None) {
    const at::Tensor all = fresh({rows * (wide + scale_wide)}, at::kByte, like);
    return {bytes_of(all, 0, rows, wide), bytes_of(all, rows * wide, rows, scale_wide)};
  }
  const Eight out{output(codes, like, {rows, wide}, at::kByte, "codes"), output(scales, like, {rows, scale_wide}, at::kByte, "scales")};
  apart(out.codes, out.scales, "codes", "scales");
  return out;
}

// quantize(x, gate or None, codes or None, scales or None) -> codes, scales, cols
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 4);
    const at::Tensor& x = tensor(a[0], "x");
    const int xd = float_type(x.scalar_type(), "x");
    const Matrix m = matrix(x, "x", "[rows, cols] with at least one column");
    if (m.cols == 0) bad_value("x must be [rows, cols] with at least one column");
    const at::Tensor* gate = nullptr;
    int64_t gate_stride = 0;
    if (a[1] != Py_None) {
      gate = &tensor(a[1], "gate");
      same_device(*gate, x, "gate", "tensor");
      if (gate->sizes() != x.sizes() || gate->scalar_type() != x.scalar_type()) bad_value("gate must have x's shape and dtype");
      gate_stride = matrix(*gate, "gate", "[rows, cols]").stride;
    }
    const c10::DeviceGuard guard(x.device());
    const Eight out = eight_bits(a[2], a[3], x, m.rows, m.cols);
    if (a[2] != Py_None) {
      apart(out.codes, x, "codes", "x"), apart(out.scales, x, "scales", "x");
      if (gate) apart(out.codes, *gate, "codes", "gate"), apart(out.scales, *gate, "scales", "gate");
    }
    check(api.quantize(stream_of(x.device()), x.data_ptr(), xd, m.stride, gate ? gate->data_ptr() : nullptr, gate_stride,
                       size32(m.rows, "rows"), size32(m.cols, "cols"), out.codes.data_ptr(), out.scales.data_ptr()),
          "fp8_quantize");
    return Py_BuildValue("NNL", THPVariable_Wrap(out.codes), THPVariable_Wrap(out.scales), (long long)m.cols);
  });
}

// dequantize(codes, scales, cols, dtype, out or None) -> out
PyObject* py_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 5);
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
    const int64_t rows = codes.size(0), cols = whole(a[2], "cols", kMostCols);
    const c10::DeviceGuard guard(codes.device());
    const at::ScalarType type = a[4] == Py_None ? dtype(a[3], "dtype") : tensor(a[4], "out").scalar_type();
    const int od = float_type(type, "out");
    const at::Tensor out = output(a[4], codes, {rows, cols}, type, "out");
    if (a[4] != Py_None) apart(out, codes, "out", "codes"), apart(out, scales, "out", "scales");
    check(api.dequantize(stream_of(codes.device()), codes.data_ptr(), scales.data_ptr(), (uint32_t)rows,
                         (uint32_t)cols, out.data_ptr(), od),
          "fp8_dequantize");
    return THPVariable_Wrap(out);
  });
}

// gemm(codes, scales, cols, x codes, x scales, x cols, y or None, dtype, short sums) -> y
PyObject* py_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 9);
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
    const at::Tensor &xc = tensor(a[3], "x"), &xs = tensor(a[4], "x");
    const int64_t rows = codes.size(0), cols = whole(a[2], "cols", kMostCols), have = whole(a[5], "cols", kMostCols);
    if (have != cols) bad_value("x has " + std::to_string(have) + " columns, the tensor " + std::to_string(cols));
    same_device(xc, codes, "x", "tensor");
    const c10::DeviceGuard guard(codes.device());
    const at::ScalarType type = a[6] == Py_None ? dtype(a[7], "out_dtype") : tensor(a[6], "y").scalar_type();
    int yd = float_type(type, "y");
    const int brief = PyObject_IsTrue(a[8]);
    if (brief < 0) throw Raised{};
    if (brief && yd == ECW_DT_F32) bad_value("short_sums are for float16 and bfloat16 results");
    if (brief) yd |= ECW_FP8_SHORT_SUMS;
    const at::Tensor y = output(a[6], codes, {xc.size(0), rows}, type, "y");
    if (a[6] != Py_None)
      for (const at::Tensor* in : {&codes, &scales, &xc, &xs}) apart(y, *in, "y", in == &xc || in == &xs ? "x" : "the tensor");
    const uint32_t batch = size32(xc.size(0), "batch");
    size_t bytes = 0;
    check(api.workspace((uint32_t)rows, (uint32_t)cols, batch, yd, &bytes), "fp8_gemm_workspace_size");
    at::Tensor ws;
    if (bytes) ws = fresh({(int64_t)bytes}, at::kByte, codes);
    check(api.gemm(stream_of(codes.device()), codes.data_ptr(), scales.data_ptr(), (uint32_t)rows, (uint32_t)cols,
                   xc.data_ptr(), xs.data_ptr(), batch, y.data_ptr(), yd, bytes ? ws.data_ptr() : nullptr, bytes),
          "fp8_gemm");
    return THPVariable_Wrap(y);
  });
}

// rms_norm(x, weight or None, residual or None, eps, dtype or None for 8 bits, y or codes or None, scales or None,
//          residual_out or None) -> y, or codes, scales, cols; and the new residual or None
PyObject* py_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 8);
    const at::Tensor& x = tensor(a[0], "x");
    ecw_rms_norm p{};
    p.x_dtype = float_type(x.scalar_type(), "x");
    const Matrix m = matrix(x, "x", "[rows, cols] or [cols]");
    if (m.cols == 0) bad_value("x must have at least one column");
    p.x = x.data_ptr(), p.x_stride = m.stride, p.rows = size32(m.rows, "rows"), p.cols = size32(m.cols, "cols");
    const at::Tensor* weight = nullptr;
    if (a[1] != Py_None) {
      weight = &tensor(a[1], "weight");
      same_device(*weight, x, "weight", "input");
      p.weight_dtype = float_type(weight->scalar_type(), "weight");
      if (weight->dim() != 1 || weight->size(0) != m.cols)
        bad_value("weight has shape " + shape_of(*weight) + ", expected (" + std::to_string(m.cols) + ")");
      if (m.cols > 1 && weight->stride(0) != 1) bad_type("weight must have a unit stride");
      p.weight = weight->data_ptr();
    }
    p.eps = (float)PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Raised{};
    const c10::DeviceGuard guard(x.device());
    const at::Tensor* residual = nullptr;
    at::Tensor next;
    if (a[2] != Py_None) {
      residual = &tensor(a[2], "residual");
      same_device(*residual, x, "residual", "input");
      p.residual_dtype = float_type(residual->scalar_type(), "residual");
      if (residual->scalar_type() != x.scalar_type() && residual->scalar_type() != at::kFloat)
        bad_type("residual must have x's dtype or be float32");
      if (residual->sizes() != x.sizes())
        bad_value("residual has shape " + shape_of(*residual) + ", x " + shape_of(x));
      p.residual = residual->data_ptr(), p.residual_stride = matrix(*residual, "residual", "[rows, cols]").stride;
      if (a[7] == Py_None) {
        next = fresh(x.sizes(), residual->scalar_type(), x);
      } else {
        next = tensor(a[7], "residual_out");
        same_device(next, x, "residual_out", "input");
        if (next.sizes() != x.sizes() || next.scalar_type() != residual->scalar_type())
          bad_value("residual_out must have residual's shape and dtype");
        const int64_t s = matrix(next, "residual_out", "[rows, cols]").stride;
        if (m.rows > 1 && s < m.cols) bad_value("residual_out's rows overlap");
        apart(next, *residual, "residual_out", "residual", true);
        apart(next, x, "residual_out", "x", true);
        if (weight) apart(next, *weight, "residual_out", "weight");
        written(next);
      }
      p.residual_out = next.data_ptr();
      p.residual_out_stride = m.rows > 1 ? matrix(next, "residual_out", "[rows, cols]").stride : m.cols;
    } else if (a[7] != Py_None) {
      bad_value("residual_out needs a residual");
    }
    auto clear_of_inputs = [&](const at::Tensor& out, const char* name, bool same) {
      apart(out, x, name, "x", same);
      if (residual) apart(out, *residual, name, "residual", same && !next.is_same(*residual));
      if (weight) apart(out, *weight, name, "weight");
      if (next.defined()) apart(out, next, name, "residual_out");
    };
    if (a[4] == Py_None) {
      p.y_dtype = ECW_DT_FP8_E4M3;
      const Eight out = eight_bits(a[5], a[6], x, m.rows, m.cols);
      if (a[5] != Py_None) clear_of_inputs(out.codes, "codes", false), clear_of_inputs(out.scales, "scales", false);
      p.y = out.codes.data_ptr(), p.y_scales = out.scales.data_ptr();
      check(api.norm(stream_of(x.device()), &p), "rms_norm");
      PyObject* h = next.defined() ? THPVariable_Wrap(next) : Py_NewRef(Py_None);
      return Py_BuildValue("NNLN", THPVariable_Wrap(out.codes), THPVariable_Wrap(out.scales), (long long)m.cols, h);
    }
    const at::ScalarType type = a[5] == Py_None ? dtype(a[4], "out_dtype") : tensor(a[5], "out").scalar_type();
    p.y_dtype = float_type(type, "out");
    const at::Tensor y = output(a[5], x, x.sizes(), type, "out");
    if (a[5] != Py_None) clear_of_inputs(y, "out", true);
    p.y = y.data_ptr();
    check(api.norm(stream_of(x.device()), &p), "rms_norm");
    if (!next.defined()) return THPVariable_Wrap(y);
    return Py_BuildValue("NN", THPVariable_Wrap(y), THPVariable_Wrap(next));
  });
}

const at::Tensor& heads(PyObject* o, const char* name, int64_t dim, const at::Tensor* with) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3 || t.size(2) != dim || (with && t.size(0) != with->size(0)))
    bad_value(std::string(name) + " has shape " + shape_of(t) + ", expected (" +
              (with ? std::to_string(with->size(0)) : "*") + ", *, " + std::to_string(dim) + ")");
  if (dim > 1 && t.stride(2) != 1) bad_type(std::string(name) + " must have a unit inner stride");
  if (with) {
    same_device(t, *with, name, "first");
    if (t.scalar_type() != with->scalar_type()) bad_value(std::string(name) + " must have q's dtype");
  }
  return t;
}

// rotary(q, k or None, positions, freqs, axis_of, axes, head_dim, neighbours, scale, q_out or None, k_out or None)
//   -> q_out or (q_out, k_out)
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 11);
    const int64_t dim = whole(a[6], "head_dim", 4096), axes = whole(a[5], "axes", 255);
    const at::Tensor& q = heads(a[0], "q", dim, nullptr);
    const at::Tensor &freqs = tensor(a[3], "freqs"), &axis_of = tensor(a[4], "axis_of");
    same_device(q, freqs, "q", "rotary");
    ecw_rotary p{};
    p.dtype = float_type(q.scalar_type(), "q");
    p.rows = size32(q.size(0), "rows"), p.q_heads = size32(q.size(1), "heads"), p.head_dim = (uint32_t)dim;
    p.q = q.data_ptr(), p.q_row = q.stride(0), p.q_head = q.stride(1);
    p.freqs = freqs.data_ptr(), p.axis_of = axis_of.data_ptr(), p.rotary_dim = 2 * (uint32_t)freqs.size(0);
    p.axes = (uint32_t)axes;
    p.neighbours = PyObject_IsTrue(a[7]);
    p.scale = (float)PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) throw Raised{};
    const at::Tensor& at = tensor(a[2], "positions");
    same_device(at, q, "positions", "first");
    if (at.scalar_type() != at::kInt && at.scalar_type() != at::kLong) bad_type("positions must be int32 or int64");
    const int64_t d = at.dim();
    if (!(d == 1 && axes == 1) && !(d == 2 && at.size(0) == axes))
      bad_value("positions has shape " + shape_of(at) + ", expected (" + std::to_string(axes) + ", rows)" +
                (axes == 1 ? " or (rows)" : ""));
    if (at.size(d - 1) != q.size(0))
      bad_value("positions has " + std::to_string(at.size(d - 1)) + " rows, q " + std::to_string(q.size(0)));
    if (at.size(d - 1) > 1 && at.stride(d - 1) != 1) bad_type("positions must have a unit inner stride");
    p.positions = at.data_ptr(), p.axis_stride = d == 2 ? at.stride(0) : 0;
    p.wide_positions = at.scalar_type() == at::kLong;
    const at::Tensor* k = nullptr;
    if (a[1] != Py_None) {
      k = &heads(a[1], "k", dim, &q);
      p.k = k->data_ptr(), p.k_row = k->stride(0), p.k_head = k->stride(1), p.k_heads = size32(k->size(1), "heads");
    } else if (a[10] != Py_None) {
      bad_value("an output for k without a k");
    }
    const c10::DeviceGuard guard(q.device());
    auto out_of = [&](PyObject* o, const at::Tensor& in, const char* name, const char* in_name) {
      if (o == Py_None) return fresh(in.sizes(), in.scalar_type(), in);
      const at::Tensor& t = tensor(o, name);
      same_device(t, q, name, "first");
      if (t.sizes() != in.sizes() || t.scalar_type() != in.scalar_type())
        bad_value(std::string(name) + " must have " + in_name + "'s shape and dtype");
      if (t.stride(2) != 1 && dim > 1) bad_type(std::string(name) + " must have a unit inner stride");
      if (box(t).folded) bad_value(std::string(name) + " overlaps itself");
      apart(t, in, name, in_name, true);
      apart(t, at, name, "positions");
      written(t);
      return t;
    };
    const at::Tensor q_out = out_of(a[9], q, "out[0]", "q");
    p.q_out = q_out.data_ptr(), p.q_out_row = q_out.stride(0), p.q_out_head = q_out.stride(1);
    at::Tensor k_out;
    if (k) {
      k_out = out_of(a[10], *k, "out[1]", "k");
      p.k_out = k_out.data_ptr(), p.k_out_row = k_out.stride(0), p.k_out_head = k_out.stride(1);
      if (a[9] != Py_None) apart(q_out, *k, "out[0]", "k");
      if (a[10] != Py_None) apart(k_out, q, "out[1]", "q"), apart(k_out, q_out, "out[1]", "out[0]");
    }
    check(api.rotary(stream_of(q.device()), &p), "rotary_apply");
    if (!k) return THPVariable_Wrap(q_out);
    return Py_BuildValue("NN", THPVariable_Wrap(q_out), THPVariable_Wrap(k_out));
  });
}

// init(path of libecw.so, EcwError)
PyObject* py_init(PyObject*, PyObject* args) {
  return load_calls(args, {{"fp8_quantize", (void**)&api.quantize}, {"fp8_dequantize", (void**)&api.dequantize},
                           {"fp8_gemm", (void**)&api.gemm},         {"fp8_gemm_workspace_size", (void**)&api.workspace},
                           {"rms_norm", (void**)&api.norm},         {"rotary_apply", (void**)&api.rotary}});
}

PyMethodDef methods[] = {FAST(quantize), FAST(dequantize), FAST(gemm), FAST(rms_norm), FAST(rotary),
                         {"init", py_init, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8() { return PyModule_Create(&module); }
