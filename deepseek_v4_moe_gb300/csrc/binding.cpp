// Python binding of the C entry points without a handle (include/moe_ffn.h): checks of
// the tensors, outputs and workspaces from PyTorch's allocator, the current stream, and the call.  The
// checks take a few tenths of a microsecond here; through ctypes they took longer than a token's kernels.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include "moe_ffn.h"

namespace py = pybind11;
using at::ScalarType;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

PyObject *g_error = nullptr;  // MoeFFNError

[[noreturn]] void refuse(const std::string &what) { throw py::value_error(what); }

void check(int64_t rc) {
  if (rc >= 0) return;
  if (!g_error) throw std::runtime_error(moe_ffn_last_error(nullptr));
  const py::object e = py::reinterpret_borrow<py::object>(g_error)(rc, moe_ffn_last_error(nullptr));
  PyErr_SetObject(g_error, e.ptr());
  throw py::error_already_set();
}

std::string text(at::IntArrayRef shape) {
  std::ostringstream s;
  s << shape;
  return s.str();
}

int type_code(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return MOE_FFN_F32;
    case ScalarType::BFloat16: return MOE_FFN_BF16;
    case ScalarType::Half: return MOE_FFN_F16;
    default: return -1;
  }
}
int fp8_code(ScalarType t) {
  switch (t) {
    case ScalarType::Float8_e4m3fn: return MOE_FFN_E4M3;
    case ScalarType::Float8_e5m2: return MOE_FFN_E5M2;
    default: return -1;
  }
}

ScalarType dtype_of(py::handle o) {
  if (!THPDtype_Check(o.ptr())) refuse("a torch.dtype is needed");
  return reinterpret_cast<THPDtype *>(o.ptr())->scalar_type;
}

// the place of a call: the tensor's device, current until the call returns, and its current stream
struct Where {
  at::Device device;
  c10::cuda::CUDAGuard guard;
  void *stream;
  Where(const char *name, const Tensor &t)
      : device(checked(name, t)), guard(device), stream(c10::cuda::getCurrentCUDAStream(device.index()).stream()) {}
  static at::Device checked(const char *name, const Tensor &t) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t.device();
  }
};

void on(const Where &w, const char *name, const Tensor &t, ScalarType type) {
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.device() != w.device) refuse(std::string(name) + " must be on " + w.device.str() + ", is on " + t.device().str());
}

// Checks a matrix; returns the distance between its rows.
int64_t matrix(const Where &w, const char *name, const Tensor &t, at::IntArrayRef shape, ScalarType type) {
  if (t.sizes() != shape) refuse(std::string(name) + " must be of shape " + text(shape) + ", got " + text(t.sizes()));
  on(w, name, t, type);
  if (shape[1] > 1 && t.stride(1) != 1) refuse(std::string(name) + " must have contiguous rows");
  return shape[0] > 1 ? t.stride(0) : shape[1];
}
// Checks a contiguous tensor; returns its address.
void *whole(const Where &w, const char *name, const Tensor &t, at::IntArrayRef shape, ScalarType type) {
  if (t.sizes() != shape || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous tensor of shape " + text(shape) + ", got " + text(t.sizes()));
  on(w, name, t, type);
  return t.data_ptr();
}
void two(const char *name, const Tensor &t) {
  if (t.dim() != 2) refuse(std::string(name) + " must be [rows, columns], got " + text(t.sizes()));
}
// sizes that the entry points' 32-bit fields hold
int32_t size32(const char *name, int64_t n) {
  if (n > INT32_MAX) refuse(std::string(name) + " is too large");
  return (int32_t)n;
}

Tensor fresh(const Where &w, at::IntArrayRef shape, ScalarType type) {
  return Tensor(at::detail::empty_cuda(shape, at::TensorOptions().dtype(type).device(w.device)));
}

// The call has written into a tensor that the caller gave: a gradient that autograd would take of what was in it
// is refused, as after PyTorch's own in-place operations.
void written(const Maybe &t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// ---- block_norm ----

moe_ffn_block_norm_args norm_args(const Where &w, const Tensor &state, const Maybe &f, const Maybe &norm_f, const Maybe &gate,
                                  double scale, const Maybe &norm_next, double eps, ScalarType block) {
  two("state", state);
  const auto shape = state.sizes();
  const int64_t rows = shape[0], hidden = shape[1];
  const ScalarType stream = state.scalar_type();
  moe_ffn_block_norm_args a = {};
  a.stream_type = type_code(stream);
  a.block_type = type_code(block);
  if (a.stream_type < 0 || a.block_type < 0 || (stream != ScalarType::Float && stream != block))
    refuse("state must be float32 or of the block's type (float32, bfloat16, float16)");
  a.rows = size32("rows", rows);
  a.hidden = size32("hidden", hidden);
  a.residual_scale = (float)scale;
  a.eps = (float)eps;
  a.ld_state = matrix(w, "state", state, shape, stream);
  a.state = state.data_ptr();
  if (f) {
    a.ld_f = matrix(w, "f", *f, shape, block);
    a.f = f->data_ptr();
  } else if (gate || norm_f) {
    refuse("gate and norm_f need f");
  }
  if (norm_f) a.norm_f = static_cast<float *>(whole(w, "norm_f", *norm_f, {hidden}, ScalarType::Float));
  if (norm_next) a.norm_next = static_cast<float *>(whole(w, "norm_next", *norm_next, {hidden}, ScalarType::Float));
  if (gate) {
    const auto g = gate->sizes();
    const ScalarType type = gate->scalar_type();
    if ((type != ScalarType::Float && type != block) || !gate->is_contiguous() || gate->device() != w.device)
      refuse("gate must be contiguous, on the state's device, float32 or of the block's type");
    if (g.size() == 1 && g[0] == hidden) {
      a.gate_kind = MOE_FFN_GATE_VECTOR;
      a.rows_per_gate = a.rows > 0 ? a.rows : 1;
    } else if (g.size() == 2 && g[1] == hidden && g[0] > 0 && rows > 0 && rows % g[0] == 0) {
      a.gate_kind = MOE_FFN_GATE_VECTOR;
      a.rows_per_gate = (int32_t)(rows / g[0]);
    } else if (g.size() == 2 && g[0] == rows && g[1] == 1) {
      a.gate_kind = MOE_FFN_GATE_TOKEN;
    } else {
      std::ostringstream s;
      s << "gate must be [" << hidden << "], [G, " << hidden << "] with G dividing " << rows << ", or [" << rows
        << ", 1]; got " << g;
      refuse(s.str());
    }
    a.gate_type = type_code(type);
    a.gate = gate->data_ptr();
  }
  return a;
}

py::tuple block_norm(const Tensor &state, const Maybe &f, const Maybe &norm_f, const Maybe &gate, double scale,
                     const Maybe &norm_next, double eps, py::object block_dtype, Maybe out, Maybe y) {
  const Where w("state", state);
  const ScalarType block = f ? f->scalar_type() : block_dtype.is_none() ? state.scalar_type() : dtype_of(block_dtype);
  if (!block_dtype.is_none() && dtype_of(block_dtype) != block) refuse("block_dtype must be f's type");
  moe_ffn_block_norm_args a = norm_args(w, state, f, norm_f, gate, scale, norm_next, eps, block);
  const auto shape = state.sizes();
  const Maybe given_out = out, given_y = y;
  if (f) {
    if (!out) out = fresh(w, shape, state.scalar_type());
    a.ld_out = matrix(w, "out", *out, shape, state.scalar_type());
    a.out = out->data_ptr();
  } else if (out) {
    refuse("out is written only with f");
  }
  if (norm_next) {
    if (!y) y = fresh(w, shape, block);
    a.ld_y = matrix(w, "y", *y, shape, block);
    a.y = y->data_ptr();
  } else if (y) {
    refuse("y is written only with norm_next");
  }
  check(moe_ffn_block_norm(&a, w.stream));
  written(given_out);
  written(given_y);
  return py::make_tuple(f ? *out : state, y ? py::cast(*y) : py::none());
}

// codes [rows, k] and scales [rows, ceil(k / 128)] of a call's result
moe_ffn_fp8_out fp8_out(const Where &w, int64_t rows, int64_t k, py::object dtype, bool pow2, Tensor &codes, Tensor &scales) {
  const ScalarType type = dtype_of(dtype);
  if (fp8_code(type) < 0) refuse("dtype must be float8_e4m3fn or float8_e5m2");
  codes = fresh(w, {rows, k}, type);
  scales = fresh(w, {rows, (k + 127) / 128}, ScalarType::Float);
  moe_ffn_fp8_out o = {};
  o.code_type = fp8_code(type);
  o.pow2 = pow2;
  o.codes = codes.data_ptr();
  o.ld_codes = k;
  o.scales = static_cast<float *>(scales.data_ptr());
  return o;
}

py::tuple block_norm_fp8(const Tensor &state, const Maybe &f, const Maybe &norm_f, const Maybe &gate, double scale,
                         const Tensor &norm_next, double eps, bool pow2, py::object dtype, Maybe out) {
  const Where w("state", state);
  const ScalarType block = f ? f->scalar_type() : state.scalar_type();
  moe_ffn_block_norm_args a = norm_args(w, state, f, norm_f, gate, scale, norm_next, eps, block);
  const auto shape = state.sizes();
  const Maybe given = out;
  if (f) {
    if (!out) out = fresh(w, shape, state.scalar_type());
    a.ld_out = matrix(w, "out", *out, shape, state.scalar_type());
    a.out = out->data_ptr();
  } else if (out) {
    refuse("out is written only with f");
  }
  Tensor codes, scales;
  const moe_ffn_fp8_out o = fp8_out(w, shape[0], shape[1], dtype, pow2, codes, scales);
  check(moe_ffn_block_norm_fp8(&a, &o, w.stream));
  written(given);
  return py::make_tuple(f ? *out : state, codes, scales);
}

py::tuple gated_quantise(const Tensor &gate, const Tensor &up, int activation, bool pow2, py::object dtype) {
  const Where w("gate", gate);
  const ScalarType t = gate.scalar_type();
  if (t != ScalarType::BFloat16 && t != ScalarType::Half) refuse("gate must be bfloat16 or float16");
  two("gate", gate);
  moe_ffn_gated_quantise_args a = {};
  a.rows = size32("rows", gate.size(0));
  a.columns = size32("columns", gate.size(1));
  a.type = type_code(t);
  a.activation = activation;
  a.ld_gate = matrix(w, "gate", gate, gate.sizes(), t);
  a.gate = gate.data_ptr();
  a.ld_up = matrix(w, "up", up, gate.sizes(), t);
  a.up = up.data_ptr();
  Tensor codes, scales;
  const moe_ffn_fp8_out o = fp8_out(w, gate.size(0), gate.size(1), dtype, pow2, codes, scales);
  check(moe_ffn_gated_quantise(&a, &o, w.stream));
  return py::make_tuple(codes, scales);
}

py::dict block_norm_backward(const Tensor &out, const Maybe &f, const Maybe &norm_f, const Maybe &gate, double scale,
                             const Maybe &norm_next, double eps, const Maybe &d_out, const Maybe &d_y) {
  const Where w("out", out);
  if (!f && !norm_next) refuse("neither f nor norm_next is given");
  if (norm_next.has_value() != d_y.has_value()) refuse("d_y goes with norm_next");
  const ScalarType block = f ? f->scalar_type() : d_y->scalar_type(), stream = out.scalar_type();
  const moe_ffn_block_norm_args a = norm_args(w, out, f, norm_f, gate, scale, norm_next, eps, block);
  const auto shape = out.sizes();
  moe_ffn_block_norm_grads g = {};
  py::dict d;
  if (d_out) {
    g.ld_d_out = matrix(w, "d_out", *d_out, shape, stream);
    g.d_out = d_out->data_ptr();
  }
  if (d_y) {
    g.ld_d_y = matrix(w, "d_y", *d_y, shape, block);
    g.d_y = d_y->data_ptr();
  }
  auto make = [&](const char *name, at::IntArrayRef s, ScalarType t) {
    const Tensor x = fresh(w, s, t);
    d[name] = x;
    return x.data_ptr();
  };
  g.d_state = make("d_state", shape, stream);
  g.ld_d_state = shape[1];
  if (f) {
    g.d_f = make("d_f", shape, block);
    g.ld_d_f = shape[1];
  }
  if (gate) g.d_gate = make("d_gate", gate->sizes(), gate->scalar_type());
  if (norm_f) g.d_norm_f = static_cast<float *>(make("d_norm_f", {shape[1]}, ScalarType::Float));
  if (norm_next) g.d_norm_next = static_cast<float *>(make("d_norm_next", {shape[1]}, ScalarType::Float));
  const int64_t need = moe_ffn_block_norm_workspace(&a, &g);
  check(need);
  Tensor ws;
  if (need) {
    ws = fresh(w, {need}, ScalarType::Byte);
    g.workspace = ws.data_ptr();
    g.workspace_bytes = (size_t)need;
  }
  check(moe_ffn_block_norm_backward(&a, &g, w.stream));
  return d;
}

// ---- gated block ----

moe_ffn_gated_args gated_args(const Where &w, const Tensor &x, const Tensor &w_gate, const Tensor &w_up,
                              const Tensor &w_down, int activation) {
  two("x", x);
  const ScalarType t = x.scalar_type();
  if (t != ScalarType::BFloat16 && t != ScalarType::Half) refuse("x must be bfloat16 or float16");
  two("w_gate", w_gate);
  const int64_t rows = x.size(0), hidden = x.size(1), inter = w_gate.size(0);
  moe_ffn_gated_args a = {};
  a.rows = size32("rows", rows);
  a.hidden = size32("hidden", hidden);
  a.inter = size32("inter", inter);
  a.type = type_code(t);
  a.activation = activation;
  a.ld_x = matrix(w, "x", x, x.sizes(), t);
  a.x = x.data_ptr();
  a.w_gate = whole(w, "w_gate", w_gate, {inter, hidden}, t);
  a.w_up = whole(w, "w_up", w_up, {inter, hidden}, t);
  a.w_down = whole(w, "w_down", w_down, {hidden, inter}, t);
  return a;
}

Tensor gated_workspace(const Where &w, moe_ffn_gated_args &a, int backward) {
  const int64_t need = moe_ffn_gated_workspace(&a, backward);
  check(need);
  const Tensor ws = fresh(w, {need}, ScalarType::Byte);
  a.workspace = ws.data_ptr();
  a.workspace_bytes = (size_t)need;
  return ws;
}

py::object gated_ffn(const Tensor &x, const Tensor &w_gate, const Tensor &w_up, const Tensor &w_down, int activation,
                     bool save, Maybe out) {
  const Where w("x", x);
  moe_ffn_gated_args a = gated_args(w, x, w_gate, w_up, w_down, activation);
  const ScalarType t = x.scalar_type();
  const Maybe given = out;
  if (!out) out = fresh(w, x.sizes(), t);
  a.ld_y = matrix(w, "out", *out, x.sizes(), t);
  a.y = out->data_ptr();
  Tensor g, u;
  if (save) {
    g = fresh(w, {a.rows, a.inter}, t);
    u = fresh(w, {a.rows, a.inter}, t);
    a.gate = g.data_ptr();
    a.up = u.data_ptr();
  }
  const Tensor ws = gated_workspace(w, a, 0);
  check(moe_ffn_gated_forward(&a, w.stream));
  written(given);
  if (save) return py::make_tuple(*out, py::make_tuple(g, u));
  return py::cast(*out);
}

py::dict gated_ffn_backward(const Tensor &x, const Tensor &w_gate, const Tensor &w_up, const Tensor &w_down,
                            const Tensor &g, const Tensor &u, const Tensor &d_y, int activation, bool need_x,
                            bool need_weights) {
  const Where w("x", x);
  moe_ffn_gated_args a = gated_args(w, x, w_gate, w_up, w_down, activation);
  const ScalarType t = x.scalar_type();
  a.gate = whole(w, "saved[0]", g, {a.rows, a.inter}, t);
  a.up = whole(w, "saved[1]", u, {a.rows, a.inter}, t);
  a.ld_d_y = matrix(w, "d_y", d_y, x.sizes(), t);
  a.d_y = d_y.data_ptr();
  py::dict d;
  auto make = [&](const char *name, at::IntArrayRef s) {
    const Tensor y = fresh(w, s, t);
    d[name] = y;
    return y.data_ptr();
  };
  if (need_x) {
    a.d_x = make("d_x", x.sizes());
    a.ld_d_x = a.hidden;
  }
  if (need_weights) {
    a.d_w_gate = make("d_w_gate", w_gate.sizes());
    a.d_w_up = make("d_w_up", w_up.sizes());
    a.d_w_down = make("d_w_down", w_down.sizes());
  }
  const Tensor ws = gated_workspace(w, a, 1);
  check(moe_ffn_gated_backward(&a, w.stream));
  return d;
}

// ---- FP8 ----

py::tuple fp8_quantise(const Tensor &x, int block_rows, bool pow2, py::object dtype) {
  const Where w("x", x);
  const ScalarType code = dtype_of(dtype);
  if (type_code(x.scalar_type()) < 0 || fp8_code(code) < 0)
    refuse("x must be float32, bfloat16 or float16, dtype float8_e4m3fn or float8_e5m2");
  if (block_rows != 1 && block_rows != 128) refuse("block_rows must be 1 or 128");
  two("x", x);
  const int64_t rows = x.size(0), k = x.size(1);
  const Tensor codes = fresh(w, {rows, k}, code);
  const Tensor scales = fresh(w, {(rows + block_rows - 1) / block_rows, (k + 127) / 128}, ScalarType::Float);
  moe_ffn_fp8_quantise_args a = {};
  a.rows = size32("rows", rows);
  a.k = size32("k", k);
  a.type = type_code(x.scalar_type());
  a.code_type = fp8_code(code);
  a.block_rows = block_rows;
  a.pow2 = pow2;
  a.ld_x = matrix(w, "x", x, x.sizes(), x.scalar_type());
  a.x = x.data_ptr();
  a.codes = codes.data_ptr();
  a.ld_codes = k;
  a.scales = static_cast<float *>(scales.data_ptr());
  check(moe_ffn_fp8_quantise(&a, w.stream));
  return py::make_tuple(codes, scales);
}

Tensor fp8_matmul(const Tensor &a, const Tensor &a_scale, const Tensor &b, const Tensor &b_scale, py::object out_dtype,
                  Maybe out) {
  const Where w("a", a);
  const ScalarType type = dtype_of(out_dtype);
  if (fp8_code(a.scalar_type()) < 0 || fp8_code(b.scalar_type()) < 0 || type_code(type) < 0)
    refuse("a and b must be float8_e4m3fn or float8_e5m2, out_dtype float32, bfloat16 or float16");
  two("a", a);
  two("b", b);
  const int64_t rows = a.size(0), k = a.size(1), n = b.size(0), kb = (k + 127) / 128;
  moe_ffn_fp8_matmul_args p = {};
  p.rows = size32("rows", rows);
  p.n = size32("n", n);
  p.k = size32("k", k);
  p.a_type = fp8_code(a.scalar_type());
  p.b_type = fp8_code(b.scalar_type());
  p.out_type = type_code(type);
  p.ld_a = matrix(w, "a", a, a.sizes(), a.scalar_type());
  p.a = a.data_ptr();
  p.ld_b = matrix(w, "b", b, {n, k}, b.scalar_type());
  p.b = b.data_ptr();
  p.a_scale = static_cast<float *>(whole(w, "a_scale", a_scale, {rows, kb}, ScalarType::Float));
  p.b_scale = static_cast<float *>(whole(w, "b_scale", b_scale, {(n + 127) / 128, kb}, ScalarType::Float));
  const Maybe given = out;
  if (!out) out = fresh(w, {rows, n}, type);
  p.ld_out = matrix(w, "out", *out, {rows, n}, type);
  p.out = out->data_ptr();
  check(moe_ffn_fp8_matmul(&p, w.stream));
  written(given);
  return *out;
}

// ---- 4-bit weights and the routed layer ----

// Weights as the package's Int4 (codes, scales, zeros or None, group), or a plain tensor of values.
struct Weights {
  Tensor w, scales;
  Maybe zeros;
  int64_t group = 0;  // 0: values
  int64_t dim() const { return w.dim(); }
  int64_t n() const { return w.size(w.dim() - 2); }
  int64_t k() const { return w.size(w.dim() - 1) * (group ? 2 : 1); }
};
Weights weights_of(const char *name, py::handle o) {
  Weights r;
  if (THPVariable_Check(o.ptr())) {
    r.w = THPVariable_Unpack(o.ptr());
  } else if (PyTuple_Check(o.ptr()) && PyTuple_GET_SIZE(o.ptr()) == 4) {
    PyObject *item[4];
    for (int i = 0; i < 4; ++i) item[i] = PyTuple_GET_ITEM(o.ptr(), i);
    if (!THPVariable_Check(item[0]) || !THPVariable_Check(item[1]) || (item[2] != Py_None && !THPVariable_Check(item[2])))
      throw py::type_error(std::string(name) + " must hold tensors: codes, scales and zeros (or None)");
    r.w = THPVariable_Unpack(item[0]);
    r.scales = THPVariable_Unpack(item[1]);
    if (item[2] != Py_None) r.zeros = THPVariable_Unpack(item[2]);
    r.group = py::cast<int64_t>(py::handle(item[3]));
    if (r.group != 32 && r.group != 64 && r.group != 128) refuse(std::string(name) + " must have groups of 32, 64 or 128");
  } else {
    throw py::type_error(std::string(name) + " must be a torch.Tensor or an Int4");
  }
  if (r.w.dim() < 2) refuse(std::string(name) + " must be [..., rows, columns], got " + text(r.w.sizes()));
  return r;
}
// Checks 4-bit weights of any leading sizes; type: of the scales.
void check_codes(const Where &w, const char *name, const Weights &m, ScalarType type) {
  const std::string s = name;
  if (!m.group) refuse(s + " must be an Int4");
  whole(w, (s + ".codes").c_str(), m.w, m.w.sizes(), ScalarType::Byte);
  auto groups = m.w.sizes().vec();
  groups.back() = (m.k() + m.group - 1) / m.group;
  whole(w, (s + ".scales").c_str(), m.scales, groups, type);
  if (m.zeros) whole(w, (s + ".zeros").c_str(), *m.zeros, groups, ScalarType::Byte);
}
uint8_t *zeros_of(const Weights &m) { return m.zeros ? static_cast<uint8_t *>(m.zeros->data_ptr()) : nullptr; }

moe_ffn_int4_weights_args int4_args(const Weights &m) {
  moe_ffn_int4_weights_args a = {};
  a.n = size32("the number of rows", m.w.numel() / (m.w.size(-1) ? m.w.size(-1) : 1));
  a.k = size32("the number of columns", m.k());
  a.group = (int32_t)m.group;
  a.scale_type = type_code(m.scales.scalar_type());
  a.codes = static_cast<uint8_t *>(m.w.data_ptr());
  a.scales = m.scales.data_ptr();
  a.zeros = zeros_of(m);
  return a;
}

py::tuple int4_quantise(const Tensor &w, int64_t group, bool zero_points, py::object scale_dtype) {
  const Where at("w", w);
  const ScalarType t = w.scalar_type();
  const ScalarType st = scale_dtype.is_none() ? (t == ScalarType::Float ? ScalarType::BFloat16 : t) : dtype_of(scale_dtype);
  if (type_code(t) < 0 || (st != ScalarType::BFloat16 && st != ScalarType::Half))
    refuse("w must be float32, bfloat16 or float16, scale_dtype bfloat16 or float16");
  if (group != 32 && group != 64 && group != 128) refuse("group must be 32, 64 or 128");
  if (w.dim() < 2) refuse("w must be [..., rows, columns], got " + text(w.sizes()));
  const int64_t k = w.size(-1);
  if (w.dim() > 2 && !w.is_contiguous()) refuse("w of more than two dimensions must be contiguous");
  const int64_t ld = w.dim() == 2 ? matrix(at, "w", w, w.sizes(), t) : k;
  if (k % 32) refuse("w must have a multiple of 32 columns");
  auto shape = w.sizes().vec();
  Weights m;
  m.group = group;
  shape.back() = k / 2;
  m.w = fresh(at, shape, ScalarType::Byte);
  shape.back() = (k + group - 1) / group;
  m.scales = fresh(at, shape, st);
  if (zero_points) m.zeros = fresh(at, shape, ScalarType::Byte);
  const moe_ffn_int4_weights_args a = int4_args(m);
  check(moe_ffn_int4_quantise(&a, w.data_ptr(), type_code(t), ld, at.stream));
  return py::make_tuple(m.w, m.scales, m.zeros ? py::cast(*m.zeros) : py::none(), group);
}

Tensor int4_widen(py::object o, Maybe out) {
  const Weights m = weights_of("w", o);
  const Where w("w.codes", m.w);
  if (!m.group) refuse("w must be an Int4");
  const ScalarType t = m.scales.scalar_type();
  if (t != ScalarType::BFloat16 && t != ScalarType::Half) refuse("w.scales must be bfloat16 or float16");
  check_codes(w, "w", m, t);
  auto shape = m.w.sizes().vec();
  shape.back() = m.k();
  const Maybe given = out;
  if (!out) out = fresh(w, shape, t);
  int64_t ld = m.k();
  if (shape.size() == 2) ld = matrix(w, "out", *out, shape, t);
  else whole(w, "out", *out, shape, t);
  const moe_ffn_int4_weights_args a = int4_args(m);
  check(moe_ffn_int4_widen(&a, out->data_ptr(), ld, w.stream));
  written(given);
  return *out;
}

Tensor int4_matmul(const Tensor &x, py::object o, Maybe out) {
  const Where w("x", x);
  const ScalarType t = x.scalar_type();
  if (t != ScalarType::BFloat16 && t != ScalarType::Half) refuse("x must be bfloat16 or float16");
  two("x", x);
  const Weights m = weights_of("w", o);
  two("w.codes", m.w);
  check_codes(w, "w", m, t);
  const int64_t rows = x.size(0), n = m.n(), k = m.k();
  moe_ffn_int4_matmul_args a = {};
  a.rows = size32("rows", rows);
  a.n = size32("n", n);
  a.k = size32("k", k);
  a.type = type_code(t);
  a.group = (int32_t)m.group;
  a.ld_x = matrix(w, "x", x, {rows, k}, t);
  a.x = x.data_ptr();
  a.codes = static_cast<uint8_t *>(m.w.data_ptr());
  a.scales = m.scales.data_ptr();
  a.zeros = zeros_of(m);
  const Maybe given = out;
  if (!out) out = fresh(w, {rows, n}, t);
  a.ld_out = matrix(w, "out", *out, {rows, n}, t);
  a.out = out->data_ptr();
  const int64_t need = moe_ffn_int4_matmul_workspace(&a);
  check(need);
  Tensor ws;
  if (need) {
    ws = fresh(w, {need}, ScalarType::Byte);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = (size_t)need;
  }
  check(moe_ffn_int4_matmul(&a, w.stream));
  written(given);
  return *out;
}

py::tuple routed_ffn(const Tensor &x, const Tensor &router, py::object w_gate, py::object w_up, py::object w_down, int64_t top_k,
                     const Maybe &bias, int score, bool normalise, double route_scale, py::object shared, int activation, Maybe out) {
  const Where w("x", x);
  const ScalarType t = x.scalar_type();
  if (t != ScalarType::BFloat16 && t != ScalarType::Half) refuse("x must be bfloat16 or float16");
  two("x", x);
  two("w_router", router);
  const int64_t rows = x.size(0), hidden = x.size(1), experts = router.size(0);
  const ScalarType tr = router.scalar_type();
  if (tr != t && tr != ScalarType::Float) refuse("w_router must be float32 or of x's type");
  Weights m[6];
  const char *names[] = {"w_gate", "w_up", "w_down", "shared[0]", "shared[1]", "shared[2]"};
  m[0] = weights_of(names[0], w_gate);
  m[1] = weights_of(names[1], w_up);
  m[2] = weights_of(names[2], w_down);
  int64_t n_shared = 0;
  if (!shared.is_none()) {
    if (!PyTuple_Check(shared.ptr()) || PyTuple_GET_SIZE(shared.ptr()) != 3) refuse("shared must be three weights: gate, up and down");
    for (int i = 0; i < 3; ++i) m[3 + i] = weights_of(names[3 + i], PyTuple_GET_ITEM(shared.ptr(), i));
    n_shared = m[3].dim() == 2 ? 1 : m[3].w.size(0);
    if (n_shared < 1) refuse("shared must hold at least one expert");
  }
  const int64_t inter = m[0].n(), group = m[0].group;
  moe_ffn_routed_args a = {};
  moe_ffn_matrices *to[] = {&a.gate, &a.up, &a.down, &a.shared_gate, &a.shared_up, &a.shared_down};
  for (int i = 0; i < (n_shared ? 6 : 3); ++i) {
    const int64_t count = i < 3 ? experts : n_shared, n = i % 3 == 2 ? hidden : inter, k = i % 3 == 2 ? inter : hidden;
    if (m[i].group != group) refuse(std::string(names[i]) + " must be of w_gate's kind (values, or 4 bits with its group)");
    std::vector<int64_t> shape = {count, n, group ? k / 2 : k};
    if (i >= 3 && m[3].dim() == 2) shape.erase(shape.begin());
    if (group) {
      if (k % 32) refuse("hidden and inter must be multiples of 32 with 4-bit weights");
      if (m[i].w.sizes() != at::IntArrayRef(shape))
        refuse(std::string(names[i]) + ".codes must be of shape " + text(shape) + ", got " + text(m[i].w.sizes()));
      check_codes(w, names[i], m[i], t);
      to[i]->scales = m[i].scales.data_ptr();
      to[i]->zeros = zeros_of(m[i]);
    } else {
      whole(w, names[i], m[i].w, shape, t);
    }
    to[i]->w = m[i].w.data_ptr();
  }
  a.rows = size32("rows", rows);
  a.hidden = size32("hidden", hidden);
  a.inter = size32("inter", inter);
  a.experts = size32("experts", experts);
  a.top_k = size32("top_k", top_k);
  a.shared = size32("shared", n_shared);
  a.type = type_code(t);
  a.router_type = type_code(tr);
  a.bits = group ? 4 : 16;
  a.group = (int32_t)group;
  a.score = score;
  a.normalise = normalise;
  a.activation = activation;
  a.route_scale = (float)route_scale;
  a.ld_x = matrix(w, "x", x, x.sizes(), t);
  a.x = x.data_ptr();
  a.router = whole(w, "w_router", router, {experts, hidden}, tr);
  if (bias) a.bias = static_cast<float *>(whole(w, "bias", *bias, {experts}, ScalarType::Float));
  const int64_t need = moe_ffn_routed_workspace(&a);
  check(need);
  const Maybe given = out;
  if (!out) out = fresh(w, {rows, hidden}, t);
  a.ld_y = matrix(w, "out", *out, {rows, hidden}, t);
  a.y = out->data_ptr();
  const Tensor indices = fresh(w, {rows, top_k}, ScalarType::Int), chosen = fresh(w, {rows, top_k}, ScalarType::Float);
  a.indices = static_cast<int32_t *>(indices.data_ptr());
  a.weights = static_cast<float *>(chosen.data_ptr());
  const Tensor ws = fresh(w, {need}, ScalarType::Byte);
  a.workspace = ws.data_ptr();
  a.workspace_bytes = (size_t)need;
  check(moe_ffn_routed_forward(&a, w.stream));
  written(given);
  return py::make_tuple(*out, indices, chosen);
}

}  // namespace

// wrap_pybind_function: errors of PyTorch's own (a failed allocation) keep their Python types
PYBIND11_MODULE(_native, m) {
  m.def("set_error", [](py::object cls) { g_error = cls.release().ptr(); });
  m.def("block_norm", torch::wrap_pybind_function(&block_norm));
  m.def("block_norm_fp8", torch::wrap_pybind_function(&block_norm_fp8));
  m.def("gated_quantise", torch::wrap_pybind_function(&gated_quantise));
  m.def("block_norm_backward", torch::wrap_pybind_function(&block_norm_backward));
  m.def("gated_ffn", torch::wrap_pybind_function(&gated_ffn));
  m.def("gated_ffn_backward", torch::wrap_pybind_function(&gated_ffn_backward));
  m.def("fp8_quantise", torch::wrap_pybind_function(&fp8_quantise));
  m.def("int4_quantise", torch::wrap_pybind_function(&int4_quantise));
  m.def("int4_widen", torch::wrap_pybind_function(&int4_widen));
  m.def("int4_matmul", torch::wrap_pybind_function(&int4_matmul));
  m.def("routed_ffn", torch::wrap_pybind_function(&routed_ffn));
  m.def("fp8_matmul", torch::wrap_pybind_function(&fp8_matmul));
}
