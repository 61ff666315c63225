// Python binding of the dense feed-forward sublayer's C entry points (include/moe_ffn.h): checks of
// the tensors, outputs and workspaces from PyTorch's allocator, the current stream, and the call.  The
// checks take a few tenths of a microsecond here; through ctypes they took longer than a token's kernels.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <sstream>
#include <string>

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
  m.def("fp8_matmul", torch::wrap_pybind_function(&fp8_matmul));
}
