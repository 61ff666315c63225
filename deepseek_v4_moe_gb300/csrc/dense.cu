// C entry points of the dense feed-forward sublayer on a plain residual stream: argument checks and
// launches (include/moe_ffn.h documents each).  No handle: the only state is what is known of each
// device.
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>

#include "dense.h"
#include "kernels.h"
#include "moe_ffn.h"

namespace {

constexpr int kMaxDevices = 64;

int fail(int code, const char *fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  moe::set_global_error(buf);
  return code;
}

// SMs of the current device; a negative code where it is no sm_103 device
int current_sms() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return fail(MOE_FFN_ERR_CUDA, "no usable current device");
  }
  int sms = known[dev].load(std::memory_order_relaxed);
  if (sms) return sms;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(MOE_FFN_ERR_CUDA, "cannot query device %d", dev);
  }
  if (major != 10 || minor != 3) return fail(MOE_FFN_ERR_UNSUPPORTED, "needs an sm_103 device, found sm_%d%d", major, minor);
  known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// A tensor argument's memory: `rows` rows of `cols` elements, `ld` elements apart.
struct Span {
  const void *p;
  uintptr_t end;
  int64_t ld;
  const char *name;
};
Span span(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{p, p && rows > 0 ? a + (uintptr_t)((rows - 1) * ld + cols) * bytes : a, ld, name};
}
bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < b.end && y < a.end;
}
// An output may overlap no input and no other output, but for the one input it may be itself.
int check_overlaps(const char *who, const Span *outs, int n_outs, const Span *ins, int n_ins, int same_out, int same_in) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i], ins[j]) &&
          !(i == same_out && j == same_in && outs[i].p == ins[j].p && outs[i].ld == ins[j].ld))
        return fail(MOE_FFN_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, ins[j].name);
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(MOE_FFN_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, outs[j].name);
  }
  return MOE_FFN_OK;
}

int type_bytes(int t) { return t == MOE_FFN_F32 ? 4 : 2; }
bool is_type(int t) { return t == MOE_FFN_F32 || t == MOE_FFN_BF16 || t == MOE_FFN_F16; }
bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

int launched(const char *who, cudaError_t e) {
  return e == cudaSuccess ? MOE_FFN_OK : fail(MOE_FFN_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

// an error left by earlier work is reported with nothing enqueued
int pending(const char *who) {
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? MOE_FFN_OK
                          : fail(MOE_FFN_ERR_CUDA, "%s: a CUDA error is pending from earlier work: %s", who, cudaGetErrorString(e));
}

// ---- block_norm ----

int check_norm(const char *who, const moe_ffn_block_norm_args *a) {
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows is negative", who);
  if (a->hidden < 1 || a->hidden > moe::kNormHiddenMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: hidden must be in 1..%d", who, moe::kNormHiddenMax);
  if (!is_type(a->block_type) || (a->stream_type != MOE_FFN_F32 && a->stream_type != a->block_type))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: stream_type must be f32 or block_type", who);
  if (!(a->eps >= 0.f)) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: eps must be >= 0", who);
  if (!a->state) return fail(MOE_FFN_ERR_NULL_PTR, "%s: state is NULL", who);
  if (!a->f && (a->gate_kind != MOE_FFN_GATE_NONE || a->norm_f))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a gate or norm_f without f", who);
  if (!a->f && !a->norm_next) return fail(MOE_FFN_ERR_NULL_PTR, "%s: neither f nor norm_next is given", who);
  if (a->gate_kind != MOE_FFN_GATE_NONE) {
    if (a->gate_kind != MOE_FFN_GATE_VECTOR && a->gate_kind != MOE_FFN_GATE_TOKEN)
      return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown gate_kind", who);
    if (a->gate_type != MOE_FFN_F32 && a->gate_type != a->block_type)
      return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: gate_type must be f32 or block_type", who);
    if (!a->gate) return fail(MOE_FFN_ERR_NULL_PTR, "%s: gate is NULL", who);
    if (a->gate_kind == MOE_FFN_GATE_VECTOR && a->rows_per_gate < 1)
      return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: rows_per_gate must be at least 1", who);
    if (!aligned(a->gate, type_bytes(a->gate_type))) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: gate is misaligned", who);
  }
  const int sb = type_bytes(a->stream_type), bb = type_bytes(a->block_type);
  if (a->ld_state < a->hidden || (a->f && a->ld_f < a->hidden))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a row stride is below hidden", who);
  if (!aligned(a->state, sb) || !aligned(a->f, bb) || !aligned(a->norm_f, 4) || !aligned(a->norm_next, 4))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: a pointer is not aligned to its type", who);
  return MOE_FFN_OK;
}

moe::NormParams norm_params(const moe_ffn_block_norm_args *a) {
  moe::NormParams p = {};
  p.rows = a->rows;
  p.hidden = a->hidden;
  p.stream_type = a->stream_type;
  p.block_type = a->block_type;
  p.gate_type = a->gate_type;
  p.gate_kind = a->f ? a->gate_kind : MOE_FFN_GATE_NONE;
  // rows that share nothing but the norms, or a group longer than the rows, count as one group
  p.rows_per_gate = p.gate_kind == MOE_FFN_GATE_VECTOR && a->rows_per_gate < a->rows ? a->rows_per_gate : a->rows;
  p.scale = a->residual_scale;
  p.eps = a->eps;
  p.state = a->state;
  p.ld_state = a->ld_state;
  p.f = a->f;
  p.ld_f = a->ld_f;
  p.gate = a->gate;
  p.w_post = a->norm_f;
  p.w_next = a->norm_next;
  return p;
}

int64_t gate_rows(const moe_ffn_block_norm_args *a) {
  return a->gate_kind == MOE_FFN_GATE_VECTOR ? ((int64_t)a->rows + a->rows_per_gate - 1) / a->rows_per_gate : a->rows;
}

// the tensors that both directions read
int norm_inputs(const moe_ffn_block_norm_args *a, Span *ins) {
  const bool vec = a->gate_kind == MOE_FFN_GATE_VECTOR;
  ins[0] = span("state", a->state, a->rows, a->hidden, a->ld_state, type_bytes(a->stream_type));
  ins[1] = span("f", a->f, a->rows, a->hidden, a->ld_f, type_bytes(a->block_type));
  ins[2] = a->gate_kind == MOE_FFN_GATE_NONE
               ? span("gate", nullptr, 0, 0, 0, 1)
               : span("gate", a->gate, gate_rows(a), vec ? a->hidden : 1, vec ? a->hidden : 1, type_bytes(a->gate_type));
  ins[3] = span("norm_f", a->norm_f, 1, a->hidden, a->hidden, 4);
  ins[4] = span("norm_next", a->norm_next, 1, a->hidden, a->hidden, 4);
  return 5;
}

int check_norm_grads(const char *who, const moe_ffn_block_norm_args *a, const moe_ffn_block_norm_grads *g) {
  int rc = check_norm(who, a);
  if (rc) return rc;
  if (!g) return fail(MOE_FFN_ERR_NULL_PTR, "%s: grads is NULL", who);
  if (!g->d_state || (a->f && !g->d_f) || (a->norm_next && !g->d_y))
    return fail(MOE_FFN_ERR_NULL_PTR, "%s: d_state, d_f or d_y is NULL", who);
  if ((!a->norm_next && (g->d_y || g->d_norm_next)) || (!a->f && g->d_f) || (!a->norm_f && g->d_norm_f) ||
      (a->gate_kind == MOE_FFN_GATE_NONE && g->d_gate))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a gradient of something that is not given", who);
  if ((g->d_out && g->ld_d_out < a->hidden) || (g->d_y && g->ld_d_y < a->hidden) || g->ld_d_state < a->hidden ||
      (g->d_f && g->ld_d_f < a->hidden))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a row stride is below hidden", who);
  return MOE_FFN_OK;
}

moe::NormParams norm_grad_params(const moe_ffn_block_norm_args *a, const moe_ffn_block_norm_grads *g) {
  moe::NormParams p = norm_params(a);
  p.d_out = g->d_out;
  p.ld_d_out = g->ld_d_out;
  p.d_y = g->d_y;
  p.ld_d_y = g->ld_d_y;
  p.d_state = g->d_state;
  p.ld_d_state = g->ld_d_state;
  p.d_f = g->d_f;
  p.ld_d_f = g->ld_d_f;
  p.d_gate = g->d_gate;
  p.d_w_post = g->d_norm_f;
  p.d_w_next = g->d_norm_next;
  p.part = static_cast<float *>(g->workspace);
  return p;
}

}  // namespace

extern "C" int moe_ffn_block_norm(const moe_ffn_block_norm_args *a, void *stream) {
  const char *who = "block_norm";
  int rc = check_norm(who, a);
  if (rc) return rc;
  if ((a->f != nullptr) != (a->out != nullptr)) return fail(MOE_FFN_ERR_NULL_PTR, "%s: out goes with f", who);
  if ((a->norm_next != nullptr) != (a->y != nullptr)) return fail(MOE_FFN_ERR_NULL_PTR, "%s: y goes with norm_next", who);
  if ((a->out && a->ld_out < a->hidden) || (a->y && a->ld_y < a->hidden))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a row stride is below hidden", who);
  const int sb = type_bytes(a->stream_type), bb = type_bytes(a->block_type);
  if (!aligned(a->out, sb) || !aligned(a->y, bb))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: a pointer is not aligned to its type", who);
  Span ins[5], outs[2] = {span("out", a->out, a->rows, a->hidden, a->ld_out, sb),
                          span("y", a->y, a->rows, a->hidden, a->ld_y, bb)};
  const int n_ins = norm_inputs(a, ins);
  if ((rc = check_overlaps(who, outs, 2, ins, n_ins, 0, 0))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::NormParams p = norm_params(a);
  p.out = a->out;
  p.ld_out = a->ld_out;
  p.y = a->y;
  p.ld_y = a->ld_y;
  return launched(who, moe::launch_block_norm(p, sms, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t moe_ffn_block_norm_workspace(const moe_ffn_block_norm_args *a, const moe_ffn_block_norm_grads *g) {
  const int rc = check_norm_grads("block_norm_workspace", a, g);
  if (rc) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  return (int64_t)(moe::norm_bwd_plan(norm_grad_params(a, g), sms).floats * sizeof(float));
}

extern "C" int moe_ffn_block_norm_backward(const moe_ffn_block_norm_args *a, const moe_ffn_block_norm_grads *g,
                                           void *stream) {
  const char *who = "block_norm_backward";
  int rc = check_norm_grads(who, a, g);
  if (rc) return rc;
  const int sb = type_bytes(a->stream_type), bb = type_bytes(a->block_type), gb = type_bytes(a->gate_type);
  if (!aligned(g->d_out, sb) || !aligned(g->d_y, bb) || !aligned(g->d_state, sb) || !aligned(g->d_f, bb) ||
      !aligned(g->d_gate, gb) || !aligned(g->d_norm_f, 4) || !aligned(g->d_norm_next, 4) || !aligned(g->workspace, 16))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: a pointer is not aligned to its type (workspace: 16 bytes)", who);
  const bool vec = a->gate_kind == MOE_FFN_GATE_VECTOR;
  const int64_t R = a->rows, H = a->hidden;
  Span ins[7], outs[6] = {span("d_state", g->d_state, R, H, g->ld_d_state, sb), span("d_f", g->d_f, R, H, g->ld_d_f, bb),
                          span("d_gate", g->d_gate, g->d_gate ? gate_rows(a) : 0, vec ? H : 1, vec ? H : 1, gb),
                          span("d_norm_f", g->d_norm_f, 1, H, H, 4), span("d_norm_next", g->d_norm_next, 1, H, H, 4),
                          span("workspace", g->workspace, 1, (int64_t)g->workspace_bytes, 0, 1)};
  ins[0] = span("d_out", g->d_out, R, H, g->ld_d_out, sb);
  ins[1] = span("d_y", g->d_y, R, H, g->ld_d_y, bb);
  norm_inputs(a, ins + 2);
  if ((rc = check_overlaps(who, outs, 6, ins, 7, 0, 0))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  const moe::NormParams p = norm_grad_params(a, g);
  const size_t need = moe::norm_bwd_plan(p, sms).floats * sizeof(float);
  if (need && !g->workspace) return fail(MOE_FFN_ERR_NULL_PTR, "%s: workspace is NULL", who);
  if (g->workspace_bytes < need)
    return fail(MOE_FFN_ERR_NO_MEMORY, "%s: workspace of %zu bytes, needs %zu", who, g->workspace_bytes, need);
  if ((rc = pending(who))) return rc;
  return launched(who, moe::launch_block_norm_backward(p, sms, static_cast<cudaStream_t>(stream)));
}
