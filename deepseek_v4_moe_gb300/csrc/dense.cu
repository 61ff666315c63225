// C entry points of the dense feed-forward sublayer on a plain residual stream: argument checks and
// launches (include/moe_ffn.h documents each).  No handle: the only state is what is known of each
// device.
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>
#include <mutex>

#include "dense.h"
#include "entry.h"
#include "kernels.h"
#include "moe_ffn.h"

namespace {

using namespace moe::entry;

// ---- what the tensor-core kernels share: status word, wait bound, tensor maps ----

__device__ int g_status;      // device status bits since the last moe_ffn_dense_status
__device__ int g_status_out;  // what that call reads

__global__ void take_status_kernel() { g_status_out = atomicExch(&g_status, 0); }

std::atomic<int> g_inject{0};
std::atomic<unsigned> g_wait_us{0};

}  // namespace

int moe::entry::device_side(const char *who, DeviceSide *d) {
  static std::atomic<int *> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return fail(MOE_FFN_ERR_CUDA, "%s: no usable current device", who);
  }
  d->status = known[dev].load(std::memory_order_acquire);
  if (!d->status) {
    void *p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_status);
    if (e != cudaSuccess || !p) return cuda_failed(who, "cudaGetSymbolAddress", e);
    d->status = static_cast<int *>(p);
    known[dev].store(d->status, std::memory_order_release);
  }
  const unsigned us = g_wait_us.load(std::memory_order_relaxed);
  d->wait_ns = us ? (uint64_t)us * 1000u : 2000000000ull;
  d->inject = g_inject.load(std::memory_order_relaxed);
  return MOE_FFN_OK;
}

namespace {

// ---- block_norm ----

int check_norm(const char *who, const moe_ffn_block_norm_args *a) {
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  // a group of rows past the last, or the rows of all CTAs, added to a row's number stay below 2^31
  if (a->rows < 0 || a->rows > (1 << 30)) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most 2^30", who);
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
  int rc = check_stride(who, "state", a->ld_state, a->rows, a->hidden);
  if (!rc && a->f) rc = check_stride(who, "f", a->ld_f, a->rows, a->hidden);
  if (rc) return rc;
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
  const int64_t R = a->rows, H = a->hidden;
  if ((g->d_out && (rc = check_stride(who, "d_out", g->ld_d_out, R, H))) ||
      (g->d_y && (rc = check_stride(who, "d_y", g->ld_d_y, R, H))) ||
      (rc = check_stride(who, "d_state", g->ld_d_state, R, H)) ||
      (g->d_f && (rc = check_stride(who, "d_f", g->ld_d_f, R, H))))
    return rc;
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

// ---- gated block ----

int check_gated(const char *who, const moe_ffn_gated_args *a) {
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0 || a->rows > (1 << 24)) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most 2^24", who);
  if (a->hidden < 8 || a->hidden % 8 || a->hidden > 65536 || a->inter < 8 || a->inter % 8 || a->inter > 65536)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: hidden and inter must be multiples of 8 in 8..65536", who);
  if (a->type != MOE_FFN_BF16 && a->type != MOE_FFN_F16)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: type must be bf16 or f16", who);
  if (a->activation != MOE_FFN_ACT_SILU && a->activation != MOE_FFN_ACT_GELU)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown activation", who);
  return MOE_FFN_OK;
}

int check_rows_of(const char *who, const char *name, const void *p, int64_t ld, int64_t cols) {
  if (!p) return fail(MOE_FFN_ERR_NULL_PTR, "%s: %s is NULL", who, name);
  if (ld < cols || ld % 8 || ld > kLdMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of %s must be a multiple of 8, at least %lld", who, name, (long long)cols);
  if (!aligned(p, 16)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: %s is not 16-byte aligned", who, name);
  return MOE_FFN_OK;
}

moe::GemmParams gemm_params(const moe_ffn_gated_args *a, const DeviceSide &d) {
  moe::GemmParams p = {};
  p.act = a->activation;
  p.f16 = a->type == MOE_FFN_F16;
  p.a_rows = moe::a_box(a->rows);
  p.odd_rows = a->hidden % 64 != 0 || a->inter % 64 != 0 || a->ld_x % 64 != 0;
  p.status = d.status;
  p.wait_ns = d.wait_ns;
  p.inject = d.inject;
  return p;
}
void add_problem(moe::GemmParams &p, int m, int n, int kb0, int kb, int a, int b, bool a_mn, void *c, int64_t ldc) {
  p.problem[p.problems++] = moe::GemmProblem{m, n, kb0, kb, a, b, a_mn, 0, 0, 0, c, ldc};
}

// inter columns of a row of the workspace's buffers: h forward; dg, du and h backward
int64_t gated_workspace(const moe_ffn_gated_args *a, bool backward) {
  return (int64_t)a->rows * a->inter * 2 * (backward ? 3 : 1);
}

int kblocks(int k) { return (k + 63) / 64; }

// A launch of a call: its products, and the tile that they take on a GPU of so many SMs.
struct Launch {
  int mode;
  moe::GemmParams p;
  moe::DenseTile tile;
};
void pick(Launch &l, int sms) {
  double t;
  l.tile = moe::gemm_pick_tile(l.mode, l.p, sms, &t);
}

void forward_launches(const moe_ffn_gated_args *a, const DeviceSide &dev, int sms, Launch (&l)[2]) {
  const int kh = kblocks(a->hidden), ki = kblocks(a->inter);
  Launch &up = l[0], &down = l[1];
  up.mode = moe::kGateUp;
  down.mode = moe::kDown;
  up.p = down.p = gemm_params(a, dev);
  add_problem(up.p, a->rows, a->inter, kh, kh, 0, 0, false, nullptr, 0);
  up.p.out[0] = a->workspace;
  up.p.out[1] = a->gate;
  up.p.out[2] = a->up;
  add_problem(down.p, a->rows, a->hidden, ki, ki, 0, 0, false, a->y, a->ld_y);
  pick(up, sms);
  pick(down, sms);
}

// The backward pass's launches, two or three; `x`, `weights`: which gradients are wanted.
int backward_launches(const moe_ffn_gated_args *a, bool x, bool weights, const DeviceSide &dev, int sms, Launch (&l)[3]) {
  const int kh = kblocks(a->hidden), ki = kblocks(a->inter), kr = kblocks(a->rows);
  const int64_t H = a->hidden, I = a->inter;
  Launch &hid = l[0];
  hid.mode = moe::kHiddenGrad;
  hid.p = gemm_params(a, dev);
  moe::GemmParams all = hid.p, dx = all, dw = all;
  char *dg = static_cast<char *>(a->workspace);
  add_problem(hid.p, a->rows, a->inter, kh, kh, 0, 0, false, nullptr, 0);
  hid.p.out[0] = dg;
  hid.p.out[1] = dg + a->rows * I * 2;
  hid.p.out[2] = dg + a->rows * I * 4;
  hid.p.e[0] = a->gate;
  hid.p.e[1] = a->up;
  pick(hid, sms);
  if (x) add_problem(dx, a->rows, a->hidden, ki, 2 * ki, 0, 0, false, a->d_x, a->ld_d_x);
  dw.a_rows = 128;  // its A is MN-major
  if (weights) {
    add_problem(dw, a->inter, a->hidden, kr, kr, 2, 2, true, a->d_w_gate, H);
    add_problem(dw, a->inter, a->hidden, kr, kr, 3, 2, true, a->d_w_up, H);
    add_problem(dw, a->hidden, a->inter, kr, kr, 4, 3, true, a->d_w_down, I);
  }
  // one launch for all, the tiles with more k first, unless two take less time
  for (const moe::GemmParams *p : {2 * ki >= kr ? &dx : &dw, 2 * ki >= kr ? &dw : &dx})
    for (int i = 0; i < p->problems; ++i) all.problem[all.problems++] = p->problem[i];
  if (!x) all.a_rows = dw.a_rows;
  double t_all, t_dx, t_dw;
  l[1] = Launch{moe::kGrads, all, moe::gemm_pick_tile(moe::kGrads, all, sms, &t_all)};
  if (x && weights) {
    const moe::DenseTile tx = moe::gemm_pick_tile(moe::kGrads, dx, sms, &t_dx), tw = moe::gemm_pick_tile(moe::kGrads, dw, sms, &t_dw);
    if (t_dx + t_dw < t_all) {
      l[1] = Launch{moe::kGrads, dx, tx};
      l[2] = Launch{moe::kGrads, dw, tw};
      return 3;
    }
  }
  return 2;
}

}  // namespace

extern "C" int64_t moe_ffn_gated_workspace(const moe_ffn_gated_args *a, int32_t backward) {
  const int rc = check_gated("gated_workspace", a);
  return rc ? rc : gated_workspace(a, backward != 0);
}

extern "C" int moe_ffn_gated_forward(const moe_ffn_gated_args *a, void *stream) {
  const char *who = "gated_forward";
  int rc = check_gated(who, a);
  if (rc) return rc;
  const int64_t R = a->rows, H = a->hidden, I = a->inter;
  if ((rc = check_rows_of(who, "x", a->x, a->ld_x, H)) || (rc = check_rows_of(who, "y", a->y, a->ld_y, H)) ||
      (rc = check_rows_of(who, "w_gate", a->w_gate, H, H)) || (rc = check_rows_of(who, "w_up", a->w_up, H, H)) ||
      (rc = check_rows_of(who, "w_down", a->w_down, I, I)) ||
      (rc = check_rows_of(who, "workspace", a->workspace, I, I)))
    return rc;
  if ((a->gate != nullptr) != (a->up != nullptr)) return fail(MOE_FFN_ERR_NULL_PTR, "%s: gate and up go together", who);
  if (!aligned(a->gate, 16) || !aligned(a->up, 16)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: gate or up is not 16-byte aligned", who);
  const int64_t need = gated_workspace(a, false);
  if (a->workspace_bytes < (size_t)need)
    return fail(MOE_FFN_ERR_NO_MEMORY, "%s: workspace of %zu bytes, needs %lld", who, a->workspace_bytes, (long long)need);
  const Span ins[] = {span("x", a->x, R, H, a->ld_x, 2), span("w_gate", a->w_gate, I, H, H, 2),
                      span("w_up", a->w_up, I, H, H, 2), span("w_down", a->w_down, H, I, I, 2)};
  const Span outs[] = {span("y", a->y, R, H, a->ld_y, 2), span("gate", a->gate, R, I, I, 2), span("up", a->up, R, I, I, 2),
                       span("workspace", a->workspace, 1, need, 0, 1)};
  if ((rc = check_overlaps(who, outs, 4, ins, 4, -1, -1))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (moe::gated_gemv(a->rows, a->hidden, a->inter)) {
    moe::GemvParams p = {};
    p.n = a->inter;
    p.k = a->hidden;
    p.act = a->activation;
    p.x = a->x;
    p.ld_x = a->ld_x;
    p.w[0] = a->w_gate;
    p.w[1] = a->w_up;
    p.out = a->workspace;
    p.gate = a->gate;
    p.up = a->up;
    cudaError_t e = moe::launch_gated_gemv(true, p, a->rows, a->type == MOE_FFN_F16, st);
    if (e != cudaSuccess) return launched(who, e);
    p.n = a->hidden;
    p.k = a->inter;
    p.x = a->workspace;
    p.ld_x = I;
    p.w[0] = a->w_down;
    p.out = a->y;
    p.ld_out = a->ld_y;
    return launched(who, moe::launch_gated_gemv(false, p, a->rows, a->type == MOE_FFN_F16, st));
  }
  DeviceSide dev;
  if ((rc = device_side(who, &dev))) return rc;
  Launch l[2];
  forward_launches(a, dev, sms, l);
  const Launch &up = l[0], &down = l[1];
  const int bu = moe::gemm_b_box(moe::kGateUp, up.tile), bd = moe::gemm_b_box(moe::kDown, down.tile);
  moe::GemmMaps mu, md;
  if (!encode_map(&mu.a[0], a->x, 2, H, R, a->ld_x, up.p.a_rows) || !encode_map(&mu.b[0], a->w_gate, 2, H, I, H, bu) ||
      !encode_map(&mu.b[1], a->w_up, 2, H, I, H, bu) || !encode_map(&md.a[0], a->workspace, 2, I, R, I, down.p.a_rows) ||
      !encode_map(&md.b[0], a->w_down, 2, I, H, I, bd))
    return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  cudaError_t e = moe::launch_dense_gemm(up.mode, up.tile, mu, up.p, sms, st);
  if (e == cudaSuccess) e = moe::launch_dense_gemm(down.mode, down.tile, md, down.p, sms, st);
  return launched(who, e);
}

extern "C" int moe_ffn_gated_backward(const moe_ffn_gated_args *a, void *stream) {
  const char *who = "gated_backward";
  int rc = check_gated(who, a);
  if (rc) return rc;
  const int64_t R = a->rows, H = a->hidden, I = a->inter;
  const bool weights = a->d_w_gate || a->d_w_up || a->d_w_down;
  if ((rc = check_rows_of(who, "x", a->x, a->ld_x, H)) || (rc = check_rows_of(who, "w_gate", a->w_gate, H, H)) ||
      (rc = check_rows_of(who, "w_up", a->w_up, H, H)) || (rc = check_rows_of(who, "w_down", a->w_down, I, I)) ||
      (rc = check_rows_of(who, "gate", a->gate, I, I)) || (rc = check_rows_of(who, "up", a->up, I, I)) ||
      (rc = check_rows_of(who, "d_y", a->d_y, a->ld_d_y, H)) ||
      (rc = check_rows_of(who, "workspace", a->workspace, I, I)) ||
      (a->d_x && (rc = check_rows_of(who, "d_x", a->d_x, a->ld_d_x, H))) ||
      (weights && ((rc = check_rows_of(who, "d_w_gate", a->d_w_gate, H, H)) ||
                   (rc = check_rows_of(who, "d_w_up", a->d_w_up, H, H)) ||
                   (rc = check_rows_of(who, "d_w_down", a->d_w_down, I, I)))))
    return rc;
  if (!a->d_x && !weights) return fail(MOE_FFN_ERR_NULL_PTR, "%s: no gradient is asked for", who);
  const int64_t need = gated_workspace(a, true);
  if (a->workspace_bytes < (size_t)need)
    return fail(MOE_FFN_ERR_NO_MEMORY, "%s: workspace of %zu bytes, needs %lld", who, a->workspace_bytes, (long long)need);
  const Span ins[] = {span("x", a->x, R, H, a->ld_x, 2),       span("w_gate", a->w_gate, I, H, H, 2),
                      span("w_up", a->w_up, I, H, H, 2),       span("w_down", a->w_down, H, I, I, 2),
                      span("gate", a->gate, R, I, I, 2),       span("up", a->up, R, I, I, 2),
                      span("d_y", a->d_y, R, H, a->ld_d_y, 2)};
  const Span outs[] = {span("d_x", a->d_x, R, H, a->ld_d_x, 2),       span("d_w_gate", a->d_w_gate, I, H, H, 2),
                       span("d_w_up", a->d_w_up, I, H, H, 2),         span("d_w_down", a->d_w_down, H, I, I, 2),
                       span("workspace", a->workspace, 1, need, 0, 1)};
  if ((rc = check_overlaps(who, outs, 5, ins, 7, -1, -1))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  DeviceSide dev;
  if ((rc = device_side(who, &dev))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char *dg = static_cast<char *>(a->workspace), *du = dg + R * I * 2, *h = du + R * I * 2;

  Launch l[3];
  const int launches = backward_launches(a, a->d_x != nullptr, weights, dev, sms, l), box = l[0].p.a_rows;
  moe::GemmMaps mh, mg;
  if (!encode_map(&mh.a[0], a->d_y, 2, H, R, a->ld_d_y, box) || !encode_map(&mh.b[0], a->w_down, 2, I, H, I, 64) ||
      !encode_map(&mg.a[0], dg, 2, I, R, I, box) || !encode_map(&mg.a[1], du, 2, I, R, I, box) ||
      !encode_map(&mg.a[2], dg, 2, I, R, I, 64) || !encode_map(&mg.a[3], du, 2, I, R, I, 64) ||
      !encode_map(&mg.a[4], a->d_y, 2, H, R, a->ld_d_y, 64) || !encode_map(&mg.b[0], a->w_gate, 2, H, I, H, 64) ||
      !encode_map(&mg.b[1], a->w_up, 2, H, I, H, 64) || !encode_map(&mg.b[2], a->x, 2, H, R, a->ld_x, 64) ||
      !encode_map(&mg.b[3], h, 2, I, R, I, 64))
    return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < launches && e == cudaSuccess; ++i)
    e = moe::launch_dense_gemm(l[i].mode, l[i].tile, i ? mg : mh, l[i].p, sms, st);
  return launched(who, e);
}

extern "C" int moe_ffn_fp8_matmul(const moe_ffn_fp8_matmul_args *a, void *stream) {
  const char *who = "fp8_matmul";
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0 || a->rows > (1 << 24)) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most 2^24", who);
  if (a->n < 1 || a->n > (1 << 20) || a->k < 16 || a->k % 16 || a->k > (1 << 20))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: n must be in 1..2^20, k a multiple of 16 in 16..2^20", who);
  if ((a->a_type != MOE_FFN_E4M3 && a->a_type != MOE_FFN_E5M2) || (a->b_type != MOE_FFN_E4M3 && a->b_type != MOE_FFN_E5M2) ||
      !is_type(a->out_type))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown type", who);
  if (!a->a || !a->a_scale || !a->b || !a->b_scale || !a->out)
    return fail(MOE_FFN_ERR_NULL_PTR, "%s: a pointer is NULL", who);
  if (a->ld_a < a->k || a->ld_a % 16 || a->ld_a > kLdMax || a->ld_b < a->k || a->ld_b % 16 || a->ld_b > kLdMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row strides of a and b must be multiples of 16, at least k", who);
  if (a->ld_out < a->n || a->ld_out > kLdMax) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of out is below n", who);
  const int ob = type_bytes(a->out_type);
  if (!aligned(a->a, 16) || !aligned(a->b, 16) || !aligned(a->a_scale, 4) || !aligned(a->b_scale, 4) || !aligned(a->out, ob))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: a and b must be 16-byte aligned, the others to their type", who);
  const int64_t R = a->rows, N = a->n, K = a->k, KB = (K + 127) / 128;
  const Span ins[] = {span("a", a->a, R, K, a->ld_a, 1), span("a_scale", a->a_scale, R, KB, KB, 4),
                      span("b", a->b, N, K, a->ld_b, 1), span("b_scale", a->b_scale, (N + 127) / 128, KB, KB, 4)};
  const Span outs[] = {span("out", a->out, R, N, a->ld_out, ob)};
  int rc = check_overlaps(who, outs, 1, ins, 4, -1, -1);
  if (rc) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  if (moe::fp8_gemv(a->rows, a->n, a->k)) {
    moe::Fp8GemvParams p = {};
    p.n = a->n;
    p.k = a->k;
    p.kb = (int)KB;
    p.a_e5m2 = a->a_type == MOE_FFN_E5M2;
    p.b_e5m2 = a->b_type == MOE_FFN_E5M2;
    p.a = static_cast<const uint8_t *>(a->a);
    p.b = static_cast<const uint8_t *>(a->b);
    p.ld_a = a->ld_a;
    p.ld_b = a->ld_b;
    p.a_scale = a->a_scale;
    p.b_scale = a->b_scale;
    p.out = a->out;
    p.ld_out = a->ld_out;
    return launched(who, moe::launch_fp8_gemv(p, a->rows, sms, a->out_type, static_cast<cudaStream_t>(stream)));
  }
  DeviceSide dev;
  if ((rc = device_side(who, &dev))) return rc;
  moe::Fp8Params p = {};
  p.m = a->rows;
  p.n = a->n;
  p.kb = (int)KB;
  p.a_e5m2 = a->a_type == MOE_FFN_E5M2;
  p.b_e5m2 = a->b_type == MOE_FFN_E5M2;
  p.out_type = a->out_type;
  p.a_scale = a->a_scale;
  p.b_scale = a->b_scale;
  p.out = a->out;
  p.ld_out = a->ld_out;
  p.wide = aligned(a->out, 16) && a->ld_out * ob % 16 == 0;
  p.status = dev.status;
  p.wait_ns = dev.wait_ns;
  p.inject = dev.inject;
  p.a_rows = moe::a_box(a->rows);
  const moe::DenseTile t = moe::fp8_pick_tile(p, sms);
  CUtensorMap ma, mb;
  if (!encode_map(&ma, a->a, 1, K, R, a->ld_a, p.a_rows) ||
      !encode_map(&mb, a->b, 1, K, N, a->ld_b, t.kind == moe::kPairTile ? t.bn / 2 : t.bn))
    return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  return launched(who, moe::launch_fp8_matmul(t, ma, mb, p, sms, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_ffn_fp8_quantise(const moe_ffn_fp8_quantise_args *a, void *stream) {
  const char *who = "fp8_quantise";
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0 || a->rows > (1 << 24)) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most 2^24", who);
  if (a->k < 1 || a->k > (1 << 20)) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: k must be in 1..2^20", who);
  if (!is_type(a->type) || (a->code_type != MOE_FFN_E4M3 && a->code_type != MOE_FFN_E5M2))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown type", who);
  if (a->block_rows != 1 && a->block_rows != 128) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: block_rows must be 1 or 128", who);
  if (!a->x || !a->codes || !a->scales) return fail(MOE_FFN_ERR_NULL_PTR, "%s: a pointer is NULL", who);
  if (a->ld_x < a->k || a->ld_codes < a->k || a->ld_x > kLdMax || a->ld_codes > kLdMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a row stride is below k", who);
  const int xb = type_bytes(a->type);
  if (!aligned(a->x, xb) || !aligned(a->scales, 4)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: x or scales is misaligned", who);
  const int64_t R = a->rows, K = a->k, KB = (K + 127) / 128;
  const Span ins[] = {span("x", a->x, R, K, a->ld_x, xb)};
  const Span outs[] = {span("codes", a->codes, R, K, a->ld_codes, 1),
                       span("scales", a->scales, (R + a->block_rows - 1) / a->block_rows, KB, KB, 4)};
  int rc = check_overlaps(who, outs, 2, ins, 1, -1, -1);
  if (rc) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::QuantiseParams p = {};
  p.rows = a->rows;
  p.k = a->k;
  p.type = a->type;
  p.e5m2 = a->code_type == MOE_FFN_E5M2;
  p.pow2 = a->pow2 != 0;
  p.tall = a->block_rows;
  p.x = a->x;
  p.ld_x = a->ld_x;
  p.codes = static_cast<uint8_t *>(a->codes);
  p.ld_codes = a->ld_codes;
  p.scales = a->scales;
  p.wide = a->k % 8 == 0 && aligned(a->x, 8 * xb) && a->ld_x % 8 == 0 && aligned(a->codes, 8) && a->ld_codes % 8 == 0;
  return launched(who, moe::launch_fp8_quantise(p, sms, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_ffn_dense_status(void *stream) {
  const char *who = "dense_status";
  const int sms = current_sms();
  if (sms < 0) return sms;
  int rc = pending(who);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(st, &capture);
  if (e != cudaSuccess) return cuda_failed(who, "cudaStreamIsCapturing", e);
  if (capture != cudaStreamCaptureStatusNone)
    return fail(MOE_FFN_ERR_UNSUPPORTED, "%s: the stream is being captured", who);
  static std::mutex one_at_a_time;  // g_status_out holds one call's bits until they are copied
  const std::lock_guard<std::mutex> lock(one_at_a_time);
  take_status_kernel<<<1, 1, 0, st>>>();
  int bits = 0;
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&bits, g_status_out, sizeof bits, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return e == cudaSuccess ? bits : cuda_failed(who, "reading the status", e);
}

extern "C" int moe_ffn_dense_tiles(int32_t call, int32_t rows, int32_t n, int32_t k, int32_t num_sms, int32_t *tiles) {
  const char *who = "dense_tiles";
  if (!tiles) return fail(MOE_FFN_ERR_NULL_PTR, "%s: tiles is NULL", who);
  if (num_sms < 8 || num_sms > 4096) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: num_sms must be in 8..4096", who);
  int count = 0;
  auto add = [&](int product, moe::DenseTile t) {
    *tiles++ = product;
    *tiles++ = t.bn;
    *tiles++ = t.kind;
    ++count;
  };
  if (call == MOE_FFN_TILES_FP8) {
    if (rows < 1 || rows > (1 << 24) || n < 1 || n > (1 << 20) || k < 16 || k % 16 || k > (1 << 20))
      return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: rows, n or k is not one of an fp8_matmul", who);
    if (moe::fp8_gemv(rows, n, k)) return 0;
    moe::Fp8Params p = {};
    p.m = rows;
    p.n = n;
    p.kb = (k + 127) / 128;
    add(4, moe::fp8_pick_tile(p, num_sms));
    return count;
  }
  moe_ffn_gated_args a = {};
  a.rows = rows;
  a.hidden = k;
  a.inter = n;
  a.type = MOE_FFN_BF16;
  a.ld_x = k;
  int rc = check_gated(who, &a);
  if (rc) return rc;
  if (call == MOE_FFN_TILES_FORWARD) {
    if (moe::gated_gemv(rows, k, n)) return 0;
    Launch l[2];
    forward_launches(&a, DeviceSide{}, num_sms, l);
    for (const Launch &x : l) add(x.mode, x.tile);
    return count;
  }
  if (call != MOE_FFN_TILES_BACKWARD && call != MOE_FFN_TILES_BACKWARD_X && call != MOE_FFN_TILES_BACKWARD_WEIGHTS)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown call", who);
  Launch l[3];
  const int launches = backward_launches(&a, call != MOE_FFN_TILES_BACKWARD_WEIGHTS, call != MOE_FFN_TILES_BACKWARD_X,
                                         DeviceSide{}, num_sms, l);
  for (int i = 0; i < launches; ++i) add(l[i].mode, l[i].tile);
  return count;
}

extern "C" int moe_ffn_dense_fault_injection(int32_t enable, uint32_t wait_limit_us) {
  g_inject.store(enable != 0, std::memory_order_relaxed);
  g_wait_us.store(wait_limit_us, std::memory_order_relaxed);
  return MOE_FFN_OK;
}

namespace {

// block_norm, with y in its type or (o) as FP8 codes and scales
int block_norm(const char *who, const moe_ffn_block_norm_args *a, const moe_ffn_fp8_out *o, void *stream) {
  int rc = check_norm(who, a);
  if (rc) return rc;
  if ((a->f != nullptr) != (a->out != nullptr)) return fail(MOE_FFN_ERR_NULL_PTR, "%s: out goes with f", who);
  if (o) {
    if (!a->norm_next || !o->codes || !o->scales) return fail(MOE_FFN_ERR_NULL_PTR, "%s: norm_next, codes or scales is NULL", who);
    if (a->y) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: y is not written", who);
    if (o->code_type != MOE_FFN_E4M3 && o->code_type != MOE_FFN_E5M2) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown type", who);
    if ((rc = check_stride(who, "codes", o->ld_codes, a->rows, a->hidden))) return rc;
  } else if ((a->norm_next != nullptr) != (a->y != nullptr)) {
    return fail(MOE_FFN_ERR_NULL_PTR, "%s: y goes with norm_next", who);
  }
  if ((a->out && (rc = check_stride(who, "out", a->ld_out, a->rows, a->hidden))) ||
      (a->y && (rc = check_stride(who, "y", a->ld_y, a->rows, a->hidden))))
    return rc;
  const int sb = type_bytes(a->stream_type), bb = type_bytes(a->block_type);
  if (!aligned(a->out, sb) || !aligned(a->y, bb) || (o && !aligned(o->scales, 4)))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: a pointer is not aligned to its type", who);
  const int64_t blocks = (a->hidden + moe::kScaleBlock - 1) / moe::kScaleBlock;
  Span ins[5], outs[4] = {span("out", a->out, a->rows, a->hidden, a->ld_out, sb), span("y", a->y, a->rows, a->hidden, a->ld_y, bb),
                          span("codes", o ? o->codes : nullptr, a->rows, a->hidden, o ? o->ld_codes : 0, 1),
                          span("scales", o ? o->scales : nullptr, a->rows, blocks, blocks, 4)};
  const int n_ins = norm_inputs(a, ins);
  if ((rc = check_overlaps(who, outs, 4, ins, n_ins, 0, 0))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::NormParams p = norm_params(a);
  p.out = a->out;
  p.ld_out = a->ld_out;
  p.y = a->y;
  p.ld_y = a->ld_y;
  if (o) {
    p.codes = static_cast<uint8_t *>(o->codes);
    p.ld_codes = o->ld_codes;
    p.scales = o->scales;
    p.e5m2 = o->code_type == MOE_FFN_E5M2;
    p.pow2 = o->pow2 != 0;
  }
  return launched(who, moe::launch_block_norm(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" int moe_ffn_block_norm(const moe_ffn_block_norm_args *a, void *stream) {
  return block_norm("block_norm", a, nullptr, stream);
}

extern "C" int moe_ffn_block_norm_fp8(const moe_ffn_block_norm_args *a, const moe_ffn_fp8_out *o, void *stream) {
  const char *who = "block_norm_fp8";
  if (!o) return fail(MOE_FFN_ERR_NULL_PTR, "%s: out is NULL", who);
  return block_norm(who, a, o, stream);
}

extern "C" int moe_ffn_gated_quantise(const moe_ffn_gated_quantise_args *a, const moe_ffn_fp8_out *o, void *stream) {
  const char *who = "gated_quantise";
  if (!a || !o) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args or out is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0 || a->rows > (1 << 24)) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most 2^24", who);
  if (a->columns < 1 || a->columns > (1 << 20)) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: columns must be in 1..2^20", who);
  if ((a->type != MOE_FFN_BF16 && a->type != MOE_FFN_F16) || (o->code_type != MOE_FFN_E4M3 && o->code_type != MOE_FFN_E5M2))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown type", who);
  if (a->activation != MOE_FFN_ACT_SILU && a->activation != MOE_FFN_ACT_GELU)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown activation", who);
  if (!a->gate || !a->up || !o->codes || !o->scales) return fail(MOE_FFN_ERR_NULL_PTR, "%s: a pointer is NULL", who);
  if (a->ld_gate < a->columns || a->ld_up < a->columns || o->ld_codes < a->columns || a->ld_gate > kLdMax ||
      a->ld_up > kLdMax || o->ld_codes > kLdMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: a row stride is below the columns", who);
  if (!aligned(a->gate, 2) || !aligned(a->up, 2) || !aligned(o->scales, 4))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: gate, up or scales is misaligned", who);
  const int64_t R = a->rows, K = a->columns, KB = (K + 127) / 128;
  const Span ins[] = {span("gate", a->gate, R, K, a->ld_gate, 2), span("up", a->up, R, K, a->ld_up, 2)};
  const Span outs[] = {span("codes", o->codes, R, K, o->ld_codes, 1), span("scales", o->scales, R, KB, KB, 4)};
  int rc = check_overlaps(who, outs, 2, ins, 2, -1, -1);
  if (rc) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::GatedQuantiseParams p = {};
  p.q.rows = a->rows;
  p.q.k = a->columns;
  p.q.type = a->type;
  p.q.e5m2 = o->code_type == MOE_FFN_E5M2;
  p.q.pow2 = o->pow2 != 0;
  p.q.tall = 1;
  p.q.x = a->gate;
  p.q.ld_x = a->ld_gate;
  p.q.codes = static_cast<uint8_t *>(o->codes);
  p.q.ld_codes = o->ld_codes;
  p.q.scales = o->scales;
  p.q.wide = K % 8 == 0 && aligned(a->gate, 16) && a->ld_gate % 8 == 0 && aligned(a->up, 16) && a->ld_up % 8 == 0 &&
             aligned(o->codes, 8) && o->ld_codes % 8 == 0;
  p.up = a->up;
  p.ld_up = a->ld_up;
  p.act = a->activation;
  return launched(who, moe::launch_gated_quantise(p, sms, static_cast<cudaStream_t>(stream)));
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
      !aligned(g->d_gate, gb) || !aligned(g->d_norm_f, 4) || !aligned(g->d_norm_next, 4) || !aligned(g->workspace, 32))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: a pointer is not aligned to its type (workspace: 32 bytes)", who);
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
