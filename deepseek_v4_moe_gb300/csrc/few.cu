// C entry points of the products with 4-bit weights and of the routed layer without a handle: argument checks and
// launches (include/moe_ffn.h documents each).
#include "few.h"

#include "entry.h"

namespace {

using namespace moe::entry;

constexpr int kCodesMax = 1 << 20, kCodeRowsMax = 1 << 24;

int check_group(const char *who, int group) {
  if (group != 32 && group != 64 && group != 128) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: group must be 32, 64 or 128", who);
  return MOE_FFN_OK;
}
bool type16(int t) { return t == MOE_FFN_BF16 || t == MOE_FFN_F16; }

int check_int4_sizes(const char *who, int64_t n, int64_t k, int group) {
  if (n < 1 || n > kCodeRowsMax || k < 32 || k % 32 || k > kCodesMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: n must be in 1..2^24, k a multiple of 32 in 32..2^20", who);
  return check_group(who, group);
}

int check_int4(const char *who, int64_t n, int64_t k, int group, const void *codes, const void *scales, const void *zeros) {
  const int rc = check_int4_sizes(who, n, k, group);
  if (rc) return rc;
  if (!codes || !scales) return fail(MOE_FFN_ERR_NULL_PTR, "%s: codes or scales is NULL", who);
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(zeros, 16))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: codes, scales and zeros must be 16-byte aligned", who);
  return MOE_FFN_OK;
}

int log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

moe::FewMatrix matrix(const void *w, const void *scales, const uint8_t *zeros, int64_t n, int64_t k, int group) {
  const int groups = (int)((k + group - 1) / group);
  return moe::FewMatrix{w, static_cast<const uint16_t *>(scales), zeros, (int)n, (int)k, groups, log2_of(group)};
}

// rows of x or of a result in 16-byte pieces
int check_rows16(const char *who, const char *name, const void *p, int64_t ld, int64_t cols) {
  if (!p) return fail(MOE_FFN_ERR_NULL_PTR, "%s: %s is NULL", who, name);
  if (ld < cols || ld % 8 || ld > kLdMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of %s must be a multiple of 8, at least %lld", who, name, (long long)cols);
  if (!aligned(p, 16)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: %s is not 16-byte aligned", who, name);
  return MOE_FFN_OK;
}
// rows that are written value by value
int check_rows2(const char *who, const char *name, const void *p, int64_t ld, int64_t cols) {
  if (!p) return fail(MOE_FFN_ERR_NULL_PTR, "%s: %s is NULL", who, name);
  if (ld < cols || ld > kLdMax) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of %s is below %lld", who, name, (long long)cols);
  if (!aligned(p, 2)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: %s is misaligned", who, name);
  return MOE_FFN_OK;
}

int check_weights(const char *who, const moe_ffn_int4_weights_args *a) {
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  int rc = check_int4(who, a->n, a->k, a->group, a->codes, a->scales, a->zeros);
  if (rc) return rc;
  if (!type16(a->scale_type)) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: scale_type must be bf16 or f16", who);
  return MOE_FFN_OK;
}

moe::Int4WeightParams weight_params(const moe_ffn_int4_weights_args *a) {
  moe::Int4WeightParams p = {};
  p.n = a->n;
  p.k = a->k;
  p.group = a->group;
  p.codes = a->codes;
  p.scales = a->scales;
  p.zeros = a->zeros;
  p.f16 = a->scale_type == MOE_FFN_F16;
  return p;
}

int weight_spans(const moe_ffn_int4_weights_args *a, Span *s) {
  const int64_t groups = (a->k + a->group - 1) / a->group;
  s[0] = span("codes", a->codes, a->n, a->k / 2, a->k / 2, 1);
  s[1] = span("scales", a->scales, a->n, groups, groups, 2);
  s[2] = span("zeros", a->zeros, a->n, groups, groups, 1);
  return 3;
}

}  // namespace

extern "C" int moe_ffn_int4_quantise(const moe_ffn_int4_weights_args *a, const void *w, int32_t type, int64_t ld_w, void *stream) {
  const char *who = "int4_quantise";
  int rc = check_weights(who, a);
  if (rc) return rc;
  if (!is_type(type)) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown type", who);
  if (!w) return fail(MOE_FFN_ERR_NULL_PTR, "%s: w is NULL", who);
  if (ld_w < a->k || ld_w % 8 || ld_w > kLdMax)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of w must be a multiple of 8, at least k", who);
  const int bytes = type_bytes(type);
  if (!aligned(w, 8 * bytes)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: w is not aligned to eight values", who);
  Span outs[3];
  const Span ins[] = {span("w", w, a->n, a->k, ld_w, bytes)};
  if ((rc = check_overlaps(who, outs, weight_spans(a, outs), ins, 1, -1, -1))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::Int4WeightParams p = weight_params(a);
  p.type = type;
  p.w = w;
  p.ld_w = ld_w;
  return launched(who, moe::launch_int4_quantise(p, sms, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_ffn_int4_widen(const moe_ffn_int4_weights_args *a, void *out, int64_t ld_out, void *stream) {
  const char *who = "int4_widen";
  int rc = check_weights(who, a);
  if (rc) return rc;
  if ((rc = check_rows16(who, "out", out, ld_out, a->k))) return rc;
  Span ins[3];
  const Span outs[] = {span("out", out, a->n, a->k, ld_out, 2)};
  if ((rc = check_overlaps(who, outs, 1, ins, weight_spans(a, ins), -1, -1))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::Int4WeightParams p = weight_params(a);
  p.out = out;
  p.ld_out = ld_out;
  return launched(who, moe::launch_int4_widen(p, sms, static_cast<cudaStream_t>(stream)));
}

namespace {

// where the parts of the FP8 form lie in the workspace
struct Int4Space {
  int64_t sums, back, bytes;
  int groups, rows;  // rows of the planes
};
Int4Space int4_space(const moe_ffn_int4_matmul_args *a, int tokens) {
  Int4Space s;
  const int planes = a->type == MOE_FFN_F16 ? 3 : 2;
  const int64_t blocks = (a->rows + tokens - 1) / tokens;
  const int columns = 128 * moe::code_halves(tokens, planes, 128 / a->group);  // of a tile
  s.groups = (int)((a->k + columns - 1) / columns * (columns / a->group));
  s.rows = (int)(blocks * planes * tokens);
  s.sums = ((int64_t)s.rows * a->k + 255) / 256 * 256;
  s.back = s.sums + (blocks * s.groups * tokens * 4 + 255) / 256 * 256;
  s.bytes = s.back + (int64_t)a->rows * 4;
  return s;
}

int check_int4_matmul(const char *who, const moe_ffn_int4_matmul_args *a) {
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0 || a->rows > (1 << 16)) return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most 2^16", who);
  if (!type16(a->type)) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: type must be bf16 or f16", who);
  return check_int4_sizes(who, a->n, a->k, a->group);
}

}  // namespace

extern "C" int64_t moe_ffn_int4_matmul_workspace(const moe_ffn_int4_matmul_args *a) {
  const int rc = check_int4_matmul("int4_matmul_workspace", a);
  if (rc) return rc;
  const int tokens = moe::int4_tc_tokens(a->rows, a->n, a->k, a->group);
  return tokens ? int4_space(a, tokens).bytes : 0;
}

extern "C" int moe_ffn_int4_matmul(const moe_ffn_int4_matmul_args *a, void *stream) {
  const char *who = "int4_matmul";
  int rc = check_int4_matmul(who, a);
  if (rc) return rc;
  rc = check_int4(who, a->n, a->k, a->group, a->codes, a->scales, a->zeros);
  if (rc) return rc;
  const int64_t R = a->rows, N = a->n, K = a->k, G = (K + a->group - 1) / a->group;
  if ((rc = check_rows16(who, "x", a->x, a->ld_x, K)) || (rc = check_rows2(who, "out", a->out, a->ld_out, N))) return rc;
  const Span ins[] = {span("x", a->x, R, K, a->ld_x, 2), span("codes", a->codes, N, K / 2, K / 2, 1),
                      span("scales", a->scales, N, G, G, 2), span("zeros", a->zeros, N, G, G, 1)};
  if (!aligned(a->workspace, 256)) return fail(MOE_FFN_ERR_ALIGNMENT, "%s: workspace is not 256-byte aligned", who);
  const Span outs[] = {span("out", a->out, R, N, a->ld_out, 2),
                       span("workspace", a->workspace, 1, (int64_t)a->workspace_bytes, 0, 1)};
  if ((rc = check_overlaps(who, outs, 2, ins, 4, -1, -1))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::Int4MatmulParams p = {};
  p.w = matrix(a->codes, a->scales, a->zeros, N, K, a->group);
  p.rows = a->rows;
  p.x = a->x;
  p.ld_x = a->ld_x;
  p.out = a->out;
  p.ld_out = a->ld_out;
  DeviceSide dev;
  if ((rc = device_side(who, &dev))) return rc;
  p.waits = moe::Waits{dev.status, dev.wait_ns, dev.inject};
  const bool f16 = a->type == MOE_FFN_F16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  moe::Int4Maps maps;
  if (const int tokens = moe::int4_tc_tokens(a->rows, a->n, a->k, a->group)) {
    const Int4Space space = int4_space(a, tokens);
    if (!a->workspace) return fail(MOE_FFN_ERR_NULL_PTR, "%s: workspace is NULL", who);
    if (a->workspace_bytes < (size_t)space.bytes)
      return fail(MOE_FFN_ERR_NO_MEMORY, "%s: workspace of %zu bytes, needs %lld", who, a->workspace_bytes, (long long)space.bytes);
    char *ws = static_cast<char *>(a->workspace);
    p.planes = reinterpret_cast<uint2 *>(ws);
    p.sums = reinterpret_cast<float *>(ws + space.sums);
    p.back = reinterpret_cast<float *>(ws + space.back);
    p.sum_groups = space.groups;
    if (!encode_map(&maps.w, a->codes, 1, K / 2, N, K / 2, 128, 64 * moe::code_halves(tokens, f16 ? 3 : 2, 128 / a->group)) ||
        !encode_map(&maps.x, ws, 1, K, space.rows, K, tokens * (f16 ? 3 : 2)))
      return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
    return launched(who, moe::launch_int4_tc(p, maps, tokens, f16, sms, st));
  }
  const moe::Int4Tiles t = moe::int4_pick_tiles(a->rows, a->n, a->k, sms);
  if (!encode_map(&maps.w, a->codes, 1, K / 2, N, K / 2, t.w_box(), 64) ||
      !encode_pieces(&maps.x, a->x, K / 32, R, a->ld_x, t.box_rows, t.x_box_pieces()))
    return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  return launched(who, moe::launch_int4_matmul(p, maps, t, f16, sms, st));
}

namespace {

int check_routed(const char *who, const moe_ffn_routed_args *a) {
  if (!a) return fail(MOE_FFN_ERR_NULL_PTR, "%s: args is NULL", who);
  if (a->rows == 0) return fail(MOE_FFN_ERR_ROWS_ZERO, "%s: rows must be at least 1", who);
  if (a->rows < 0 || a->rows > moe::kRoutedRows)
    return fail(MOE_FFN_ERR_ROWS_RANGE, "%s: rows must be at most %d", who, moe::kRoutedRows);
  if (a->bits != 4 && a->bits != 16) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: bits must be 4 or 16", who);
  const int step = a->bits == 4 ? 32 : 8;
  if (a->hidden < step || a->hidden % step || a->hidden > 65536 || a->inter < step || a->inter % step || a->inter > 65536)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: hidden and inter must be multiples of %d, at most 65536", who, step);
  if (a->experts < 1 || a->experts > moe::kRoutedExperts || a->top_k < 1 || a->top_k > moe::kRoutedTopK || a->top_k > a->experts ||
      a->shared < 0 || a->shared > moe::kRoutedShared)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: experts must be in 1..%d, top_k in 1..%d and at most experts, shared in 0..%d", who,
                moe::kRoutedExperts, moe::kRoutedTopK, moe::kRoutedShared);
  if (!type16(a->type) || (a->router_type != MOE_FFN_F32 && a->router_type != a->type))
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: type must be bf16 or f16, router_type f32 or type", who);
  if (a->score != MOE_FFN_SCORE_SIGMOID && a->score != MOE_FFN_SCORE_SOFTMAX)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown score", who);
  if (a->activation != MOE_FFN_ACT_SILU && a->activation != MOE_FFN_ACT_GELU)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: unknown activation", who);
  return a->bits == 4 ? check_group(who, a->group) : MOE_FFN_OK;
}

// experts with tokens, at most
int64_t routed_groups(const moe_ffn_routed_args *a) {
  return (a->rows * a->top_k < a->experts ? a->rows * a->top_k : a->experts) + a->shared;
}
// Offsets of the workspace's parts, each a multiple of 256, and sizes of 4-bit weights' parts.
struct RoutedSpace {
  int64_t h, x_planes, h_planes, x_sums, h_sums, back, h_max, masks, bytes;
  int tokens, planes, x_groups, h_groups;
  int x_halves, h_halves;  // of a tile
};
RoutedSpace routed_space(const moe_ffn_routed_args *a) {
  RoutedSpace s = {};
  int64_t at = 0;
  auto part = [&](int64_t bytes) {
    const int64_t from = at;
    at += (bytes + 255) / 256 * 256;
    return from;
  };
  const int64_t R = a->rows, I = a->inter, H = a->hidden, G = routed_groups(a);
  part(R * a->experts * 4);  // the logits
  s.h = part(a->bits == 4 ? G * R * I * 4 : G * ((R + 7) / 8 * 16) * I * 2);
  if (a->bits == 4) {
    s.tokens = moe::routed_code_tokens(a->rows);
    s.planes = a->type == MOE_FFN_F16 ? 3 : 2;
    s.x_halves = moe::code_halves(s.tokens, s.planes, 128 / a->group);
    s.h_halves = moe::code_halves(s.tokens, moe::kHiddenPlanes, 128 / a->group);
    auto groups = [&](int64_t k, int columns) { return (int)((k + columns - 1) / columns * (columns / a->group)); };
    s.x_groups = groups(H, 128 * s.x_halves);
    s.h_groups = groups(I, 128 * s.h_halves);
    s.x_planes = part(s.planes * s.tokens * H);
    s.h_planes = part(G * moe::kHiddenPlanes * s.tokens * I);
    s.x_sums = part((int64_t)s.x_groups * s.tokens * 4);
    s.h_sums = part(G * s.h_groups * s.tokens * 4);
    s.back = part(R * 4);
    s.h_max = part(R * 4);
    s.masks = part(G * 4);
  }
  s.bytes = at;
  return s;
}

}  // namespace

extern "C" int64_t moe_ffn_routed_workspace(const moe_ffn_routed_args *a) {
  const int rc = check_routed("routed_workspace", a);
  return rc ? rc : routed_space(a).bytes;
}

extern "C" int moe_ffn_routed_forward(const moe_ffn_routed_args *a, void *stream) {
  const char *who = "routed_forward";
  int rc = check_routed(who, a);
  if (rc) return rc;
  const int64_t R = a->rows, H = a->hidden, I = a->inter, E = a->experts, S = a->shared, K = a->top_k;
  if ((rc = check_rows16(who, "x", a->x, a->ld_x, H)) || (rc = check_rows2(who, "y", a->y, a->ld_y, H)) ||
      (rc = check_rows16(who, "workspace", a->workspace, 8, 8)))
    return rc;
  if (!a->router) return fail(MOE_FFN_ERR_NULL_PTR, "%s: router is NULL", who);
  const int rb = type_bytes(a->router_type);
  if (!aligned(a->router, 8 * rb) || !aligned(a->bias, 4) || !aligned(a->indices, 4) || !aligned(a->weights, 4))
    return fail(MOE_FFN_ERR_ALIGNMENT, "%s: router must be aligned to eight values, bias, indices and weights to one", who);
  const moe_ffn_matrices *all[] = {&a->gate, &a->up, &a->down, &a->shared_gate, &a->shared_up, &a->shared_down};
  const char *names[] = {"gate", "up", "down", "shared_gate", "shared_up", "shared_down"};
  Span ins[3 + 18];
  int n_ins = 0;
  ins[n_ins++] = span("x", a->x, R, H, a->ld_x, 2);
  ins[n_ins++] = span("router", a->router, E, H, H, rb);
  ins[n_ins++] = span("bias", a->bias, 1, E, E, 4);
  moe::FewMatrix m[6] = {};
  for (int i = 0; i < 6; ++i) {
    const int64_t count = i < 3 ? E : S, n = i % 3 == 2 ? H : I, k = i % 3 == 2 ? I : H;
    if (!count) {
      if (all[i]->w) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: %s is given without shared experts", who, names[i]);
      continue;
    }
    if (a->bits == 4) {
      if ((rc = check_int4(names[i], n, k, a->group, all[i]->w, all[i]->scales, all[i]->zeros))) return rc;
      const int64_t G = (k + a->group - 1) / a->group;
      m[i] = matrix(all[i]->w, all[i]->scales, all[i]->zeros, n, k, a->group);
      ins[n_ins++] = span(names[i], all[i]->w, count * n, k / 2, k / 2, 1);
      ins[n_ins++] = span(names[i], all[i]->scales, count * n, G, G, 2);
      ins[n_ins++] = span(names[i], all[i]->zeros, count * n, G, G, 1);
    } else {
      if ((rc = check_rows16(who, names[i], all[i]->w, k, k))) return rc;
      if (all[i]->scales || all[i]->zeros) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: %s in 16 bits has no scales", who, names[i]);
      m[i] = moe::FewMatrix{all[i]->w, nullptr, nullptr, (int)n, (int)k, 0, 0};
      ins[n_ins++] = span(names[i], all[i]->w, count * n, k, k, 2);
    }
  }
  for (int i = 1; i < (S ? 6 : 3); ++i)  // one kernel reads several matrices, with zero points or without
    if ((m[i].zeros != nullptr) != (m[0].zeros != nullptr))
      return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: %s and %s must both have zero points or neither", who, names[0], names[i]);
  const RoutedSpace space = routed_space(a);
  const int64_t need = space.bytes;
  if (a->workspace_bytes < (size_t)need)
    return fail(MOE_FFN_ERR_NO_MEMORY, "%s: workspace of %zu bytes, needs %lld", who, a->workspace_bytes, (long long)need);
  const Span outs[] = {span("y", a->y, R, H, a->ld_y, 2), span("indices", a->indices, R, K, K, 4),
                       span("weights", a->weights, R, K, K, 4), span("workspace", a->workspace, 1, need, 0, 1)};
  if ((rc = check_overlaps(who, outs, 4, ins, n_ins, -1, -1))) return rc;
  const int sms = current_sms();
  if (sms < 0) return sms;
  if ((rc = pending(who))) return rc;
  moe::RoutedParams p = {};
  p.rows = a->rows;
  p.hidden = a->hidden;
  p.inter = a->inter;
  p.experts = a->experts;
  p.top_k = a->top_k;
  p.shared = a->shared;
  p.softmax = a->score == MOE_FFN_SCORE_SOFTMAX;
  p.normalise = a->normalise != 0;
  p.act = a->activation;
  p.router_f32 = a->router_type == MOE_FFN_F32;
  p.scale = a->route_scale;
  p.x = a->x;
  p.ld_x = a->ld_x;
  p.router = a->router;
  p.bias = a->bias;
  p.gate = m[0];
  p.up = m[1];
  p.down = m[2];
  p.s_gate = m[3];
  p.s_up = m[4];
  p.s_down = m[5];
  p.y = a->y;
  p.ld_y = a->ld_y;
  p.indices = a->indices;
  p.weights = a->weights;
  char *ws = static_cast<char *>(a->workspace);
  p.logits = reinterpret_cast<float *>(ws);
  p.h = reinterpret_cast<uint16_t *>(ws + space.h);
  p.h32 = reinterpret_cast<float *>(ws + space.h);
  p.groups = (int)routed_groups(a);
  DeviceSide dev;
  if ((rc = device_side(who, &dev))) return rc;
  p.waits = moe::Waits{dev.status, dev.wait_ns, dev.inject};
  moe::RoutedMaps maps = {}, down = {};
  CUtensorMap *to[] = {&maps.gate, &maps.up, &down.gate, &maps.s_gate, &maps.s_up, &down.s_gate};
  bool ok = true;
  for (int i = 0; i < (S ? 6 : 3); ++i) {
    const int64_t count = i < 3 ? E : S, n = m[i].n, k = m[i].k;
    const int box = i % 3 == 2 ? 128 : 64, halves = i % 3 == 2 ? space.h_halves : space.x_halves;
    ok = ok && (a->bits == 4 ? encode_map(to[i], m[i].w, 1, k / 2, count * n, k / 2, box, 64 * halves)
                             : encode_map(to[i], m[i].w, 2, k, count * n, k, box));
  }
  const bool f16 = a->type == MOE_FFN_F16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->bits == 16) {
    const int64_t R8 = (R + 7) / 8 * 8;
    if (!ok || !encode_map(&maps.tokens, a->x, 2, H, R, a->ld_x, (int)R8) ||
        !encode_map(&down.tokens, p.h, 2, I, p.groups * 2 * R8, I, (int)(2 * R8)))
      return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
    return launched(who, moe::launch_routed(p, maps, down, f16, sms, st));
  }
  p.x_planes = reinterpret_cast<uint2 *>(ws + space.x_planes);
  p.h_planes = reinterpret_cast<uint2 *>(ws + space.h_planes);
  p.x_sums = reinterpret_cast<float *>(ws + space.x_sums);
  p.h_sums = reinterpret_cast<float *>(ws + space.h_sums);
  p.back = reinterpret_cast<float *>(ws + space.back);
  p.h_max = reinterpret_cast<uint32_t *>(ws + space.h_max);
  p.masks = reinterpret_cast<uint32_t *>(ws + space.masks);
  p.x_groups = space.x_groups;
  p.h_groups = space.h_groups;
  const int rows = space.planes * space.tokens, h_rows = moe::kHiddenPlanes * space.tokens;
  if (!ok || !encode_map(&maps.tokens, p.x_planes, 1, H, rows, H, rows) ||
      !encode_map(&down.tokens, p.h_planes, 1, I, (int64_t)p.groups * h_rows, I, h_rows))
    return fail(MOE_FFN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  return launched(who, moe::launch_routed_int4(p, maps, down, f16, sms, st));
}
