// The routed layer with 4-bit weights on the FP8 tensor cores (sm_103a; few_tc.cuh), in four kernels:
//
//   route   l = x Wr^T, and x as planes
//   up      each CTA chooses the experts from l; h = weight act(x Wg_e^T) (x Wu_e^T), in f32
//   split   h as planes: three, in either type
//   down    y = sum over the experts of h Wd_e^T
//
// Bound by the chosen experts' codes on their way from memory and through registers into operands: each is read once, for
// all tokens, which are the right operand's columns for every expert.  So the down kernel, whose operand is zero where a
// token has not chosen an expert, adds all experts' products in its registers, in one order.
// 16 tokens through 256 experts of 4096 x 2048 and a shared one, six each, in groups of 128: 221 us, 4.8 TB/s (157 at the
// copy's rate; on mma.sync, each expert's tokens eight at a time, 577); one token 41 us (13.7), of which the four kernels'
// latencies are the most: gate and up have 224 strips for 152 SMs.  32 tokens 500 us (263).
//
// A token's h has one power of two for all of its experts, from the largest magnitude among them (an atomic maximum: of
// any order the same), so that their products can be added as they are: what is lost of an expert's h is at most 2^-14 of it
// or 2^-27 of the token's largest, and the sum that it goes to holds that one.  It has three planes in bf16 too: h rounded
// to 16 bits, in two planes, left the layer off by 0.0024 in 2-norm where y's rounding leaves 0.0017 (16 tokens 230 us for
// 231, 32 tokens in groups of 32 1210 for 1440).
#include "few_tc.cuh"
#include "kernels.h"
#include "routed.cuh"

namespace moe {
namespace {

// CTAs from route_ctas on: a row of x each, those of the tokens that the others have
template <typename T, typename TR, int PLANES>
__global__ void __launch_bounds__(256) routed_planes_kernel(const __grid_constant__ RoutedParams p, int tokens) {
  const int n = route_ctas(p), row = blockIdx.y * kRouteTokens + blockIdx.x - n, k8 = p.hidden / 8;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x < n) {
    route_logits<T, TR>(p, blockIdx.x * kRouteExperts, blockIdx.y * kRouteTokens);
    return;
  }
  if (row >= p.rows) return;
  const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
  const uint32_t most = row_max(x, k8);
  if (threadIdx.x == 0) {
    p.back[row] = way_back(most);
    p.h_max[row] = 0u;
  }
  split_row<T, PLANES>(x, two_to(plane_exponent(most)), k8, p.x_groups, 1 << (p.gate.group_shift - 3), p.x_planes + (size_t)row * k8,
                       (size_t)tokens * k8, p.x_sums + row, tokens);
}

// a CTA for each row of h: a token of an expert; zeros where it has not chosen it
__global__ void __launch_bounds__(256) routed_split_kernel(const __grid_constant__ RoutedParams p, int tokens) {
  const int token = blockIdx.x, group = blockIdx.y, k8 = p.inter / 8;
  pdl_wait();
  // The down kernel's CTAs may come, choose and fetch weights.
  pdl_trigger();
  const uint32_t mask = p.masks[group];
  if (!mask) return;  // no such group
  const float *h = p.h32 + ((size_t)group * p.rows + token) * p.inter;
  split_row<float, kHiddenPlanes>(mask >> token & 1 ? h : nullptr, two_to(plane_exponent(__ldcg(p.h_max + token))), k8, p.h_groups,
                                  1 << (p.gate.group_shift - 3), p.h_planes + ((size_t)group * kHiddenPlanes * tokens + token) * k8,
                                  (size_t)tokens * k8, p.h_sums + (size_t)group * p.h_groups * tokens + token, tokens);
}

// Up: a unit is 64 rows of a group's gate and 64 of its up matrix.  Down: one unit, 128 rows of all groups' matrices, whose
// tiles the CTAs of a cluster share.
template <bool UP, typename T, int TOKENS, int PLANES, int GROUPS>
struct LayerJob {
  using C = CodeCfg<TOKENS, PLANES, GROUPS>;
  const RoutedParams &p;
  const RoutedMaps &maps;
  const Choice &c;
  float *sums;                    // up: [2][TOKENS][64]; down: [TOKENS][128]
  int tiles, strips;              // of a group; up: units of a group
  int row_tile, first, end;       // down
  float back;                     // up: what this lane's token's products are multiplied by, after 512 (2^119 at most: together
                                  // they may leave f32)
  struct Place {
    int unit, group, tile, left;  // left: tiles; up: units
    __device__ __forceinline__ bool more() const { return left > 0; }
  };
  __device__ __forceinline__ void next(Place &a) const {
    if (!UP) --a.left;
    if (++a.tile < tiles) return;
    a.tile = 0;
    if (UP) {
      a.left -= gridDim.x;
      a.unit += gridDim.x;
      a.group = a.unit / strips;
    } else {
      ++a.group;
    }
  }
  __device__ __forceinline__ int count() const {
    const int units = c.groups * strips, at = blockIdx.x, step = gridDim.x;
    return !UP ? end - first : at < units ? tiles * ((units - at + step - 1) / step) : 0;
  }
  __device__ __forceinline__ Place begin() const {
    if (UP) return Place{(int)blockIdx.x, (int)blockIdx.x / strips, 0, c.groups * strips - (int)blockIdx.x};
    return Place{0, first / tiles, first % tiles, end - first};
  }
  __device__ __forceinline__ void next_unit(Place &a) const {
    if (UP) {
      a.left -= gridDim.x;
      a.unit += gridDim.x;
      a.group = a.unit / strips;
    } else {
      a.left = 0;
    }
  }
  __device__ __forceinline__ int unit_tiles() const { return UP ? tiles : end - first; }
  __device__ __forceinline__ bool skip(Place &a, int by) const {
    a.tile += by;
    if (UP) return a.tile < tiles;
    a.left -= by;
    while (a.tile >= tiles) {
      a.tile -= tiles;
      ++a.group;
    }
    return a.left > 0;
  }
  // the group's matrix among its kind's
  __device__ __forceinline__ int matrix_of(const Place &a, bool &shared) const {
    const int e = c.group_expert[a.group];
    shared = e >= p.experts;
    return shared ? e - p.experts : e;
  }
  __device__ __forceinline__ void weights(const Place &a, uint32_t at, uint32_t bar) const {
    bool shared;
    const int e = matrix_of(a, shared), x = a.tile * (64 * C::kHalves);
    if constexpr (UP) {
      const int r = e * p.inter + (a.unit - a.group * strips) * 64;
      tma_load_2d_one<false>(at, shared ? &maps.s_gate : &maps.gate, bar, x, r);
      tma_load_2d_one<false>(at + C::kW / 2, shared ? &maps.s_up : &maps.up, bar, x, r);
    } else {
      tma_load_2d_one<false>(at, shared ? &maps.s_gate : &maps.gate, bar, x, e * p.hidden + row_tile * kCodeRows);
    }
  }
  __device__ __forceinline__ void ready() const {
    if constexpr (!UP) pdl_wait();
  }
  __device__ __forceinline__ void tokens(const Place &a, uint32_t at, uint32_t to, uint32_t bar) const {
#pragma unroll
    for (int h = 0; h < C::kHalves; ++h)
      tma_load_2d_one<false>(at + h * C::kB, &maps.tokens, bar, (a.tile * C::kHalves + h) * 128, UP ? 0 : a.group * C::kRows);
    const float *from = UP ? p.x_sums : p.h_sums + (size_t)a.group * p.h_groups * TOKENS;
    tma_bulk_one(to, from + a.tile * (C::kAll * TOKENS), C::kSums, bar);
  }
  struct Lines {
    const uint16_t *scales;
    const uint8_t *zeros;
  };
  struct Row {
    Lines now, next;
    int row, group;
  };
  // row r of a group's matrices; up: 64 rows of gate, then 64 of up
  __device__ __forceinline__ Lines find(int r, int group, int strip) const {
    const int e0 = c.group_expert[group];
    const bool shared = e0 >= p.experts, up = UP && r >= 64;
    const FewMatrix &m = UP ? (shared ? (up ? p.s_up : p.s_gate) : up ? p.up : p.gate) : shared ? p.s_down : p.down;
    const int row = UP ? min(strip * 64 + r % 64, p.inter - 1) : min(row_tile * kCodeRows + r, p.hidden - 1);
    const long long at = ((long long)(shared ? e0 - p.experts : e0) * (UP ? p.inter : p.hidden) + row) * groups();
    return Lines{m.scales + at, m.zeros ? m.zeros + at : nullptr};
  }
  __device__ __forceinline__ int groups() const { return UP ? p.gate.groups : p.down.groups; }
  // what comes after a unit (up) or a group (down)
  __device__ __forceinline__ void look_ahead(Row &r, int next) const {
    const int group = UP ? next / strips : next;
    if (group >= c.groups) return;
    r.next = find(r.row, group, UP ? next - group * strips : 0);
    fetch_lines(r.next.scales, 2 * groups());
    if (r.next.zeros) fetch_lines(r.next.zeros, groups());
  }
  __device__ __forceinline__ void row_at(Row &r, const Place &a, int row) const {
    r.row = row;
    r.group = a.group;
    r.now = find(row, a.group, UP ? a.unit - a.group * strips : 0);
    look_ahead(r, UP ? a.unit + gridDim.x : a.group + 1);
  }
  __device__ __forceinline__ void next_row(Row &r, const Place &a) const {
    r.now = r.next;
    look_ahead(r, a.unit + 2 * gridDim.x);
  }
  struct Scales {
    uint16_t scales[C::kAll];
    uint8_t zeros[C::kAll];
    __device__ __forceinline__ float scale(int g) const { return to_f32(reinterpret_cast<const T *>(scales)[g]); }
    __device__ __forceinline__ float zero(int g) const { return (float)(zeros[g] & 15u); }
  };
  __device__ __forceinline__ int last(const Place &a) const { return UP || a.left > tiles - a.tile ? tiles : a.tile + a.left; }
  __device__ __forceinline__ void scales(Row &r, const Place &a, int ahead, Scales &s) const {
    if (!UP && r.group != a.group) {
      r.now = a.group == r.group + 1 ? r.next : find(r.row, a.group, 0);
      r.group = a.group;
      look_ahead(r, a.group + 1);
    }
#pragma unroll
    for (int g = 0; g < C::kAll; ++g) {
      const int i = min((a.tile + ahead) * C::kAll + g, groups() - 1);
      s.scales[g] = r.now.scales[i];
      s.zeros[g] = 8u;
      if (r.now.zeros) s.zeros[g] = r.now.zeros[i];
    }
  }
  __device__ __forceinline__ void finish(const Place &a, int row, int turn, int barrier, int t0, const float (&acc)[C::kMine]) const {
    if constexpr (UP) {
      float *u = sums + turn * (TOKENS * 64) + t0 * 64;
      if (row >= 64)
#pragma unroll
        for (int t = 0; t < C::kMine; ++t)
          if (t0 + t < p.rows) u[t * 64 + row - 64] = acc[t];
      asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");
      if (row >= 64) return;
      const int at = (a.unit - a.group * strips) * 64 + row, e = c.group_expert[a.group];
      const uint32_t mask = c.group_mask[a.group] >> t0;
      float *h = p.h32 + ((size_t)a.group * p.rows + t0) * p.inter + at;
      const float weight = weight_of(p, c, e, threadIdx.x & 31);  // this lane's token's
#pragma unroll
      for (int t = 0; t < C::kMine; ++t) {
        if (t0 + t >= p.rows) break;
        if (!(mask >> t & 1)) continue;
        const float by = __shfl_sync(0xffffffffu, back, t0 + t), w = __shfl_sync(0xffffffffu, weight, t0 + t);
        uint32_t size = 0u;
        if (at < p.inter) {
          const float out = act_value(p.act, acc[t] * 512.f * by) * (u[t * 64 + row] * 512.f * by) * w;
          h[(size_t)t * p.inter] = out;
          size = __float_as_uint(out) & 0x7FFFFFFFu;
        }
        size = __reduce_max_sync(0xffffffffu, size);
        if (row % 32 == 0) atomicMax(p.h_max + t0 + t, size);
      }
    } else {
#pragma unroll
      for (int t = 0; t < C::kMine; ++t)
        if (t0 + t < p.rows) sums[(t0 + t) * kCodeRows + row] = acc[t];
    }
  }
};

// A result from the token's own experts alone, by a warp: see the down kernel's end.
template <typename T>
__device__ __noinline__ float own_experts(const RoutedParams &p, const Choice &c, int token, int n) {
  float sum = 0.f;
  for (int g = 0; g < c.groups; ++g) {
    if (!(c.group_mask[g] >> token & 1)) continue;
    const int e = c.group_expert[g];
    const FewMatrix &m = e >= p.experts ? p.s_down : p.down;
    const long long row = (long long)(e >= p.experts ? e - p.experts : e) * p.hidden + n;
    const uint32_t *codes = static_cast<const uint32_t *>(m.w) + row * (p.inter / 8);
    const T *scales = reinterpret_cast<const T *>(m.scales) + row * m.groups;
    const float4 *h = reinterpret_cast<const float4 *>(p.h32 + ((size_t)g * p.rows + token) * p.inter);
    for (int i = threadIdx.x % 32; i < p.inter / 8; i += 32) {
      const int group = 8 * i >> m.group_shift;
      const float zero = m.zeros ? (float)(m.zeros[row * m.groups + group] & 15u) : 8.f;
      const uint32_t w = codes[i];
      const float4 lo = __ldcg(h + 2 * i), hi = __ldcg(h + 2 * i + 1);
      const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      float part = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) part = fmaf((float)(w >> (4 * k) & 15u) - zero, v[k], part);
      sum = fmaf(part, to_f32(scales[group]), sum);
    }
    if (__any_sync(0xffffffffu, sum != sum)) break;  // its own
  }
  return warp_sum(sum);
}

template <bool UP, typename T, int TOKENS, int PLANES, int GROUPS>
__global__ void __launch_bounds__(CodeCfg<TOKENS, PLANES, GROUPS>::kThreads, 1)
    routed_codes_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedMaps maps, int splits) {
  using C = CodeCfg<TOKENS, PLANES, GROUPS>;
  extern __shared__ char smem[];
  __shared__ __align__(8) CodeBars<C> bars;
  __shared__ Choice c;
  __shared__ float sums[TOKENS * kCodeRows];
  char *ring = smem + (-smem_u32(smem) & 1023u);
  code_setup<C>(bars);
  if constexpr (UP) {
    pdl_wait();
    pdl_trigger();
  }
  choose_groups(p, c, reinterpret_cast<uint32_t *>(ring), UP && blockIdx.x == 0);  // (the ring is not in use yet)
  const int tiles = ((UP ? p.hidden : p.inter) + 128 * C::kHalves - 1) / (128 * C::kHalves), strips = (p.inter + 63) / 64;
  const int rank = UP ? 0 : blockIdx.x % splits, row_tile = UP ? 0 : blockIdx.x / splits;
  const long long all = (long long)c.groups * tiles;
  if (UP && blockIdx.x == 0)
    for (int g = threadIdx.x; g < p.groups; g += C::kThreads) p.masks[g] = g < c.groups ? c.group_mask[g] : 0u;
  const LayerJob<UP, T, TOKENS, PLANES, GROUPS> job{p, maps, c, sums, tiles, strips, row_tile, (int)(all * rank / splits),
                                                    (int)(all * (rank + 1) / splits),
                                                    UP && threadIdx.x % 32 < p.rows ? __ldcg(p.back + threadIdx.x % 32) : 0.f};
  if (!UP && job.first == job.end)
    for (int i = threadIdx.x; i < TOKENS * kCodeRows; i += C::kThreads) sums[i] = 0.f;
  code_pipeline<C, TOKENS, PLANES, GROUPS>(job, ring, bars, p.waits);
  if constexpr (!UP) {  // the CTAs' sums in the order of their ranks, a part of the rows by each
    if (splits > 1) cluster_sync();
    // A scale that is not finite is NaN as 0 times it for the tokens that have not chosen its expert: such results are formed
    // again.  (Without one this is a comparison for each result; a token that is not finite itself is NaN throughout.)
    const int part = kCodeRows / splits, row0 = rank * part, count = part * p.rows;
    for (int i0 = 0; i0 < count; i0 += C::kThreads) {
      const int i = i0 + threadIdx.x, row = row0 + i % part, t = i / part, n = row_tile * kCodeRows + row;
      const bool in = i < count && n < p.hidden;
      float v = 0.f, back = 0.f, x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)  // all loads before the first sum
        if (in && r < splits)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[r]) : "r"(in_cta(&sums[t * kCodeRows + row], r)) : "memory");
      if (in) back = way_back(__ldcg(p.h_max + t));
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (in && r < splits) v += x[r];
      const bool bad = v != v && back == back;
      v = v * 512.f * back;
      for (unsigned again = __ballot_sync(0xffffffffu, bad); again; again &= again - 1) {
        const int from = __ffs(again) - 1;
        const float own = own_experts<T>(p, c, __shfl_sync(0xffffffffu, t, from), __shfl_sync(0xffffffffu, n, from));
        if (threadIdx.x % 32 == from) v = own;
      }
      if (in) static_cast<T *>(p.y)[t * p.ld_y + n] = from_f32<T>(v);
    }
    if (splits > 1) cluster_sync();
  }
  code_end(bars);
}

template <typename T, int TOKENS, int GROUPS>
cudaError_t codes_launch(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  constexpr int PLANES = std::is_same<T, __half>::value ? 3 : 2;
  using C = CodeCfg<TOKENS, PLANES, GROUPS>;
  using D = CodeCfg<TOKENS, kHiddenPlanes, GROUPS>;  // of the down kernel
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = allow_smem((const void *)routed_codes_kernel<true, T, TOKENS, PLANES, GROUPS>, C::kRing + 1024, done[0]);
  if (e == cudaSuccess)
    e = launch_pdl(p.router_f32 ? routed_planes_kernel<T, float, PLANES> : routed_planes_kernel<T, T, PLANES>, dim3(route_ctas(p) + kRouteTokens, route_turns(p)),
                   dim3(256), 0, st, p, TOKENS);
  const long long units = (long long)p.groups * ((p.inter + 63) / 64);
  if (e == cudaSuccess)
    e = launch_pdl(routed_codes_kernel<true, T, TOKENS, PLANES, GROUPS>, dim3((unsigned)(units < num_sms ? units : num_sms)),
                   dim3(C::kThreads), C::kRing + 1024, st, p, maps, 1);
  if (e == cudaSuccess) e = launch_pdl(routed_split_kernel, dim3(p.rows, p.groups), dim3(256), 0, st, p, TOKENS);
  if (e != cudaSuccess) return e;
  const int tiles = (p.hidden + kCodeRows - 1) / kCodeRows, splits = code_splits(tiles, num_sms);
  return launch_code_clusters(routed_codes_kernel<false, T, TOKENS, kHiddenPlanes, GROUPS>, D::kRing + 1024, done[1], dim3(tiles * splits),
                              D::kThreads, splits, st, p, down, splits);
}

template <typename T, int GROUPS>
cudaError_t codes_tokens(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  const int tokens = routed_code_tokens(p.rows);
  if (tokens == 8) return codes_launch<T, 8, GROUPS>(p, maps, down, num_sms, st);
  if (tokens == 16) return codes_launch<T, 16, GROUPS>(p, maps, down, num_sms, st);
  return codes_launch<T, 32, GROUPS>(p, maps, down, num_sms, st);
}
template <typename T>
cudaError_t codes_typed(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  const int shift = p.gate.group_shift;
  if (shift == 7) return codes_tokens<T, 1>(p, maps, down, num_sms, st);
  if (shift == 6) return codes_tokens<T, 2>(p, maps, down, num_sms, st);
  return codes_tokens<T, 4>(p, maps, down, num_sms, st);
}

}  // namespace

cudaError_t launch_routed_int4(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, bool f16, int num_sms,
                               cudaStream_t st) {
  return f16 ? codes_typed<__half>(p, maps, down, num_sms, st) : codes_typed<__nv_bfloat16>(p, maps, down, num_sms, st);
}

}  // namespace moe
