// A whole mixture-of-experts layer on a plain residual stream for a few tokens (sm_103a), in three kernels:
//
//   route   l = x Wr^T
//   up      each CTA chooses the experts from l; h = weight act(x Wg_e^T) (x Wu_e^T) for every token and expert
//   down    y = sum over the experts of h Wd_e^T
//
// Bound by the chosen experts' weights on their way from memory: each is read once, for all of its tokens.  Column j of
// the tensor cores' right operand is token j for every expert (zeros where it did not choose it), so the down kernel adds
// all experts' products in its accumulators: no partial results in memory, and one order of every sum.
//
// The choice costs each CTA less than a kernel of its own would cost the call, and needs no counter that a call would
// have to clear; it is a function of l alone, so every CTA of both kernels makes the same one.
#include "few.cuh"
#include "kernels.h"

namespace moe {
namespace {

// ---- router ----

constexpr int kRouteExperts = 2, kRouteTokens = 8;  // of a CTA, and of a turn

template <typename T, typename TR>
__global__ void __launch_bounds__(256) routed_logits_kernel(const __grid_constant__ RoutedParams p) {
  __shared__ float sums[8][kRouteExperts * kRouteTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = blockIdx.x * kRouteExperts;
  pdl_wait();
  pdl_trigger();
  for (int t0 = 0; t0 < p.rows; t0 += kRouteTokens) {
    float acc[kRouteExperts][kRouteTokens] = {};
    for (int k = warp * 256 + lane * 8; k < p.hidden; k += 8 * 256) {
      float w[kRouteExperts][8];
#pragma unroll
      for (int e = 0; e < kRouteExperts; ++e)
        load_eight<TR, true>(static_cast<const TR *>(p.router) + (long long)min(e0 + e, p.experts - 1) * p.hidden + k, 0, 1, 8, w[e]);
#pragma unroll
      for (int t = 0; t < kRouteTokens; ++t)
        if (t0 + t < p.rows) {
          float x[8];
          load_eight<T, true>(static_cast<const T *>(p.x) + (t0 + t) * p.ld_x + k, 0, 1, 8, x);
#pragma unroll
          for (int e = 0; e < kRouteExperts; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[e][t] = fmaf(w[e][i], x[i], acc[e][t]);
        }
    }
#pragma unroll
    for (int e = 0; e < kRouteExperts; ++e)
#pragma unroll
      for (int t = 0; t < kRouteTokens; ++t) {
        if (t0 + t >= p.rows) continue;
        const float s = warp_sum(acc[e][t]);
        if (lane == 0) sums[warp][e * kRouteTokens + t] = s;
      }
    __syncthreads();
    const int e = threadIdx.x / kRouteTokens, t = threadIdx.x % kRouteTokens;
    if (e < kRouteExperts && e0 + e < p.experts && t0 + t < p.rows) {
      float s = sums[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) s += sums[w][threadIdx.x];
      p.logits[(t0 + t) * p.experts + e0 + e] = s;
    }
    __syncthreads();
  }
}

// ---- choice ----

constexpr int kGroupsMax = kRoutedRows * kRoutedTopK + kRoutedShared;

struct Choice {
  int groups, routed;                              // experts with tokens, the shared ones last
  uint32_t mask[kRoutedExperts];                   // each expert's tokens
  uint32_t group_mask[kGroupsMax];
  uint16_t expert[kGroupsMax];
  uint16_t index[kRoutedRows][kRoutedTopK];
  float weight[kRoutedRows][kRoutedTopK];
};

// a number for each float that grows with it (the same for both zeros); NaN below all others, and 0 for none
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A warp for each token: lane l holds experts l, l + 32, ...  Every thread of the CTA.
__device__ __forceinline__ void choose(const RoutedParams &p, Choice &c, bool write) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  constexpr int kEach = kRoutedExperts / 32;
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) c.mask[e] = 0u;
  __syncthreads();
  for (int t = warp; t < p.rows; t += warps) {
    float l[kEach], top = -INFINITY, total = 0.f;
    uint32_t key[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      l[i] = 32 * i + lane < p.experts ? __ldcg(p.logits + t * p.experts + 32 * i + lane) : -INFINITY;
      top = fmaxf(top, l[i]);
    }
    if (p.softmax) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (32 * i < p.experts) total += expf(l[i] - top);
      total = warp_sum(total);
    }
    // without a bias the scores' order is the logits'
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      key[i] = 0u;
      const int e = 32 * i + lane;
      if (e < p.experts) {
        float v = l[i];
        if (p.bias) v = (p.softmax ? expf(v - top) / total : sigmoidf_(v)) + p.bias[e];
        key[i] = rank_of(v);
      }
    }
    float mine = 0.f;  // lane s: the s-th choice's logit
    int which = 0;
    for (int s = 0; s < p.top_k; ++s) {
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      const uint32_t most = __reduce_max_sync(0xffffffffu, best);
      const int e = (int)__reduce_min_sync(0xffffffffu, best == most ? (uint32_t)(32 * at + lane) : 0xFFFFFFFFu);
      float logit = 0.f;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (32 * i + lane == e) {
          key[i] = 0u;
          logit = l[i];
        }
      logit = __shfl_sync(0xffffffffu, logit, e & 31);
      if (lane == s) {
        mine = logit;
        which = e;
      }
    }
    // The chosen scores over their sum.  Both are scaled by exp(-m), m the largest of min(l, 0) (or of l): far out
    // every score may be 0 in f32 where their ratios are not.
    const bool in = lane < p.top_k;
    float w;
    if (p.normalise) {
      float m = in ? (p.softmax ? mine : fminf(mine, 0.f)) : -INFINITY;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      w = !in ? 0.f : p.softmax ? expf(mine - m) : expf(fminf(mine, 0.f) - m) / (1.f + expf(-fabsf(mine)));
      float sum = w;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w /= sum;
    } else {
      w = p.softmax ? expf(mine - top) / total : sigmoidf_(mine);
    }
    w *= p.scale;
    if (in) {
      c.index[t][lane] = (uint16_t)which;
      c.weight[t][lane] = w;
      atomicOr(&c.mask[which], 1u << t);
      if (write) {
        if (p.indices) p.indices[t * p.top_k + lane] = which;
        if (p.weights) p.weights[t * p.top_k + lane] = w;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const uint32_t mask = e0 + lane < p.experts ? c.mask[e0 + lane] : 0u;
      const uint32_t has = __ballot_sync(0xffffffffu, mask != 0u);
      if (mask) {
        const int at = n + __popc(has & ((1u << lane) - 1u));
        c.expert[at] = (uint16_t)(e0 + lane);
        c.group_mask[at] = mask;
      }
      n += __popc(has);
    }
    if (lane < p.shared) {
      c.expert[n + lane] = (uint16_t)lane;
      c.group_mask[n + lane] = 0xFFFFFFFFu >> (32 - p.rows);
    }
    if (lane == 0) {
      c.routed = n;
      c.groups = n + p.shared;
    }
  }
  __syncthreads();
}

// the place of a group among a token's, which has chosen it: that of its row of h
__device__ __forceinline__ int slot_of(const RoutedParams &p, const Choice &c, int group, int token) {
  const int e = c.expert[group];
  if (group >= c.routed) return p.top_k + e;
  int slot = 0;
  for (int s = 1; s < p.top_k; ++s)
    if (c.index[token][s] == e) slot = s;
  return slot;
}

// ---- gate and up ----

template <typename T, int BITS, int NT>
struct UpJob {
  const RoutedParams &p;
  const Choice &c;
  int units, tiles, strips;  // a unit: 16 rows of a group's gate and up matrices
  __device__ __forceinline__ void copies_begun() const {}
  __device__ __forceinline__ void copy(uint32_t place, int unit, int, int tile) const {
    const int group = unit / strips, r = (unit - group * strips) * 16, e = c.expert[group];
    const bool shared = group >= c.routed;
    const FewMatrix &g = shared ? p.s_gate : p.gate, &u = shared ? p.s_up : p.up;
    copy_strip<BITS>(place, g, e, r, tile);
    copy_strip<BITS>(place + kStripBytes, u, e, r, tile);
    if constexpr (BITS == 4) {
      const int lane = threadIdx.x & 31;
      copy_meta(place + 2 * kStripBytes + (lane >> 4) * 16 * kMetaPitch, lane < 16 ? g : u, e, r, tile, lane & 15);
    }
  }
  __device__ __forceinline__ void multiply(uint32_t place, int unit, int, int tile, float (&acc)[2][NT][4]) const {
    const int group = unit / strips, r = (unit - group * strips) * 16, e = c.expert[group], lane = threadIdx.x & 31;
    const uint32_t mask = c.group_mask[group];
    Tokens<NT> x;
    unsigned some = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int token = 8 * i + (lane >> 2);
      x.row[i] = mask >> token & 1 ? static_cast<const char *>(p.x) + token * p.ld_x * 2 : nullptr;
      some |= (mask >> (8 * i) & 255u ? 1u : 0u) << i;
    }
    const FewMatrix m[2] = {p.gate, p.up};  // (the shared experts' are of the same shape)
    const int es[2] = {e, e}, rs[2] = {r, r};
    multiply_tile<T, BITS, 2, NT>(place, m, es, rs, tile, x, some, acc);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int, int thread, int threads, Sum sum) const {
    const int group = unit / strips, r = (unit - group * strips) * 16;
    const uint32_t mask = c.group_mask[group];
    for (int i = thread; i < 16 * p.rows; i += threads) {
      const int row = i & 15, token = i >> 4;
      if (!(mask >> token & 1) || r + row >= p.inter) continue;
      const int slot = slot_of(p, c, group, token);
      const float w = group < c.routed ? c.weight[token][slot] : 1.f;
      // rounded to 16 bits as the tensor cores' operand, as the gated block does
      const T h = from_f32<T>(act_value(p.act, sum(0, row, token)) * sum(1, row, token) * w);
      p.h[((long long)token * (p.top_k + p.shared) + slot) * p.inter + r + row] = *reinterpret_cast<const uint16_t *>(&h);
    }
  }
};

// ---- down ----

template <typename T, int BITS, int NT>
struct DownJob {
  const RoutedParams &p;
  const Choice &c;
  int units, tiles, per;  // a unit: 16 rows of every group's matrix; per: tiles of a group
  __device__ __forceinline__ void copies_begun() const { pdl_wait(); }  // h comes from the kernel before
  __device__ __forceinline__ void copy(uint32_t place, int unit, int, int tile) const {
    const int group = tile / per, e = c.expert[group];
    const FewMatrix &d = group >= c.routed ? p.s_down : p.down;
    copy_strip<BITS>(place, d, e, unit * 16, tile - group * per);
    if constexpr (BITS == 4) {
      const int lane = threadIdx.x & 31;
      if (lane < 16) copy_meta(place + kStripBytes, d, e, unit * 16, tile - group * per, lane);
    }
  }
  __device__ __forceinline__ void multiply(uint32_t place, int unit, int, int tile, float (&acc)[1][NT][4]) const {
    const int group = tile / per, lane = threadIdx.x & 31;
    const uint32_t mask = c.group_mask[group];
    Tokens<NT> x;
    unsigned some = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int token = 8 * i + (lane >> 2);
      x.row[i] = nullptr;
      if (mask >> token & 1)
        x.row[i] = reinterpret_cast<const char *>(
            p.h + ((long long)token * (p.top_k + p.shared) + slot_of(p, c, group, token)) * p.inter);
      some |= (mask >> (8 * i) & 255u ? 1u : 0u) << i;
    }
    const FewMatrix m[1] = {p.down};
    const int es[1] = {c.expert[group]}, rs[1] = {unit * 16};
    multiply_tile<T, BITS, 1, NT>(place, m, es, rs, tile - group * per, x, some, acc);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int, int thread, int threads, Sum sum) const {
    for (int i = thread; i < 16 * p.rows; i += threads) {
      const int row = i & 15, token = i >> 4;
      if (unit * 16 + row < p.hidden) static_cast<T *>(p.y)[token * p.ld_y + unit * 16 + row] = from_f32<T>(sum(0, row, token));
    }
  }
};

template <bool UP, int BITS, int NT>
constexpr int kRoutedStages = !UP ? 4 : BITS == 16 && NT == 1 ? 3 : 2;

template <bool UP, typename T, int BITS, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 2) routed_kernel(const __grid_constant__ RoutedParams p) {
  constexpr int M = UP ? 2 : 1, kStages = kRoutedStages<UP, BITS, NT>, kPlace = kPlaceBytes<BITS, M>;
  extern __shared__ __align__(128) char smem[];
  __shared__ Choice c;
  float *parts = reinterpret_cast<float *>(smem + kFewWarps * kStages * kPlace);
  if constexpr (UP) {
    pdl_wait();
    // The down kernel's CTAs may come, choose and fetch weights: not earlier, as they read the logits.
    pdl_trigger();
    choose(p, c, blockIdx.x == 0);
    const int strips = (p.inter + 15) / 16;
    UpJob<T, BITS, NT> job{p, c, c.groups * strips, (p.hidden + kTileK<BITS> - 1) / kTileK<BITS>, strips};
    stream_units<M, NT, kStages, kPlace>(job, smem_u32(smem), parts, 3);
  } else {
    choose(p, c, false);
    const int per = (p.inter + kTileK<BITS> - 1) / kTileK<BITS>;
    DownJob<T, BITS, NT> job{p, c, (p.hidden + 15) / 16, c.groups * per, per};
    stream_units<M, NT, kStages, kPlace>(job, smem_u32(smem), parts, 3);
  }
}

template <bool UP, typename T, int BITS, int NT>
cudaError_t part_launch(const RoutedParams &p, int num_sms, cudaStream_t st) {
  constexpr int M = UP ? 2 : 1;
  constexpr size_t smem = kFewWarps * (kRoutedStages<UP, BITS, NT> * kPlaceBytes<BITS, M> + M * NT * kPartFloats * sizeof(float));
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem((const void *)routed_kernel<UP, T, BITS, NT>, smem, done);
  if (e != cudaSuccess) return e;
  const long long groups = (long long)(p.rows * p.top_k < p.experts ? p.rows * p.top_k : p.experts) + p.shared;
  const long long units = UP ? groups * ((p.inter + 15) / 16) : (p.hidden + 15) / 16, most = 2ll * num_sms;
  return launch_pdl(routed_kernel<UP, T, BITS, NT>, dim3((unsigned)(units < most ? units : most)), dim3(32 * kFewWarps), smem, st, p);
}

template <typename T, int BITS, int NT>
cudaError_t layer_launch(const RoutedParams &p, int num_sms, cudaStream_t st) {
  const dim3 grid((p.experts + kRouteExperts - 1) / kRouteExperts);
  cudaError_t e = launch_pdl(p.router_f32 ? routed_logits_kernel<T, float> : routed_logits_kernel<T, T>, grid, dim3(256), 0, st, p);
  if (e == cudaSuccess) e = part_launch<true, T, BITS, NT>(p, num_sms, st);
  if (e == cudaSuccess) e = part_launch<false, T, BITS, NT>(p, num_sms, st);
  return e;
}

template <typename T, int BITS>
cudaError_t routed_rows(const RoutedParams &p, int num_sms, cudaStream_t st) {
  if (p.rows <= 8) return layer_launch<T, BITS, 1>(p, num_sms, st);
  if (p.rows <= 16) return layer_launch<T, BITS, 2>(p, num_sms, st);
  return layer_launch<T, BITS, 4>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_routed(const RoutedParams &p, bool f16, bool bits4, int num_sms, cudaStream_t st) {
  if (f16) return bits4 ? routed_rows<__half, 4>(p, num_sms, st) : routed_rows<__half, 16>(p, num_sms, st);
  return bits4 ? routed_rows<__nv_bfloat16, 4>(p, num_sms, st) : routed_rows<__nv_bfloat16, 16>(p, num_sms, st);
}

}  // namespace moe
