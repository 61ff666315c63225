// The routed layer's first part, which its kernels share: the router's logits, and each token's choice of experts.
//
// The choice costs each CTA less than a kernel of its own would cost the call, and needs no counter that a call would
// have to clear; it is a function of the logits alone, so every CTA of every kernel makes the same one.
#pragma once
#include "common.cuh"
#include "dense_vec.cuh"
#include "few.h"

namespace moe {

// ---- router ----

// of a CTA
constexpr int kRouteExperts = 2, kRouteTokens = 4;
__host__ __device__ inline int route_ctas(const RoutedParams &p) { return (p.experts + kRouteExperts - 1) / kRouteExperts; }
inline int route_turns(const RoutedParams &p) { return (p.rows + kRouteTokens - 1) / kRouteTokens; }

// by a CTA of 256: experts from e0 on, tokens from t0 on
template <typename T, typename TR>
__device__ __forceinline__ void route_logits(const RoutedParams &p, int e0, int t0) {
  __shared__ float sums[8][kRouteExperts * kRouteTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float acc[kRouteExperts][kRouteTokens] = {};
#pragma unroll 2
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
}

// ---- choice ----

constexpr int kGroupsMax = kRoutedRows * kRoutedTopK + kRoutedShared;

// Shared experts have the numbers from `experts` on, and come last.
struct Choice {
  int groups;                                      // experts with tokens, each once
  int count[(kRoutedExperts + kRoutedShared + 31) / 32];
  uint16_t group_expert[kGroupsMax];
  uint32_t group_mask[kGroupsMax];
  uint32_t mask[kRoutedExperts];                   // each expert's tokens
  __align__(16) uint16_t index[kRoutedRows][kRoutedTopK];
  float weight[kRoutedRows][kRoutedTopK];
};

// a number for each float that grows with it (the same for both zeros); NaN below all others, and 0 for none
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A warp for each token.  Every thread of the CTA; ends with a barrier.  keys: 1024 words of shared memory for each warp,
// whose use by TMA afterwards needs a proxy fence by every thread and a barrier (choose_groups).
// The loops are kept short: a kernel runs this code once, and its way into the instruction caches took most of its time
// while the experts were held in registers (16 of them a lane, each loop unrolled: 8.7 us of one token of 256 experts).
// But the loads have one of their own, with all of them on their way (one token of 256 experts in 16 bits: 69.9 -> 65.5 us).
__device__ __forceinline__ void choose_tokens(const RoutedParams &p, Choice &c, uint32_t *keys, bool write) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float *raw = reinterpret_cast<float *>(keys + warp * (2 * kRoutedExperts));  // a lane's own experts', before the choice
  uint32_t *key = keys + warp * (2 * kRoutedExperts) + kRoutedExperts;
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) c.mask[e] = 0u;
  __syncthreads();
#pragma unroll 1
  for (int t = warp; t < p.rows; t += warps) {
    const float *logits = p.logits + t * p.experts;
    // all of them on their way at once: in the loops below each would wait for its own
#pragma unroll 8
    for (int e = lane; e < p.experts; e += 32) {
      raw[e] = __ldcg(logits + e);
      if (p.bias) key[e] = __float_as_uint(p.bias[e]);
    }
    float top = -INFINITY, total = 0.f;
    if (p.softmax && (p.bias || !p.normalise)) {  // a score itself is wanted, not ratios or the order alone
      for (int e = lane; e < p.experts; e += 32) top = fmaxf(top, raw[e]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
      for (int e = lane; e < p.experts; e += 32) total += expf(raw[e] - top);
      total = warp_sum(total);
    }
    if (p.bias) {
#pragma unroll 1
      for (int e = lane; e < p.experts; e += 32) {
        const float l = raw[e];
        key[e] = rank_of((p.softmax ? expf(l - top) / total : sigmoidf_(l)) + __uint_as_float(key[e]));
      }
    } else {  // the scores' order is the logits'
#pragma unroll 8
      for (int e = lane; e < p.experts; e += 32) key[e] = rank_of(raw[e]);
    }
    __syncwarp();
    int which = 0;  // lane s: the s-th choice
#pragma unroll 1
    for (int s = 0; s < p.top_k; ++s) {
      uint32_t best = 0u;
      int at = 0x7FFFFFFF;
#pragma unroll 8
      for (int e = lane; e < p.experts; e += 32) {
        const uint32_t k = key[e];
        if (k > best) {
          best = k;
          at = e;
        }
      }
      const uint32_t most = __reduce_max_sync(0xffffffffu, best);
      const int e = (int)__reduce_min_sync(0xffffffffu, best == most ? (uint32_t)at : 0xFFFFFFFFu);
      if (lane == (e & 31)) key[e] = 0u;
      __syncwarp();
      if (lane == s) which = e;
    }
    const bool in = lane < p.top_k;
    const float mine = in ? raw[which] : 0.f;
    __syncwarp();  // (the next token's come there)
    // The chosen scores over their sum.  Both are scaled by exp(-m), m the largest of min(l, 0) (or of l): far out
    // every score may be 0 in f32 where their ratios are not.
    float w;
    if (p.normalise) {
      float m = in ? (p.softmax ? mine : fminf(mine, 0.f)) : -INFINITY;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      w = !in ? 0.f : expf((p.softmax ? mine : fminf(mine, 0.f)) - m);
      if (!p.softmax) w /= 1.f + expf(-fabsf(mine));
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
}

// The experts with tokens, each once, in the order of their numbers.  A warp for each 32 of them.
__device__ __forceinline__ void choose_groups(const RoutedParams &p, Choice &c, uint32_t *keys, bool write) {
  choose_tokens(p, c, keys, write);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int all = p.experts + p.shared, parts = (all + 31) >> 5;
  // The keys' place is TMA's next: their loads and stores (behind choose_tokens' last barrier) come before its writes, which
  // no barrier alone orders after them.
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  auto tokens_of = [&](int e) { return e < p.experts ? c.mask[e] : e < all ? 0xFFFFFFFFu >> (32 - p.rows) : 0u; };
  for (int i = warp; i < parts; i += warps) {
    const uint32_t has = __ballot_sync(0xffffffffu, tokens_of(32 * i + lane) != 0u);
    if (lane == 0) c.count[i] = __popc(has);
  }
  __syncthreads();
  for (int i = warp; i < parts; i += warps) {
    const uint32_t mask = tokens_of(32 * i + lane), has = __ballot_sync(0xffffffffu, mask != 0u);
    const int before = __reduce_add_sync(0xffffffffu, lane < i ? c.count[lane] : 0);
    if (mask) {
      const int g = before + __popc(has & ((1u << lane) - 1u));
      c.group_expert[g] = (uint16_t)(32 * i + lane);
      c.group_mask[g] = mask;
    }
    if (i == parts - 1 && lane == 0) c.groups = before + __popc(has);
  }
  __syncthreads();
}

// expert e's weight for a token, if it has chosen it (otherwise anything)
__device__ __forceinline__ float weight_of(const RoutedParams &p, const Choice &c, int e, int token) {
  if (e >= p.experts) return 1.f;
  const uint4 v = *reinterpret_cast<const uint4 *>(c.index[token]);
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  int slot = 0;
#pragma unroll
  for (int s = 0; s < kRoutedTopK; ++s)
    if (s < p.top_k && (x[s / 2] >> (16 * (s % 2)) & 0xFFFFu) == (uint32_t)e) slot = s;
  return c.weight[token][slot];
}

}  // namespace moe
