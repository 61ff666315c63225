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

constexpr size_t kAlign = 1024;  // of the ring, whose boxes' swizzle goes by the address

// the n-th token of a mask, or -1
__device__ __forceinline__ int token_at(uint32_t mask, int n) {
  for (; n > 0 && mask; --n) mask &= mask - 1u;
  return __ffs(mask) - 1;
}

// A unit: 16 rows of a group's gate and up matrices.  Column j of the right operand is the group's j-th token.
template <typename T, int BITS, int NT>
struct UpJob {
  const RoutedParams &p;
  const RoutedMaps &maps;
  const Choice &c;
  int units, segs, tiles, strips;
  int row_ahead;
  bool shared_ahead;
  unsigned some;
  Tokens<NT> x;
  Meta meta[2];
  Tile<T, BITS, 2, NT> t;
  __device__ __forceinline__ void copies_begun() const {}
  __device__ __forceinline__ void load_at(int unit, int, int) {
    const int group = unit / strips;
    row_ahead = c.expert[group] * p.inter + (unit - group * strips) * 16;
    shared_ahead = group >= c.routed;
  }
  __device__ __forceinline__ void load(char *place, uint64_t *bar, int tile) const {
    const int i = threadIdx.x & 31, box = i % kBoxes<BITS>;
    if (i >= 2 * kBoxes<BITS>) return;
    const CUtensorMap *gate = shared_ahead ? &maps.s_gate : &maps.gate, *up = shared_ahead ? &maps.s_up : &maps.up;
    tma_load_2d(place + i * kBoxBytes, i < kBoxes<BITS> ? gate : up, bar, (tile * kBoxes<BITS> + box) * (BITS == 16 ? 32 : 64), row_ahead);
  }
  __device__ __forceinline__ void use_at(int unit, int, int) {
    const int group = unit / strips, r = (unit - group * strips) * 16, e = c.expert[group], lane = threadIdx.x & 31;
    const uint32_t mask = c.group_mask[group];
    some = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int token = token_at(mask, 8 * i + (lane >> 2));
      x.row[i] = token >= 0 ? static_cast<const char *>(p.x) + token * p.ld_x * 2 : nullptr;
      some |= (__popc(mask) > 8 * i ? 1u : 0u) << i;
    }
    if constexpr (BITS == 4) {
      const bool sh = group >= c.routed;
      const long long row = (long long)e * p.inter + r;
      meta[0].at(sh ? p.s_gate : p.gate, row, p.inter - r);
      meta[1].at(sh ? p.s_up : p.up, row, p.inter - r);
    }
  }
  __device__ __forceinline__ void fetch(int tile) {
    t.fetch(x, tile * kTileK<BITS>, p.hidden);
    if constexpr (BITS == 4) t.fetch_meta(meta, tile * kTileK<BITS>, p.gate.group_shift);
  }
  __device__ __forceinline__ void multiply(uint32_t place, float (&acc)[2][NT][4]) {
    if constexpr (BITS == 4) t.multiply(place, some, acc, p.gate.group_shift, p.gate.zeros || p.up.zeros);
    else t.multiply(place, some, acc);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int, int, int thread, int threads, Sum sum) const {
    const int group = unit / strips, r = (unit - group * strips) * 16;
    const uint32_t mask = c.group_mask[group];
    const int count = __popc(mask);
    for (int i = thread; i < 16 * count; i += threads) {
      const int row = i & 15, column = i >> 4, token = token_at(mask, column);
      if (r + row >= p.inter) continue;
      const int slot = slot_of(p, c, group, token);
      const float w = group < c.routed ? c.weight[token][slot] : 1.f;
      // rounded to 16 bits as the tensor cores' operand, as the gated block does
      const T h = from_f32<T>(act_value(p.act, sum(0, row, column)) * sum(1, row, column) * w);
      p.h[((long long)token * (p.top_k + p.shared) + slot) * p.inter + r + row] = *reinterpret_cast<const uint16_t *>(&h);
    }
  }
};

// ---- down ----

// A unit: 16 rows of every group's matrix.  Column j of the right operand is token j for every group.
template <typename T, int BITS, int NT>
struct DownJob {
  const RoutedParams &p;
  const RoutedDownMaps &maps;
  const Choice &c;
  int units, segs, tiles;
  int row_ahead;
  bool shared_ahead;
  unsigned some;
  Tokens<NT> x;
  Meta meta[1];
  Tile<T, BITS, 1, NT> t;
  __device__ __forceinline__ void copies_begun() const { pdl_wait(); }  // h comes from the kernel before
  __device__ __forceinline__ void load_at(int unit, int, int group) {
    row_ahead = c.expert[group] * p.hidden + unit * 16;
    shared_ahead = group >= c.routed;
  }
  __device__ __forceinline__ void load(char *place, uint64_t *bar, int tile) const {
    const int i = threadIdx.x & 31;
    if (i < kBoxes<BITS>)
      tma_load_2d(place + i * kBoxBytes, shared_ahead ? &maps.s_down : &maps.down, bar,
                  (tile * kBoxes<BITS> + i) * (BITS == 16 ? 32 : 64), row_ahead);
  }
  __device__ __forceinline__ void use_at(int unit, int, int group) {
    const int e = c.expert[group], lane = threadIdx.x & 31;
    const uint32_t mask = c.group_mask[group];
    some = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int token = 8 * i + (lane >> 2);
      x.row[i] = nullptr;
      if (mask >> token & 1)
        x.row[i] = reinterpret_cast<const char *>(
            p.h + ((long long)token * (p.top_k + p.shared) + slot_of(p, c, group, token)) * p.inter);
      some |= (mask >> (8 * i) & 255u ? 1u : 0u) << i;
    }
    if constexpr (BITS == 4) meta[0].at(group >= c.routed ? p.s_down : p.down, (long long)e * p.hidden + unit * 16, p.hidden - unit * 16);
  }
  __device__ __forceinline__ void fetch(int tile) {
    t.fetch(x, tile * kTileK<BITS>, p.inter);
    if constexpr (BITS == 4) t.fetch_meta(meta, tile * kTileK<BITS>, p.down.group_shift);
  }
  __device__ __forceinline__ void multiply(uint32_t place, float (&acc)[1][NT][4]) {
    if constexpr (BITS == 4) t.multiply(place, some, acc, p.down.group_shift, p.down.zeros != nullptr);
    else t.multiply(place, some, acc);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int, int, int thread, int threads, Sum sum) const {
    for (int i = thread; i < 16 * p.rows; i += threads) {
      const int row = i & 15, token = i >> 4;
      if (unit * 16 + row < p.hidden) static_cast<T *>(p.y)[token * p.ld_y + unit * 16 + row] = from_f32<T>(sum(0, row, token));
    }
  }
};

template <bool UP, int BITS>
constexpr int kRoutedStages = UP ? (BITS == 16 ? 2 : 4) : (BITS == 16 ? 5 : 8);
template <bool UP, int BITS, int NT>
constexpr size_t kRoutedSmem =
    kFewWarps * (kRoutedStages<UP, BITS> * (UP ? 2 : 1) * kBoxes<BITS> * kBoxBytes + (UP ? 2 : 1) * NT * kPartFloats * sizeof(float)) + kAlign;

template <typename T, int BITS, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
    routed_up_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedMaps maps) {
  extern __shared__ char smem[];
  __shared__ Choice c;
  char *ring = smem + (-smem_u32(smem) & (kAlign - 1));
  pdl_wait();
  // The down kernel's CTAs may come, choose and fetch weights: not earlier, as they read the logits.
  pdl_trigger();
  choose(p, c, blockIdx.x == 0);
  const int strips = (p.inter + 15) / 16;
  UpJob<T, BITS, NT> job{p, maps, c, c.groups * strips, 1, (p.hidden + kTileK<BITS> - 1) / kTileK<BITS>, strips};
  stream_units<2, 2, NT, kRoutedStages<true, BITS>, 2 * kBoxes<BITS>>(job, ring, 3, p.waits.status, p.waits.ns, p.waits.inject);
}

template <typename T, int BITS, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
    routed_down_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedDownMaps maps) {
  extern __shared__ char smem[];
  __shared__ Choice c;
  char *ring = smem + (-smem_u32(smem) & (kAlign - 1));
  choose(p, c, false);
  DownJob<T, BITS, NT> job{p, maps, c, (p.hidden + 15) / 16, c.groups, (p.inter + kTileK<BITS> - 1) / kTileK<BITS>};
  stream_units<1, 1, NT, kRoutedStages<false, BITS>, kBoxes<BITS>>(job, ring, 3, p.waits.status, p.waits.ns, p.waits.inject);
}

template <typename T, int BITS, int NT>
cudaError_t layer_launch(const RoutedParams &p, const RoutedMaps &maps, const RoutedDownMaps &down, int num_sms, cudaStream_t st) {
  constexpr size_t smem_up = kRoutedSmem<true, BITS, NT>, smem_down = kRoutedSmem<false, BITS, NT>;
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = allow_smem((const void *)routed_up_kernel<T, BITS, NT>, smem_up, done[0]);
  if (e == cudaSuccess) e = allow_smem((const void *)routed_down_kernel<T, BITS, NT>, smem_down, done[1]);
  const dim3 threads(32 * kFewWarps);
  if (e == cudaSuccess)
    e = launch_pdl(p.router_f32 ? routed_logits_kernel<T, float> : routed_logits_kernel<T, T>,
                   dim3((p.experts + kRouteExperts - 1) / kRouteExperts), dim3(256), 0, st, p);
  const long long groups = (long long)(p.rows * p.top_k < p.experts ? p.rows * p.top_k : p.experts) + p.shared;
  const long long units = groups * ((p.inter + 15) / 16), units_down = (p.hidden + 15) / 16, most = 2ll * num_sms;
  if (e == cudaSuccess)
    e = launch_pdl(routed_up_kernel<T, BITS, NT>, dim3((unsigned)(units < most ? units : most)), threads, smem_up, st, p, maps);
  if (e == cudaSuccess)
    e = launch_pdl(routed_down_kernel<T, BITS, NT>, dim3((unsigned)(units_down < most ? units_down : most)), threads, smem_down, st, p, down);
  return e;
}

template <typename T, int BITS>
cudaError_t routed_rows(const RoutedParams &p, const RoutedMaps &maps, const RoutedDownMaps &down, int num_sms, cudaStream_t st) {
  if (p.rows <= 8) return layer_launch<T, BITS, 1>(p, maps, down, num_sms, st);
  if (p.rows <= 16) return layer_launch<T, BITS, 2>(p, maps, down, num_sms, st);
  return layer_launch<T, BITS, 4>(p, maps, down, num_sms, st);
}

}  // namespace

cudaError_t launch_routed(const RoutedParams &p, const RoutedMaps &maps, const RoutedDownMaps &down, bool f16, bool bits4,
                          int num_sms, cudaStream_t st) {
  if (f16) return bits4 ? routed_rows<__half, 4>(p, maps, down, num_sms, st) : routed_rows<__half, 16>(p, maps, down, num_sms, st);
  return bits4 ? routed_rows<__nv_bfloat16, 4>(p, maps, down, num_sms, st) : routed_rows<__nv_bfloat16, 16>(p, maps, down, num_sms, st);
}

}  // namespace moe
