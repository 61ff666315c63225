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

// The experts' tokens, eight at a time, which are the columns of the tensor cores' right operand.  Gate and up take any
// eight tokens of an expert together; down takes tokens 8 j .. 8 j + 7 for every expert, so that its accumulators may add
// all experts' products.  An expert with more tokens, or tokens of several eights, comes several times, one after
// another: its weights then come from the L2.  Shared experts have the numbers from `experts` on, and come last.
constexpr int kEightsMax = kRoutedRows / 8, kUpMax = kRoutedRows * kRoutedTopK + kRoutedShared * kEightsMax;
constexpr int kDownMax = 8 * kRoutedTopK + kRoutedShared;

constexpr int kGroupsMax = kRoutedRows * kRoutedTopK + kRoutedShared;

struct Choice {
  int up, down[kEightsMax];                        // entries
  int groups;                                      // experts with tokens, each once
  int count[(kRoutedExperts + kRoutedShared + 31) / 32];
  uint16_t group_expert[kGroupsMax];
  uint32_t group_mask[kGroupsMax];
  uint32_t mask[kRoutedExperts];                   // each expert's tokens
  uint32_t up_mask[kUpMax];
  uint16_t up_expert[kUpMax];
  uint16_t down_expert[kEightsMax][kDownMax];
  uint16_t index[kRoutedRows][kRoutedTopK];
  float weight[kRoutedRows][kRoutedTopK];
};

// a number for each float that grows with it (the same for both zeros); NaN below all others, and 0 for none
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A warp for each token.  Every thread of the CTA; ends with a barrier.  keys: 512 words of shared memory for each warp.
// The loops are kept short: a kernel runs this code once, and its way into the instruction caches took most of its time
// while the experts were held in registers (16 of them a lane, each loop unrolled: 8.7 us of one token of 256 experts).
__device__ __forceinline__ void choose_tokens(const RoutedParams &p, Choice &c, uint32_t *keys, bool write) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  uint32_t *key = keys + warp * kRoutedExperts;
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) c.mask[e] = 0u;
  __syncthreads();
#pragma unroll 1
  for (int t = warp; t < p.rows; t += warps) {
    const float *logits = p.logits + t * p.experts;
    float top = -INFINITY, total = 0.f;
    if (p.softmax && (p.bias || !p.normalise)) {  // a score itself is wanted, not ratios or the order alone
#pragma unroll 4
      for (int e = lane; e < p.experts; e += 32) top = fmaxf(top, __ldcg(logits + e));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
      for (int e = lane; e < p.experts; e += 32) total += expf(__ldcg(logits + e) - top);
      total = warp_sum(total);
    }
    if (p.bias) {
#pragma unroll 1
      for (int e = lane; e < p.experts; e += 32) {
        const float l = __ldcg(logits + e);
        key[e] = rank_of((p.softmax ? expf(l - top) / total : sigmoidf_(l)) + p.bias[e]);
      }
    } else {  // the scores' order is the logits'
#pragma unroll 8
      for (int e = lane; e < p.experts; e += 32) key[e] = rank_of(__ldcg(logits + e));
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
    const float mine = in ? __ldcg(logits + which) : 0.f;
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

// The same as lists of eights of tokens.
__device__ __forceinline__ void choose(const RoutedParams &p, Choice &c, uint32_t *keys, bool write) {
  choose_tokens(p, c, keys, write);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const int all = p.experts + p.shared;
    int up = 0, down[kEightsMax] = {};
    for (int e0 = 0; e0 < all; e0 += 32) {
      const int e = e0 + lane;
      uint32_t mask = e < p.experts ? c.mask[e] : e < all ? 0xFFFFFFFFu >> (32 - p.rows) : 0u;
#pragma unroll
      for (int j = 0; j < kEightsMax; ++j) {
        const uint32_t has = __ballot_sync(0xffffffffu, mask >> (8 * j) & 255u);
        if (mask >> (8 * j) & 255u) c.down_expert[j][down[j] + __popc(has & ((1u << lane) - 1u))] = (uint16_t)e;
        down[j] += __popc(has);
      }
      const int passes = (__popc(mask) + 7) / 8;
      int at = passes;  // the entries of the lanes up to this one
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
      }
      const int added = __shfl_sync(0xffffffffu, at, 31);
      at += up - passes;
      up += added;
      for (; mask; ++at) {  // eight tokens at a time
        uint32_t rest = mask;
        for (int i = 0; i < 8 && rest; ++i) rest &= rest - 1u;
        c.up_expert[at] = (uint16_t)e;
        c.up_mask[at] = mask ^ rest;
        mask = rest;
      }
    }
    if (lane == 0) {
      c.up = up;
#pragma unroll
      for (int j = 0; j < kEightsMax; ++j) c.down[j] = down[j];
    }
  }
  __syncthreads();
}

// the place of expert e among token's, which has chosen it: that of its row of h
__device__ __forceinline__ int slot_of(const RoutedParams &p, const Choice &c, int e, int token) {
  if (e >= p.experts) return p.top_k + e - p.experts;
  int slot = 0;
  for (int s = 1; s < p.top_k; ++s)
    if (c.index[token][s] == e) slot = s;
  return slot;
}
__device__ __forceinline__ uint16_t *h_row(const RoutedParams &p, const Choice &c, int e, int token) {
  return p.h + ((long long)token * (p.top_k + p.shared) + slot_of(p, c, e, token)) * p.inter;
}
// the n-th token of a mask, or -1
__device__ __forceinline__ int token_at(uint32_t mask, int n) {
  for (; n > 0 && mask; --n) mask &= mask - 1u;
  return __ffs(mask) - 1;
}

// ---- the weights' way through a warp ----
//
// A unit is 16 rows of the result; its `segs` matrices of `tiles` tiles each are dealt to the CTA's 8 warps, whose sums
// meet in shared memory in the warps' order.  Each warp has a ring of its own, filled across units: a place holds a tile of
// M strips, brought by TMA, and the tokens' columns, brought by the lanes (cp.async), of which there may be few.  Both
// arrive on one barrier, and no barrier of several warps is met before a unit ends.

// place: M strips, then the tokens' columns
template <int BITS, int M>
struct Place {
  static constexpr int kWeights = M * kBoxes<BITS> * kBoxBytes, kPieces = BITS == 16 ? 2 : 4, kTokens = kPieces * 8 * 64;
  static constexpr int kBytes = kWeights + kTokens;
};

// Copies a lane's part of the tokens' columns: row g's 16 bytes t of each piece; zeros where there are none.
template <int PIECES>
__device__ __forceinline__ void copy_tokens(uint32_t dst, const uint16_t *row, const void *any, int k, int end) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    const int col = k + 32 * c + 8 * t, line = 8 * c + g;
    const bool in = row && col < end;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst + line * 64 + ((t ^ (line >> 1 & 3)) << 4)),
                 "l"(in ? static_cast<const void *>(row + col) : any), "r"(in ? 16 : 0)
                 : "memory");
  }
}

//   int units, tiles, k;  int segs(unit)
//   void weights_at(unit, seg);  void weights(place, barrier, tile)      by one lane
//   void tokens_at(unit, seg)    sets `row`, the lane's token
//   void use_at(unit, seg);  void multiply(place, tile, acc);  void finish(unit, thread, sum)
template <int BITS, int M, int STAGES, typename Job>
__device__ __forceinline__ void stream_units(Job &job, char *smem, const Waits &waits) {
  using P = Place<BITS, M>;
  constexpr int kw = kFewWarps;
  __shared__ uint64_t full[kFewWarps][STAGES], never;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char *own = smem + warp * (STAGES * P::kBytes);
  float *parts = reinterpret_cast<float *>(smem + kw * STAGES * P::kBytes);
  if (threadIdx.x < kw * STAGES) mbar_init(&full[0][0] + threadIdx.x, 1 + 32);
  if (threadIdx.x == 0) {
    mbar_init(&never, 1);
    abort_flag = 0;
  }
  if (threadIdx.x < kw * STAGES) fence_mbar_init();
  __syncthreads();
  // a place in the job's tiles that this warp has come to
  struct At {
    int unit, seg, tile, segs;
  };
  auto settle = [&](At &a) {  // past the end of a matrix: the next one that has a tile for this warp
    while (a.unit < job.units && a.tile >= job.tiles) {
      a.tile -= job.tiles;
      if (++a.seg >= a.segs) {
        a.unit += gridDim.x;
        a.seg = 0;
        a.tile = warp;
        if (a.unit < job.units) a.segs = job.segs(a.unit);
      }
    }
  };
  auto start = [&] {
    At a = {(int)blockIdx.x, 0, warp, 0};
    if (a.unit < job.units) a.segs = job.segs(a.unit);
    settle(a);
    return a;
  };
  auto weights = [&](At &a, int stage) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[warp][stage], P::kWeights);
      job.weights(own + stage * P::kBytes, &full[warp][stage], a.tile);
    }
  };
  auto tokens = [&](At &a, int stage) {
    copy_tokens<P::kPieces>(smem_u32(own) + stage * P::kBytes + P::kWeights, job.row, job.p.x, a.tile * kTileK<BITS>, job.k);
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[warp][stage])) : "memory");
  };
  int begun = 0, used = 0;
  // the first weights need not wait for what makes the tokens' columns
  At ahead = start();
  if (ahead.unit < job.units) job.weights_at(ahead.unit, ahead.seg);
  for (int s = 0; s < STAGES && ahead.unit < job.units; ++s) {
    weights(ahead, s);
    ahead.tile += kw;
    if (ahead.tile >= job.tiles) {
      settle(ahead);
      if (ahead.unit < job.units) job.weights_at(ahead.unit, ahead.seg);
    }
  }
  job.tokens_ready();
  ahead = start();
  if (ahead.unit < job.units) job.tokens_at(ahead.unit, ahead.seg);
  for (; begun < STAGES && ahead.unit < job.units; ++begun) {
    tokens(ahead, begun);
    ahead.tile += kw;
    if (ahead.tile >= job.tiles) {
      settle(ahead);
      if (ahead.unit < job.units) job.tokens_at(ahead.unit, ahead.seg);
    }
  }
  if (waits.inject && blockIdx.x == 0) wait_bounded(&never, 0, &abort_flag, waits.status, waits.ns);  // test hook: a wait that runs out
  int stage = 0, phase = 0;
  for (int unit = blockIdx.x; unit < job.units; unit += gridDim.x) {
    float acc[M][1][4];
#pragma unroll
    for (int m = 0; m < M; ++m) acc[m][0][0] = acc[m][0][1] = acc[m][0][2] = acc[m][0][3] = 0.f;
    const int segs = job.segs(unit);
    int tile = warp;
    for (int seg = 0; seg < segs; ++seg, tile -= job.tiles) {
      if (tile >= job.tiles) continue;
      job.use_at(unit, seg, tile);
      for (; tile < job.tiles; tile += kw) {
        job.meta_at(tile);
        // (the lanes agree: one that gave up takes the warp with it)
        if (!__all_sync(0xffffffffu, wait_bounded(&full[warp][stage], phase, &abort_flag, waits.status, waits.ns))) continue;
        const uint32_t place = smem_u32(own) + stage * P::kBytes;
        job.multiply(place, place + P::kWeights, acc);
        __syncwarp();
        ++used;
        if (ahead.unit < job.units) {
          weights(ahead, stage);
          tokens(ahead, stage);
          ++begun;
          ahead.tile += kw;
          if (ahead.tile >= job.tiles) {
            settle(ahead);
            if (ahead.unit < job.units) {
              job.weights_at(ahead.unit, ahead.seg);
              job.tokens_at(ahead.unit, ahead.seg);
            }
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) put_part(parts + (warp * M + m) * kPartFloats, acc[m][0]);
    __syncthreads();
    if (threadIdx.x < 128)
      job.finish(unit, threadIdx.x & 15, threadIdx.x >> 4, [&](int m) {
        const float *at = parts + m * kPartFloats + part_at(threadIdx.x & 15, threadIdx.x >> 4);
        float v = at[0];
#pragma unroll
        for (int w = 1; w < kw; ++w) v += at[w * M * kPartFloats];
        return v;
      });
    __syncthreads();
  }
  // after a wait that ran out: no copy may land in memory that the CTA has left
  for (int nobody = 0; used < begun; ++used) {
    mbar_wait_bounded(&full[warp][stage], phase, &nobody, waits.status, waits.ns);
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
}

// ---- gate and up ----

constexpr size_t kAlign = 512;  // of the ring, whose boxes' swizzle goes by the address

// A unit: 16 rows of an entry's gate and up matrices.
template <typename T, int BITS, int PIECES, bool ZP>
struct UpJob {
  const RoutedParams &p;
  const RoutedMaps &maps;
  const Choice &c;
  int units, tiles, k, strips;
  int map_row;
  bool shared_ahead;
  const uint16_t *row;
  Tile<T, BITS, PIECES, ZP, 2, 1, false> t;
  __device__ __forceinline__ int segs(int) const { return 1; }
  __device__ __forceinline__ void weights_at(int unit, int) {
    const int entry = unit / strips, e = c.up_expert[entry];
    shared_ahead = e >= p.experts;
    map_row = (shared_ahead ? e - p.experts : e) * p.inter + (unit - entry * strips) * 16;
  }
  __device__ __forceinline__ void weights(char *place, uint64_t *bar, int tile) const {
    const CUtensorMap *gate = shared_ahead ? &maps.s_gate : &maps.gate, *up = shared_ahead ? &maps.s_up : &maps.up;
#pragma unroll
    for (int b = 0; b < kBoxes<BITS>; ++b) {
      const int x = (tile * kBoxes<BITS> + b) * (BITS == 16 ? 32 : 64);
      tma_load_2d(place + b * kBoxBytes, gate, bar, x, map_row);
      tma_load_2d(place + (kBoxes<BITS> + b) * kBoxBytes, up, bar, x, map_row);
    }
  }
  __device__ __forceinline__ void tokens_ready() const {}
  __device__ __forceinline__ void tokens_at(int unit, int) {
    const int token = token_at(c.up_mask[unit / strips], (threadIdx.x & 31) >> 2);
    row = token >= 0 ? static_cast<const uint16_t *>(p.x) + token * p.ld_x : nullptr;
  }
  __device__ __forceinline__ void use_at(int unit, int, int tile) {
    if constexpr (BITS == 4) {
      const int entry = unit / strips, r = (unit - entry * strips) * 16, e = c.up_expert[entry];
      const bool sh = e >= p.experts;
      const long long first = (long long)(sh ? e - p.experts : e) * p.inter + r;
      t.meta.row[0].at(sh ? p.s_gate : p.gate, first, p.inter - r);
      t.meta.row[1].at(sh ? p.s_up : p.up, first, p.inter - r);
      t.meta.begin(tile, kFewWarps, p.gate.groups);
    }
  }
  __device__ __forceinline__ void meta_at(int tile) {
    if constexpr (BITS == 4) t.meta.advance(tile);
  }
  __device__ __forceinline__ void multiply(uint32_t place, uint32_t tokens, float (&acc)[2][1][4]) {
    t.multiply(place, tokens, 1u, acc);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int r, int column, Sum sum) const {
    const int entry = unit / strips, at = (unit - entry * strips) * 16 + r, e = c.up_expert[entry];
    const int token = token_at(c.up_mask[entry], column);
    if (token < 0 || at >= p.inter) return;
    const float w = e < p.experts ? c.weight[token][slot_of(p, c, e, token)] : 1.f;
    // rounded to 16 bits as the tensor cores' operand, as the gated block does
    const T h = from_f32<T>(act_value(p.act, sum(0)) * sum(1) * w);
    h_row(p, c, e, token)[at] = *reinterpret_cast<const uint16_t *>(&h);
  }
};

// ---- down ----

// A unit: 16 rows of every expert's matrix that one of eight tokens has chosen.
template <typename T, int BITS, int PIECES, bool ZP>
struct DownJob {
  const RoutedParams &p;
  const RoutedMaps &maps;
  const Choice &c;
  int units, tiles, k, eights;
  int map_row;
  bool shared_ahead;
  const uint16_t *row;
  Tile<T, BITS, PIECES, ZP, 1, 1, false> t;
  __device__ __forceinline__ int segs(int unit) const { return c.down[unit % eights]; }
  __device__ __forceinline__ void weights_at(int unit, int seg) {
    const int e = c.down_expert[unit % eights][seg];
    shared_ahead = e >= p.experts;
    map_row = (shared_ahead ? e - p.experts : e) * p.hidden + unit / eights * 16;
  }
  __device__ __forceinline__ void weights(char *place, uint64_t *bar, int tile) const {
#pragma unroll
    for (int b = 0; b < kBoxes<BITS>; ++b)
      tma_load_2d(place + b * kBoxBytes, shared_ahead ? &maps.s_gate : &maps.gate, bar, (tile * kBoxes<BITS> + b) * (BITS == 16 ? 32 : 64),
                  map_row);
  }
  __device__ __forceinline__ void tokens_ready() const { pdl_wait(); }  // h comes from the kernel before
  __device__ __forceinline__ void tokens_at(int unit, int seg) {
    const int eight = unit % eights, e = c.down_expert[eight][seg], token = 8 * eight + ((threadIdx.x & 31) >> 2);
    const uint32_t mask = e >= p.experts ? 0xFFFFFFFFu >> (32 - p.rows) : c.mask[e];
    row = mask >> token & 1 ? h_row(p, c, e, token) : nullptr;
  }
  __device__ __forceinline__ void use_at(int unit, int seg, int tile) {
    if constexpr (BITS == 4) {
      const int e = c.down_expert[unit % eights][seg], r = unit / eights * 16;
      const bool sh = e >= p.experts;
      t.meta.row[0].at(sh ? p.s_down : p.down, (long long)(sh ? e - p.experts : e) * p.hidden + r, p.hidden - r);
      t.meta.begin(tile, kFewWarps, p.down.groups);
    }
  }
  __device__ __forceinline__ void meta_at(int tile) {
    if constexpr (BITS == 4) t.meta.advance(tile);
  }
  __device__ __forceinline__ void multiply(uint32_t place, uint32_t tokens, float (&acc)[1][1][4]) {
    t.multiply(place, tokens, 1u, acc);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int r, int column, Sum sum) const {
    const int at = unit / eights * 16 + r, token = unit % eights * 8 + column;
    if (token < p.rows && at < p.hidden) static_cast<T *>(p.y)[token * p.ld_y + at] = from_f32<T>(sum(0));
  }
};

// ---- 16-bit weights: tcgen05 ----
//
// The weights are the left operand as they lie (128 rows x 64 columns a step, K-major, by TMA), all tokens' columns the
// right one, so that nothing but copies and one instruction for 16 columns is left: the kernels run at the pace of memory.
// (On mma.sync, a warp's strips of 16 rows as above, one token of 256 experts of 4096 x 2048 took 72 to 83 us: copies of
// 16 rows x 64 bytes do not come faster than 3.2 TB/s.)
//
// Up: a tile is 64 rows of gate and 64 of up; two accumulators in TMEM, so that a tile's epilogue runs beside the next
// tile's products.  h lies by experts, [expert's place among the chosen][tokens, up to a multiple of 8][inter], with zeros
// for the tokens that have not chosen it: the down kernel's right operand, as it needs it.
// Down: a tile is 128 rows; the experts' steps are shared by the CTAs of a cluster, whose sums meet in shared memory.

constexpr int kTcThreads = 192, kTcRows = 128, kTcW = kTcRows * 128;
template <int NC>
constexpr int kTcStage = kTcW + NC * 128;
template <int NC>
constexpr int kTcRing = NC == 16 ? 5 : 4;  // two CTAs on an SM: the down kernel's come while the up kernel's end
template <int NC>
constexpr size_t kTcSmem = kTcRing<NC> * kTcStage<NC> + 1024;

// NC columns of this thread's lane of an accumulator
template <int NC>
__device__ __forceinline__ void read_accumulator(uint32_t at, float (&v)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; i += 16) tmem_ld16(at + i, reinterpret_cast<float(&)[16]>(v[i]));
}

template <bool UP, typename T, int NC>
__global__ void __launch_bounds__(kTcThreads, 2)
    routed_tc_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedMaps maps, int splits) {
  constexpr int kTcStages = kTcRing<NC>;
  extern __shared__ char smem[];
  __shared__ Choice c;
  __shared__ __align__(8) uint64_t full[kTcStages], empty[kTcStages], tfull[2], tempty[2], mma_done, never;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;
  __shared__ float sums[UP ? 2 : 1][NC * (UP ? 64 : kTcRows)];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  char *ring = smem + (-smem_u32(smem) & 1023u);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(&mma_done, 1);
    mbar_init(&never, 1);
    abort_flag = 0;
    issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, 64);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if constexpr (UP) {
    pdl_wait();
    // The down kernel's CTAs may come, choose and fetch weights: not earlier, as they read the logits.
    pdl_trigger();
  }
  choose_groups(p, c, reinterpret_cast<uint32_t *>(ring), UP && blockIdx.x == 0);  // (the ring is not in use yet)
  volatile int *abort_p = &abort_flag;
  const Waits &w = p.waits;
  const int rows8 = (p.rows + 7) / 8 * 8, depth = UP ? p.hidden : p.inter, steps = (depth + 63) / 64;
  const int tiles = UP ? (p.inter + 63) / 64 : 1;  // of an expert
  // UP: units of an expert's tile, one after another; otherwise one tile, and this CTA's share of all experts' steps
  const int rank = UP ? 0 : blockIdx.x % splits, tile_down = UP ? 0 : blockIdx.x / splits;
  const int units = UP ? c.groups * tiles : 1, unit0 = UP ? blockIdx.x : 0, unit_step = UP ? gridDim.x : 1;
  const long long all = (long long)c.groups * steps;
  const int first = UP ? 0 : (int)(all * rank / splits), end = UP ? steps : (int)(all * (rank + 1) / splits);

  if (warp == 0) {
    // ---------------- copies ----------------
    const uint32_t ring0 = smem_u32(ring), bytes = kTcW + rows8 * 128;
    RingPos<kTcStages> pos;
    int j = 0, group = UP ? 0 : first / steps, k = UP ? 0 : first % steps, unit = unit0, step = first;
    auto weights = [&](int s) {
      const uint32_t at = ring0 + s * kTcStage<NC>, bar = smem_u32(&full[s]);
      mbar_expect_one(bar, bytes);
      const int e = c.group_expert[group];
      const bool shared = e >= p.experts;
      const int row = (shared ? e - p.experts : e) * (UP ? p.inter : p.hidden);
      if constexpr (UP) {
        const int r = row + (unit - group * tiles) * 64;
        tma_load_2d_one<false>(at, shared ? &maps.s_gate : &maps.gate, bar, k * 64, r);
        tma_load_2d_one<false>(at + 64 * 128, shared ? &maps.s_up : &maps.up, bar, k * 64, r);
      } else {
        tma_load_2d_one<false>(at, shared ? &maps.s_gate : &maps.gate, bar, k * 64, row + tile_down * kTcRows);
      }
    };
    auto tokens = [&](int s, int g, int kk) {
      tma_load_2d_one<false>(ring0 + s * kTcStage<NC> + kTcW, &maps.tokens, smem_u32(&full[s]), kk * 64, UP ? 0 : g * rows8);
    };
    auto next = [&] {
      ++step;
      if (++k == steps) {
        k = 0;
        if (!UP) ++group;
      }
      if (UP && step == end) {
        step = 0;
        unit += unit_step;
        group = unit / tiles;
      }
    };
    if (UP) group = unit / tiles;
    bool ok = true;
    if constexpr (!UP) {  // the first weights need not wait for h
      const int g0 = group, k0 = k;
      for (; j < kTcStages && step < end; ++j, next()) weights(j);
      pdl_wait();
      pdl_trigger();
      int g = g0, kk = k0;
      for (int i = 0; i < j; ++i) {
        tokens(i, g, kk);
        if (++kk == steps) {
          kk = 0;
          ++g;
        }
      }
      for (int i = 0; i < j; ++i) pos.next();
    }
    for (; unit < units && step < end; ++j, pos.next(), next()) {
      if (!warp_wait(&empty[pos.slot], pos.round ^ 1u, abort_p, w.status, w.ns)) {
        ok = false;
        break;
      }
      weights(pos.slot);
      tokens(pos.slot, group, k);
    }
    (void)ok;
    if (lane == 0) issued = j;
  } else if (warp == 1) {
    // ---------------- products ----------------
    if (w.inject && blockIdx.x == 0) (void)warp_wait(&never, 0u, abort_p, w.status, w.ns);  // test hook: a wait that runs out
    const uint32_t idesc = std::is_same<T, __half>::value ? idesc_f16_f32(kTcRows, NC) : idesc_bf16_f32(kTcRows, NC);
    const uint64_t a0 = smem_desc_sw128(smem_u32(ring)), b0 = a0 + (kTcW >> 4);
    RingPos<kTcStages> pos;
    RingPos<2> acc;
    bool ok = true;
    for (int unit = unit0; ok && unit < units; unit += unit_step, acc.next()) {
      if (!warp_wait(&tempty[acc.slot], acc.round ^ 1u, abort_p, w.status, w.ns)) break;
      for (int step = first; step < end; ++step, pos.next()) {
        if (!warp_wait(&full[pos.slot], pos.round, abort_p, w.status, w.ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = pos.slot * (kTcStage<NC> >> 4), d = tmem + acc.slot * 32;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_one<false, false>(d, a0 + (at + k * 2), b0 + (at + k * 2), idesc, step > first || k > 0 ? 1u : 0u);
        tc_commit_one<false>(smem_u32(&empty[pos.slot]));
      }
      if (ok) tc_commit_one<false>(smem_u32(&tfull[acc.slot]));
    }
    // every MMA this warp issued completes before TMEM is freed
    tc_commit_one<false>(smem_u32(&mma_done));
    int no_abort = 0;
    (void)wait_bounded(&mma_done, 0u, &no_abort, w.status, w.ns);
  } else {
    // ---------------- results ----------------
    const int q = warp & 3, row = q * 32 + lane;
    RingPos<2> acc;
    for (int unit = unit0; unit < units; unit += unit_step, acc.next()) {
      float v[NC];
      const bool ok = (UP || first < end) && warp_wait(&tfull[acc.slot], acc.round, abort_p, w.status, w.ns);
      if (ok) {
        tc_fence_after();
        read_accumulator<NC>(tmem + ((uint32_t)(q * 32) << 16) + acc.slot * 32, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc.slot]);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] = 0.f;
      }
      if constexpr (UP) {
        float *u = sums[acc.slot];
        if (q >= 2)
#pragma unroll
          for (int t = 0; t < NC; ++t)
            if (t < p.rows) u[t * 64 + row - 64] = v[t];
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int group = unit / tiles, at = (unit - group * tiles) * 64 + row, e = c.group_expert[group];
        const uint32_t mask = c.group_mask[group];
        if (q < 2 && at < p.inter) {
          uint16_t *h = p.h + (long long)group * rows8 * p.inter + at;
#pragma unroll
          for (int t = 0; t < NC; ++t) {
            if (t >= p.rows) break;
            T out = from_f32<T>(0.f);
            if (mask >> t & 1) {
              const float weight = e < p.experts ? c.weight[t][slot_of(p, c, e, t)] : 1.f;
              // rounded to 16 bits as the tensor cores' operand, as the gated block does
              out = from_f32<T>(act_value(p.act, v[t]) * u[t * 64 + row] * weight);
            }
            h[(long long)t * p.inter] = *reinterpret_cast<const uint16_t *>(&out);
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < NC; ++t)
          if (t < p.rows) sums[0][t * kTcRows + row] = v[t];
      }
    }
  }
  // Copies still in flight after an abort land before the CTA may leave (bounded; otherwise each has landed).
  tc_fence_before();
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) {
    int no_abort = 0;
    for (int s = 0; s < kTcStages; ++s) {
      const int n = issued / kTcStages + (s < issued % kTcStages ? 1 : 0);
      if (n > 0) (void)wait_bounded(&full[s], (uint32_t)((n - 1) & 1), &no_abort, w.status, w.ns);
    }
  }
  if constexpr (!UP) {
    // the CTAs' sums in the order of their ranks, a part of the rows by each
    if (splits > 1) cluster_sync();
    const int part = kTcRows / splits, row0 = rank * part;
    for (int i = threadIdx.x; i < part * p.rows; i += kTcThreads) {
      const int row = row0 + i % part, t = i / part, at = tile_down * kTcRows + row;
      float v = 0.f, x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)  // all loads before the first sum
        if (r < splits)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[r]) : "r"(in_cta(&sums[0][t * kTcRows + row], r)) : "memory");
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < splits) v += x[r];
      if (at < p.hidden) static_cast<T *>(p.y)[t * p.ld_y + at] = from_f32<T>(v);
    }
    if (splits > 1) cluster_sync();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

template <typename T, int NC>
cudaError_t tc_launch(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = allow_smem((const void *)routed_tc_kernel<true, T, NC>, kTcSmem<NC>, done[0]);
  if (e == cudaSuccess)
    e = launch_pdl(p.router_f32 ? routed_logits_kernel<T, float> : routed_logits_kernel<T, T>,
                   dim3((p.experts + kRouteExperts - 1) / kRouteExperts), dim3(256), 0, st, p);
  const long long groups = (p.rows * p.top_k < p.experts ? p.rows * p.top_k : p.experts) + p.shared;
  const long long units = groups * ((p.inter + 63) / 64);
  if (e == cudaSuccess)
    e = launch_pdl(routed_tc_kernel<true, T, NC>, dim3((unsigned)(units < 2 * num_sms ? units : 2 * num_sms)), dim3(kTcThreads), kTcSmem<NC>, st, p,
                   maps, 1);
  if (e != cudaSuccess) return e;
  // as many CTAs to a tile as run at one time, two on an SM (of clusters of 8, 4 and 2 on 152 SMs 32, 72 and 150)
  const int tiles = (p.hidden + kTcRows - 1) / kTcRows;
  const int splits = tiles <= num_sms * 32 / 152 ? 8 : tiles <= num_sms * 72 / 152 ? 4 : tiles <= num_sms * 150 / 152 ? 2 : 1;
  return launch_clusters(routed_tc_kernel<false, T, NC>, kTcSmem<NC>, done[1], tiles, splits, kTcThreads, st, p, down, splits);
}

template <bool UP, int BITS>
constexpr int kRoutedStages = UP ? (BITS == 16 ? 2 : 3) : 4;
template <bool UP, int BITS>
constexpr size_t kRoutedSmem =
    kFewWarps * (kRoutedStages<UP, BITS> * Place<BITS, UP ? 2 : 1>::kBytes + (UP ? 2 : 1) * kPartFloats * sizeof(float)) + kAlign;

template <typename T, int BITS, int PIECES, bool ZP>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
    routed_up_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedMaps maps) {
  extern __shared__ char smem[];
  __shared__ Choice c;
  char *ring = smem + (-smem_u32(smem) & (kAlign - 1));
  pdl_wait();
  // The down kernel's CTAs may come, choose and fetch weights: not earlier, as they read the logits.
  pdl_trigger();
  choose(p, c, reinterpret_cast<uint32_t *>(ring), blockIdx.x == 0);
  const int strips = (p.inter + 15) / 16;
  UpJob<T, BITS, PIECES, ZP> job{p, maps, c, c.up * strips, (p.hidden + kTileK<BITS> - 1) / kTileK<BITS>, p.hidden, strips};
  job.t.x.set(0, 8);
  stream_units<BITS, 2, kRoutedStages<true, BITS>>(job, ring, p.waits);
}

template <typename T, int BITS, int PIECES, bool ZP>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
    routed_down_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedMaps maps) {
  extern __shared__ char smem[];
  __shared__ Choice c;
  char *ring = smem + (-smem_u32(smem) & (kAlign - 1));
  choose(p, c, reinterpret_cast<uint32_t *>(ring), false);
  const int eights = (p.rows + 7) / 8;
  DownJob<T, BITS, PIECES, ZP> job{p, maps, c, (p.hidden + 15) / 16 * eights, (p.inter + kTileK<BITS> - 1) / kTileK<BITS>, p.inter, eights};
  job.t.x.set(0, 8);
  stream_units<BITS, 1, kRoutedStages<false, BITS>>(job, ring, p.waits);
}

template <typename T, int BITS, int PIECES, bool ZP>
cudaError_t layer_launch(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  constexpr size_t smem_up = kRoutedSmem<true, BITS>, smem_down = kRoutedSmem<false, BITS>;
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = allow_smem((const void *)routed_up_kernel<T, BITS, PIECES, ZP>, smem_up, done[0]);
  if (e == cudaSuccess) e = allow_smem((const void *)routed_down_kernel<T, BITS, PIECES, ZP>, smem_down, done[1]);
  const dim3 threads(32 * kFewWarps);
  if (e == cudaSuccess)
    e = launch_pdl(p.router_f32 ? routed_logits_kernel<T, float> : routed_logits_kernel<T, T>,
                   dim3((p.experts + kRouteExperts - 1) / kRouteExperts), dim3(256), 0, st, p);
  const int eights = (p.rows + 7) / 8;
  const long long entries = p.rows * p.top_k + p.shared * eights;  // at most
  const long long units = entries * ((p.inter + 15) / 16), units_down = (long long)eights * ((p.hidden + 15) / 16), most = 2ll * num_sms;
  if (e == cudaSuccess)
    e = launch_pdl(routed_up_kernel<T, BITS, PIECES, ZP>, dim3((unsigned)(units < most ? units : most)), threads, smem_up, st, p, maps);
  if (e == cudaSuccess)
    e = launch_pdl(routed_down_kernel<T, BITS, PIECES, ZP>, dim3((unsigned)(units_down < most ? units_down : most)), threads, smem_down,
                   st, p, down);
  return e;
}

template <typename T>
cudaError_t routed_typed(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, bool bits4, int num_sms,
                         cudaStream_t st) {
  if (!bits4) return p.rows <= 16 ? tc_launch<T, 16>(p, maps, down, num_sms, st) : tc_launch<T, 32>(p, maps, down, num_sms, st);
  const bool zp = p.gate.zeros != nullptr;
  if (p.gate.group_shift == 5)
    return zp ? layer_launch<T, 4, 1, true>(p, maps, down, num_sms, st) : layer_launch<T, 4, 1, false>(p, maps, down, num_sms, st);
  if (p.gate.group_shift == 6)
    return zp ? layer_launch<T, 4, 2, true>(p, maps, down, num_sms, st) : layer_launch<T, 4, 2, false>(p, maps, down, num_sms, st);
  return zp ? layer_launch<T, 4, 4, true>(p, maps, down, num_sms, st) : layer_launch<T, 4, 4, false>(p, maps, down, num_sms, st);
}

}  // namespace

cudaError_t launch_routed(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, bool f16, bool bits4,
                          int num_sms, cudaStream_t st) {
  return f16 ? routed_typed<__half>(p, maps, down, bits4, num_sms, st) : routed_typed<__nv_bfloat16>(p, maps, down, bits4, num_sms, st);
}

}  // namespace moe
