// The norms before and after a block on a plain residual stream, fused with the block's gate and
// residual scale, forward and backward (sm_103a).
//
//   n   = f * rsqrt(mean(f^2) + eps) * w_post           (n = f without w_post)
//   s   = state + scale * gate * n                      (rounded to the stream's type as it is stored)
//   y   = s * rsqrt(mean(s^2) + eps) * w_next           (the next block's input)
//
// Backward, from the stored s and f, with r = rsqrt(mean(.^2) + eps) of each:
//   ds       = d_out + r_s (d_y w_next - s r_s^2 mean(d_y w_next s));   d_state = ds
//   d_w_next = sum over rows of d_y s r_s
//   dn       = scale gate ds;   d_gate = scale n ds summed over what the gate is broadcast to
//   d_f      = r_f (dn w_post - f r_f^2 mean(dn w_post f));   d_w_post = sum over rows of dn f r_f
//
// All arithmetic is in f32; a value is rounded once, where it is stored.  The norm of s takes s as
// stored, so that the backward pass, which reads s, differentiates what the forward pass computed.
//
// Both kernels move each row once.  A group of n threads (a power of two, one thread for each two sets
// of 8 columns) holds a row; a reduction over the row is a warp butterfly and one exchange through
// shared memory, with a barrier of the group's own.
//
// The backward pass needs the mean of dn w_post f, which contains ds and with it the row's first sums.
// It is linear in them: with q = gate w_post f and gw = d_y w_next,
//   sum(q ds) = sum(q d_out) + r_s sum(q gw) - r_s^3 mean(gw s) sum(q s),
// so that one reduction of six sums serves a row.  Its time is instructions and latency rather than
// bytes: with two reductions, a CTA-wide barrier each and the weights read through the L1 that a large
// ring leaves (28 KB), 4096 rows of 4096 took 103 to 124 us.  So the weights lie in shared memory beside
// the ring, arithmetic is on pairs, and the groups of a CTA run on their own.  The weights' gradients are
// summed over a group's rows in registers, one partial row for each group goes to memory, and a second
// kernel adds the partial rows in a fixed order: no atomics, the same bits every run.
#include <string.h>

#include <type_traits>

#include "dense.h"
#include "dense_tc.cuh"
#include "dense_vec.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Sums v[0..K-1] over a group of n threads (n a power of two, >= 32), every thread getting the sums.
// `buf` holds two buffers used in turn, so one barrier a call is enough: a buffer is written again two
// calls later, with a barrier in between.  The group's threads call it together; no other group waits.
template <int K>
__device__ __forceinline__ void group_sums(float (&v)[K], int n, float *buf, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (n == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = n >> 5, first = warp & ~(per - 1);
  float *b = buf + turn * (16 * K);  // at most 16 warps
  turn ^= 1;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.x / n), "r"(n) : "memory");
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = b[(first + (lane & (per - 1))) * K + k];
  for (int o = per >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

// Eight values as four pairs: the arithmetic below takes two values an instruction.
struct Pairs {
  float2 v[4];
};
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
__device__ __forceinline__ Pairs splat(float x) { return Pairs{{pair(x), pair(x), pair(x), pair(x)}}; }
__device__ __forceinline__ Pairs mul(const Pairs &a, const Pairs &b) {
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], b.v[i]);
  return r;
}
__device__ __forceinline__ Pairs mul(const Pairs &a, float b) {
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], pair(b));
  return r;
}
// a * b + c
__device__ __forceinline__ Pairs fma(const Pairs &a, const Pairs &b, const Pairs &c) {
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
  return r;
}
__device__ __forceinline__ Pairs fma(const Pairs &a, float b, const Pairs &c) {
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], pair(b), c.v[i]);
  return r;
}
// adds the products to a running pair of sums
__device__ __forceinline__ void dot(const Pairs &a, const Pairs &b, float2 &sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = __ffma2_rn(a.v[i], b.v[i], sum);
}
__device__ __forceinline__ void add(const Pairs &a, float2 &sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = __fadd2_rn(a.v[i], sum);
}
__device__ __forceinline__ float (&flat(Pairs &p))[8] { return reinterpret_cast<float(&)[8]>(p); }
__device__ __forceinline__ const float (&flat(const Pairs &p))[8] { return reinterpret_cast<const float(&)[8]>(p); }

// Set v of a thread's columns: columns 8 (v n + t) .. + 7, or (not VEC) v 8 n + t, + n, + 2n, ...: the
// thread's place among the n kSets that Eight takes.
constexpr int kSets = 2;

template <typename T, bool VEC>
__device__ __forceinline__ Pairs load_set(const T *row, int v, int t, int n, int hidden) {
  Pairs o;
  if constexpr (VEC) load_eight<T, true>(row, v * n + t, n, hidden, flat(o));
  else load_eight<T, false>(row + v * 8 * n, t, n, hidden - v * 8 * n, flat(o));
  return o;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_set(T *row, int v, int t, int n, int hidden, const Pairs &o) {
  if constexpr (VEC) Eight<T, true>::store(row, v * n + t, n, hidden, flat(o));
  else Eight<T, false>::store(row + v * 8 * n, t, n, hidden - v * 8 * n, flat(o));
}

// the gate's values for a set of a row: its vector's, or one value for the whole row
template <typename TB, bool VEC>
__device__ __forceinline__ Pairs gate_set(const NormParams &p, int row, int gate_row, int v, int t, int n) {
  if (p.gate_kind == kGateVector) {
    const size_t at = (size_t)gate_row * p.hidden;
    if (p.gate_type == kF32) return load_set<float, VEC>(static_cast<const float *>(p.gate) + at, v, t, n, p.hidden);
    return load_set<TB, VEC>(static_cast<const TB *>(p.gate) + at, v, t, n, p.hidden);
  }
  float x = 1.f;
  if (p.gate_kind == kGateToken)
    x = p.gate_type == kF32 ? static_cast<const float *>(p.gate)[row] : to_f32(static_cast<const TB *>(p.gate)[row]);
  return splat(x);
}

// (Single values: 64 registers and 32 warps on an SM, some of them spilled, in place of 124 and 16 warps: 2000 x 4001
// bf16 39 -> 28 us, 4096 x 3001 f32 57 -> 44.)
template <typename TS, typename TB, bool VEC>
__global__ void __launch_bounds__(512, VEC ? 1 : 2) block_norm_kernel(const __grid_constant__ NormParams p, int n) {
  __shared__ float buf[2 * 16];
  const int t = threadIdx.x & (n - 1), group = threadIdx.x / n, groups = blockDim.x / n;
  const float inv = 1.f / (float)p.hidden;
  int turn = 0;
  const int step = gridDim.x * groups;
  pdl_wait();
  for (int base = blockIdx.x * groups; base < p.rows; base += step) {
    const int row = base + group;
    const bool in = row < p.rows;
    const size_t r = in ? row : 0;  // a group without a row reads the first one and stores nothing
    Pairs s[kSets];
#pragma unroll
    for (int v = 0; v < kSets; ++v)
      s[v] = load_set<TS, VEC>(static_cast<const TS *>(p.state) + r * p.ld_state, v, t, n, p.hidden);
    if (p.f) {
      Pairs f[kSets];
#pragma unroll
      for (int v = 0; v < kSets; ++v)
        f[v] = load_set<TB, VEC>(static_cast<const TB *>(p.f) + r * p.ld_f, v, t, n, p.hidden);
      float scale = p.scale;
      if (p.w_post) {
        float2 ss = pair(0.f);
#pragma unroll
        for (int v = 0; v < kSets; ++v) dot(f[v], f[v], ss);
        float sums[1] = {ss.x + ss.y};
        group_sums(sums, n, buf, turn);
        scale *= rsqrtf(fmaf(sums[0], inv, p.eps));
      }
      const int gate_row = p.gate_kind == kGateVector ? (int)r / p.rows_per_gate : 0;
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        Pairs w = gate_set<TB, VEC>(p, (int)r, gate_row, v, t, n);
        if (p.w_post) w = mul(w, load_set<float, VEC>(p.w_post, v, t, n, p.hidden));
        s[v] = fma(mul(w, scale), f[v], s[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) flat(s[v])[e] = to_f32(from_f32<TS>(flat(s[v])[e]));
        if (in) store_set<TS, VEC>(static_cast<TS *>(p.out) + r * p.ld_out, v, t, n, p.hidden, s[v]);
      }
    }
    if (p.w_next) {
      float2 ss = pair(0.f);
#pragma unroll
      for (int v = 0; v < kSets; ++v) dot(s[v], s[v], ss);
      float sums[1] = {ss.x + ss.y};
      group_sums(sums, n, buf, turn);
      const float rs = rsqrtf(fmaf(sums[0], inv, p.eps));
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        const Pairs w = load_set<float, VEC>(p.w_next, v, t, n, p.hidden);
        if (in) store_set<TB, VEC>(static_cast<TB *>(p.y) + r * p.ld_y, v, t, n, p.hidden, mul(w, mul(s[v], rs)));
      }
    }
  }
}

// writes a set of a gate row's gradient in the gate's type
template <typename TB, bool VEC>
__device__ __forceinline__ void store_gate(const NormParams &p, size_t at, int v, int t, int n, const Pairs &g) {
  if (p.gate_type == kF32)
    store_set<float, VEC>(static_cast<float *>(p.d_gate) + at, v, t, n, p.hidden, g);
  else
    store_set<TB, VEC>(static_cast<TB *>(p.d_gate) + at, v, t, n, p.hidden, g);
}

// A worker's place in its rows: row `first + i` of its lap-th chunk; end 0 after its last chunk.
struct Place {
  int lap, row, end, gate_row;
  __device__ __forceinline__ void enter(const NormParams &p, const NormBwdPlan &pl, int worker, int lap_) {
    for (lap = lap_;; ++lap) {
      const int c = lap * pl.workers + worker;
      row = end = 0;
      if (c >= pl.chunks) return;
      gate_row = c / pl.chunks_per_gate;
      row = gate_row * p.rows_per_gate + (c - gate_row * pl.chunks_per_gate) * pl.chunk_rows;
      end = min(min(row + pl.chunk_rows, (gate_row + 1) * p.rows_per_gate), p.rows);
      if (row < end) return;  // the last gate row's chunks may have no rows left
    }
  }
  __device__ __forceinline__ bool has() const { return row < end; }
  __device__ __forceinline__ void next(const NormParams &p, const NormBwdPlan &pl, int worker) {
    if (++row == end) enter(p, pl, worker, lap + 1);
  }
};

// The rows that the backward pass reads.  VEC: each thread copies its own columns of the next rows into
// its own places in shared memory (cp.async) and reads them back itself, as often as it needs them, so no
// barrier guards the ring and none of a row's values stays in registers over the reduction.  The places of
// columns past the row's end, and of what is not given, hold zeros from the start.  Otherwise the values
// are read from memory each time (the second time from the caches).
constexpr int kBwdThreads = 512;

template <typename TS, typename TB, bool VEC>
struct Rows {
  static constexpr int kS = sizeof(TS) / 2, kB = sizeof(TB) / 2;  // 16-byte pieces of a set
  static constexpr int kState = 0, kDOut = kS, kDY = 2 * kS, kF = 2 * kS + kB, kPieces = 2 * kS + 2 * kB;
  static constexpr uint32_t kPitch = kBwdThreads * 16, kRow = kSets * kPieces * kPitch;  // a row of every group
  uint32_t base;   // this thread's first piece; pieces lie kPitch bytes apart
  uint32_t stage;  // the row at work, in bytes from base
  int t, n, row;
  bool has[kSets];
  __device__ __forceinline__ void clear(int depth) const {
    for (uint32_t at = 0; at < depth * kRow; at += kPitch) sts128(base + at, make_uint4(0u, 0u, 0u, 0u));
  }
  template <typename T, int PIECE>
  __device__ __forceinline__ void copy(uint32_t st, const void *src, long long ld, int r) const {
    const T *from = static_cast<const T *>(src) + r * ld + 8 * t;
#pragma unroll
    for (int v = 0; v < kSets; ++v, from += 8 * n)
      if (has[v])
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
          if constexpr (sizeof(T) == 4)  // by way of L1: neighbouring threads' pieces share sectors
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(base + st + (v * kPieces + PIECE + k) * kPitch),
                         "l"(from + k * (16 / sizeof(T)))
                         : "memory");
          else
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + st + (v * kPieces + PIECE + k) * kPitch),
                         "l"(from + k * (16 / sizeof(T)))
                         : "memory");
  }
  __device__ __forceinline__ void fetch(const NormParams &p, uint32_t st, const Place &to) const {
    if (to.has()) {
      if (p.w_next) copy<TS, kState>(st, p.state, p.ld_state, to.row);
      if (p.d_out) copy<TS, kDOut>(st, p.d_out, p.ld_d_out, to.row);
      if (p.w_next) copy<TB, kDY>(st, p.d_y, p.ld_d_y, to.row);
      if (p.f) copy<TB, kF>(st, p.f, p.ld_f, to.row);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // a set of the row at work as it was read
  template <typename T, int PIECE>
  __device__ __forceinline__ Eight<T, VEC> get(const void *src, long long ld, int hidden, int v) const {
    Eight<T, VEC> e;
    if constexpr (VEC) {
      uint4 w[sizeof(T) / 2];
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k) w[k] = lds128(base + stage + (v * kPieces + PIECE + k) * kPitch);
      memcpy(&e, w, sizeof e);
    } else if (src) {
      e.load(static_cast<const T *>(src) + row * ld + v * 8 * n, t, n, hidden - v * 8 * n);
    } else {
      memset(&e, 0, sizeof e);
    }
    return e;
  }
  __device__ __forceinline__ Eight<TS, VEC> state(const NormParams &p, int v) const {
    return get<TS, kState>(p.w_next ? p.state : nullptr, p.ld_state, p.hidden, v);
  }
  __device__ __forceinline__ Eight<TS, VEC> d_out(const NormParams &p, int v) const {
    return get<TS, kDOut>(p.d_out, p.ld_d_out, p.hidden, v);
  }
  __device__ __forceinline__ Eight<TB, VEC> d_y(const NormParams &p, int v) const {
    return get<TB, kDY>(p.d_y, p.ld_d_y, p.hidden, v);
  }
  __device__ __forceinline__ Eight<TB, VEC> f(const NormParams &p, int v) const {
    return get<TB, kF>(p.f, p.ld_f, p.hidden, v);
  }
};
template <typename E>
__device__ __forceinline__ Pairs pairs(const E &e) {
  Pairs o;
  e.get(flat(o));
  return o;
}

// The norms' weights.  WSMEM: in shared memory, in 16-byte pieces as the threads of a group read them, zeros
// past the row's end.
template <bool VEC, bool WSMEM>
struct Weights {
  uint32_t base;  // this thread's first piece
  int t, n;
  // all loads before the first store, which nothing passes; with a gate row, w_post times it
  template <typename TB>
  __device__ __forceinline__ void fill(const NormParams &p, bool gate) const {
    if (threadIdx.x >= n) return;
    Pairs x[2][kSets], g[kSets];
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      x[0][v] = p.w_next ? load_set<float, VEC>(p.w_next, v, t, n, p.hidden) : splat(0.f);
      x[1][v] = p.w_post ? load_set<float, VEC>(p.w_post, v, t, n, p.hidden) : splat(1.f);
      if (gate) g[v] = gate_set<TB, VEC>(p, 0, 0, v, t, n);
    }
    if (gate)
#pragma unroll
      for (int v = 0; v < kSets; ++v) x[1][v] = mul(x[1][v], g[v]);
#pragma unroll
    for (int i = 0; i < 2 * kSets * 2; ++i) {
      const float2 *y = x[i / (2 * kSets)][i / 2 % kSets].v + 2 * (i & 1);
      sts128(base + i * n * 16, make_uint4(__float_as_uint(y[0].x), __float_as_uint(y[0].y), __float_as_uint(y[1].x),
                                           __float_as_uint(y[1].y)));
    }
  }
  __device__ __forceinline__ Pairs get(const float *w, int which, int hidden, float absent, int v) const {
    if constexpr (WSMEM) {
      Pairs o;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 x = lds128(base + ((which * kSets + v) * 2 + k) * n * 16);
        o.v[2 * k] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
        o.v[2 * k + 1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
      }
      return o;
    } else {
      return w ? load_set<float, VEC>(w, v, t, n, hidden) : splat(absent);
    }
  }
};

// A CTA's partial row: its groups' sums added in shared memory (the ring's, which is done with).
template <bool VEC>
__device__ __forceinline__ void store_sums(const NormParams &p, const Pairs (&a)[kSets], int n, int t, float *part) {
  extern __shared__ uint4 dyn_smem[];
  float *row = part + (size_t)blockIdx.x * p.hidden;
  if (n == kBwdThreads) {
#pragma unroll
    for (int v = 0; v < kSets; ++v) store_set<float, VEC>(row, v, t, n, p.hidden, a[v]);
    return;
  }
  float4 *sums = reinterpret_cast<float4 *>(dyn_smem);
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kSets; ++v)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      sums[(v * 2 + k) * kBwdThreads + threadIdx.x] =
          make_float4(a[v].v[2 * k].x, a[v].v[2 * k].y, a[v].v[2 * k + 1].x, a[v].v[2 * k + 1].y);
  __syncthreads();
  for (int i = threadIdx.x; i < n * kSets * 2; i += kBwdThreads) {
    const int tt = i & (n - 1), vk = i / n, v = vk >> 1, k = vk & 1;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < kBwdThreads; g += n) {
      const float4 x = sums[vk * kBwdThreads + g + tt];
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = VEC ? 8 * (v * n + tt) + 4 * k + e : (v * 8 + 4 * k + e) * n + tt;
      if (col < p.hidden) row[col] = o[e];
    }
  }
}

// TG: the type of a vector gate of several rows.  NoGate: the gate is no vector, or one row (and WSMEM),
// which lies multiplied to w_post: fewer registers and accesses to shared memory, whose pipe was 57 % busy
// (4096 x 4096, f32 stream, 67.6 -> 63.8 us; bf16 53.3 -> 47.0).
struct NoGate {};
template <typename TS, typename TB, bool VEC, bool WSMEM, typename TG>
__global__ void __launch_bounds__(kBwdThreads)
    block_norm_backward_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormBwdPlan pl) {
  using R = Rows<TS, TB, VEC>;
  constexpr bool GATEV = !std::is_same<TG, NoGate>::value;
  using GateEight = Eight<typename std::conditional<GATEV, TG, float>::type, VEC>;
  __shared__ float buf[2 * 16 * 6];
  extern __shared__ uint4 dyn_smem[];
  const int n = pl.threads, t = threadIdx.x & (n - 1), worker = threadIdx.x / n * gridDim.x + blockIdx.x;
  R rows;
  rows.base = smem_u32(dyn_smem + threadIdx.x);
  rows.t = t;
  rows.n = n;
  rows.stage = 0;
#pragma unroll
  for (int v = 0; v < kSets; ++v) rows.has[v] = 8 * (v * n + t) < p.hidden;
  Weights<VEC, WSMEM> weights;
  weights.base = smem_u32(dyn_smem) + pl.depth * R::kRow + t * 16;  // behind the ring
  weights.t = t;
  weights.n = n;
  if constexpr (VEC) rows.clear(pl.depth);
  pdl_wait();
  const float inv = 1.f / (float)p.hidden;
  int turn = 0;
  // A column's gate and weight are the same over a chunk's rows, so one sum of scale ds f r_f serves both
  // their gradients: times the gate it is w_post's, times w_post the gate's.  Without a vector gate it is
  // w_post's.  (NoGate: the sum is a_post until the end.)
  Pairs a_next[kSets], a_post[kSets], branch[kSets];
#pragma unroll
  for (int v = 0; v < kSets; ++v) a_next[v] = a_post[v] = branch[v] = splat(0.f);
  Place here, ahead;
  here.enter(p, pl, worker, 0);
  ahead = here;
  if constexpr (VEC) {
    for (int s = 0; s < pl.depth - 1; ++s) {
      rows.fetch(p, s * R::kRow, ahead);
      if (ahead.has()) ahead.next(p, pl, worker);
    }
  }
  if constexpr (WSMEM) {
    weights.template fill<TB>(p, !GATEV && p.gate_kind == kGateVector);
    __syncthreads();
  }
  // the gate's values stay in registers; a 16-bit gate's of the next chunk are fetched a row ahead
  constexpr bool kAhead = GATEV && sizeof(TG) == 2;
  GateEight gate[kSets], gate_next[kSets];
  auto load_gate = [&](GateEight &to, int gate_row, int v) {
    if constexpr (GATEV)
      to.load(static_cast<const TG *>(p.gate) + (size_t)gate_row * p.hidden + (VEC ? 0 : v * 8 * n), VEC ? v * n + t : t, n,
              VEC ? p.hidden : p.hidden - v * 8 * n);
  };
  if constexpr (GATEV) {
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      load_gate(gate[v], here.has() ? here.gate_row : 0, v);
      gate_next[v] = gate[v];
    }
  }
  const bool any = here.has();
  while (here.has()) {
    if constexpr (VEC) {
      rows.fetch(p, rows.stage == 0 ? (pl.depth - 1) * R::kRow : rows.stage - R::kRow, ahead);  // freed by the row before
      if (ahead.has()) ahead.next(p, pl, worker);
      if (pl.depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (pl.depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      rows.row = here.row;
    }
    Place after = here;
    after.next(p, pl, worker);
    if constexpr (kAhead) {
      if (after.has() && after.gate_row != here.gate_row)
#pragma unroll
        for (int v = 0; v < kSets; ++v) load_gate(gate_next[v], after.gate_row, v);
    }
    const int row = here.row;
    // a gate value of the whole row stays out of q, so that its own gradient is a sum of q ds
    const float token = p.gate_kind != kGateToken ? 1.f
                        : p.gate_type == kF32     ? static_cast<const float *>(p.gate)[row]
                                                  : to_f32(static_cast<const TB *>(p.gate)[row]);
    // Single values stay in registers from the first pass over the row to the second (4096 x 1001, no gate: 28.1
    // -> 24.5 us); from the ring they are read again (kept, 2048 x 8192 f32 spilled: 68.0 -> 73.5).
    constexpr bool KEEP = !GATEV && !VEC;
    Eight<TB, VEC> keep_f[kSets], keep_dy[kSets];
    Eight<TS, VEC> keep_do[kSets];
    float2 ss = pair(0.f), sw = pair(0.f), sf = pair(0.f), qo = pair(0.f), qg = pair(0.f), qs = pair(0.f);
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      keep_f[v] = rows.f(p, v);
      keep_dy[v] = rows.d_y(p, v);
      keep_do[v] = rows.d_out(p, v);
      const Pairs s = pairs(rows.state(p, v)), gw = mul(pairs(keep_dy[v]), weights.get(p.w_next, 0, p.hidden, 0.f, v));
      Pairs q = pairs(keep_f[v]);
      dot(s, s, ss);
      dot(gw, s, sw);
      dot(q, q, sf);
      q = mul(q, weights.get(p.w_post, 1, p.hidden, 1.f, v));
      if constexpr (GATEV) q = mul(q, pairs(gate[v]));
      dot(q, pairs(keep_do[v]), qo);
      dot(q, gw, qg);
      dot(q, s, qs);
    }
    float sums[6] = {ss.x + ss.y, sw.x + sw.y, sf.x + sf.y, qo.x + qo.y, qg.x + qg.y, qs.x + qs.y};
    group_sums(sums, n, buf, turn);
    // (rs and rf are multiplied to the sums one at a time: a cube of theirs leaves f32's range where rows of
    // 1e13 or, with a small eps, 1e-13 do not)
    const float rs = p.w_next ? rsqrtf(fmaf(sums[0], inv, p.eps)) : 0.f, cs = rs * (rs * (rs * (sums[1] * inv)));
    const float rf = p.w_post ? rsqrtf(fmaf(sums[2], inv, p.eps)) : 1.f;
    const float q_ds = fmaf(-cs, sums[5], fmaf(rs, sums[4], sums[3]));
    const float scale = p.scale * token, cf = p.w_post ? scale * (rf * (rf * (rf * (q_ds * inv)))) : 0.f;
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      if constexpr (!KEEP) {
        keep_f[v] = rows.f(p, v);
        keep_dy[v] = rows.d_y(p, v);
        keep_do[v] = rows.d_out(p, v);
      }
      const Pairs s = pairs(rows.state(p, v)), gy = mul(pairs(keep_dy[v]), rs);
      a_next[v] = fma(gy, s, a_next[v]);
      const Pairs ds = fma(s, -cs, fma(weights.get(p.w_next, 0, p.hidden, 0.f, v), gy, pairs(keep_do[v])));
      store_set<TS, VEC>(static_cast<TS *>(p.d_state) + row * p.ld_d_state, v, t, n, p.hidden, ds);
      if (p.f) {
        // nh: the normalised branch without its weight; d: the branch's gradient
        const Pairs f = pairs(keep_f[v]), nh = mul(f, rf), sd = mul(ds, scale), w = weights.get(p.w_post, 1, p.hidden, 1.f, v);
        Pairs d = sd;
        if constexpr (GATEV) {
          d = mul(sd, pairs(gate[v]));
          branch[v] = fma(sd, nh, branch[v]);
        } else {
          a_post[v] = fma(sd, nh, a_post[v]);
        }
        store_set<TB, VEC>(static_cast<TB *>(p.d_f) + row * p.ld_d_f, v, t, n, p.hidden, fma(f, -cf, mul(mul(d, w), rf)));
      }
    }
    if (p.gate_kind == kGateToken && p.d_gate && t == 0) {
      const float d = p.scale * rf * q_ds;
      if (p.gate_type == kF32)
        static_cast<float *>(p.d_gate)[row] = d;
      else
        static_cast<TB *>(p.d_gate)[row] = from_f32<TB>(d);
    }
    if constexpr (GATEV) {
      if (row + 1 == here.end) {  // the chunk's part of the gate's gradient is complete
#pragma unroll
        for (int v = 0; v < kSets; ++v) {
          a_post[v] = fma(pairs(gate[v]), branch[v], a_post[v]);
          if (p.d_gate) branch[v] = mul(branch[v], weights.get(p.w_post, 1, p.hidden, 1.f, v));
          if (pl.one_gate) continue;  // this was the worker's only chunk: stored at the end
          if (p.d_gate) {
            if (pl.chunks_per_gate == 1)
              store_gate<TB, VEC>(p, (size_t)here.gate_row * p.hidden, v, t, n, branch[v]);
            else
              store_set<float, VEC>(p.part + pl.gate_part + (size_t)(here.lap * pl.workers + worker) * p.hidden, v, t, n,
                                    p.hidden, branch[v]);
          }
          branch[v] = splat(0.f);
          if constexpr (kAhead) gate[v] = gate_next[v];
          else if (after.has()) load_gate(gate[v], after.gate_row, v);
        }
      }
    }
    here = after;
    if constexpr (VEC) rows.stage = rows.stage + R::kRow >= pl.depth * R::kRow ? 0 : rows.stage + R::kRow;
  }
  if (!GATEV && p.f && p.gate_kind == kGateVector && any) {
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      branch[v] = p.w_post ? mul(a_post[v], load_set<float, VEC>(p.w_post, v, t, n, p.hidden)) : a_post[v];
      a_post[v] = mul(a_post[v], gate_set<TB, VEC>(p, 0, 0, v, t, n));
    }
  }
  if (p.d_w_next) store_sums<VEC>(p, a_next, n, t, p.part);
  if (p.d_w_post) store_sums<VEC>(p, a_post, n, t, p.part + (size_t)(p.d_w_next ? pl.ctas : 0) * p.hidden);
  if (p.gate_kind == kGateVector && p.d_gate && pl.one_gate) store_sums<VEC>(p, branch, n, t, p.part + pl.gate_part);
}

// Adds the partial rows: job 0 and 1 the norm weights' over the CTAs, job 2 + i gate row i's over its
// chunks (a gate of one row: over the CTAs).  A CTA takes 32 columns; its warps take every kPartWarps-th
// partial row, and the first warp adds their sums in order.  (Of 32 warps, few CTAs fit on an SM: 9 us where
// these take 4.)
constexpr int kPartWarps = 8;
template <typename TB>
__global__ void __launch_bounds__(32 * kPartWarps)
    norm_partials_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormBwdPlan pl) {
  __shared__ float buf[kPartWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  pdl_wait();  // launched while the kernel that writes the partial rows runs
  for (int job = blockIdx.y; job < pl.jobs; job += gridDim.y) {
    if ((job == 0 && !p.d_w_next) || (job == 1 && !p.d_w_post)) continue;
    const float *src = p.part;
    int count = pl.ctas;
    if (job == 1) src += (size_t)(p.d_w_next ? pl.ctas : 0) * p.hidden;
    if (job == 2 && pl.one_gate) {
      src += pl.gate_part;
    } else if (job >= 2) {
      src += pl.gate_part + (size_t)(job - 2) * pl.chunks_per_gate * p.hidden;
      // the last gate row may have fewer rows than the others
      count = (min(p.rows_per_gate, p.rows - (job - 2) * p.rows_per_gate) + pl.chunk_rows - 1) / pl.chunk_rows;
    }
    float a = 0.f;
    if (col < p.hidden)
#pragma unroll 8
      for (int i = warp; i < count; i += kPartWarps) a += src[(size_t)i * p.hidden + col];
    __syncthreads();
    buf[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < p.hidden) {
      a = 0.f;
#pragma unroll
      for (int i = 0; i < kPartWarps; ++i) a += buf[i][lane];
      if (job == 0) p.d_w_next[col] = a;
      else if (job == 1) p.d_w_post[col] = a;
      else if (p.gate_type == kF32) static_cast<float *>(p.d_gate)[(size_t)(job - 2) * p.hidden + col] = a;
      else static_cast<TB *>(p.d_gate)[(size_t)(job - 2) * p.hidden + col] = from_f32<TB>(a);
    }
  }
}

int group_threads(int hidden) {
  int n = 32;
  while (n * 8 * kSets < hidden) n *= 2;
  return n;  // at most 512: kNormHiddenMax
}

size_t type_bytes(int t) { return t == kF32 ? 4 : 2; }

// a row can be read and written eight values at a time: address and row stride are multiples of their bytes
bool wide(const void *q, long long ld, int type) {
  const int bytes = 8 * (int)type_bytes(type);
  return !q || (reinterpret_cast<uintptr_t>(q) % bytes == 0 && (ld * (long long)type_bytes(type)) % bytes == 0);
}

bool all_wide(const NormParams &p) {
  if (p.hidden % 8) return false;
  return wide(p.state, p.ld_state, p.stream_type) && wide(p.f, p.ld_f, p.block_type) &&
         wide(p.out, p.ld_out, p.stream_type) && wide(p.y, p.ld_y, p.block_type) &&
         wide(p.d_out, p.ld_d_out, p.stream_type) && wide(p.d_y, p.ld_d_y, p.block_type) &&
         wide(p.d_state, p.ld_d_state, p.stream_type) && wide(p.d_f, p.ld_d_f, p.block_type) &&
         (p.gate_kind != kGateVector || (wide(p.gate, p.hidden, p.gate_type) && wide(p.d_gate, p.hidden, p.gate_type))) &&
         wide(p.w_post, 0, kF32) && wide(p.w_next, 0, kF32) && wide(p.part, 0, kF32);
}

template <typename TS, typename TB>
cudaError_t forward_typed(const NormParams &p, int num_sms, cudaStream_t st) {
  const int n = group_threads(p.hidden), threads = n < 256 ? 256 : n, groups = threads / n;
  const int blocks = (p.rows + groups - 1) / groups, most = num_sms * (1024 / threads);
  const int grid = blocks < most ? blocks : most;
  return launch_pdl(all_wide(p) ? block_norm_kernel<TS, TB, true> : block_norm_kernel<TS, TB, false>, dim3(grid),
                    dim3(threads), 0, st, p, n);
}

// The ring takes up to three rows of every group.  The weights go beside it unless that leaves less than
// two rows.
constexpr size_t kBwdSmem = 224 * 1024;

template <typename TS, typename TB, bool VEC, bool WSMEM>
cudaError_t backward_launch(const NormParams &p, NormBwdPlan pl, cudaStream_t st) {
  using R = Rows<TS, TB, VEC>;
  const size_t weights = WSMEM ? 2 * kSets * 2 * (size_t)pl.threads * 16 : 0, room = (kBwdSmem - weights) / R::kRow;
  // no more rows than a worker has
  const int most = (int)(room < 3 ? room : 3), its = (pl.chunks + pl.workers - 1) / pl.workers * pl.chunk_rows;
  pl.depth = !VEC ? 0 : its < most ? its : most;
  const size_t ring = pl.depth * (size_t)R::kRow, sums = kBwdThreads * kSets * 32;  // at the end the groups' sums
  const size_t smem = (ring > sums ? ring : sums) + weights;
  auto go = [&](auto kernel, std::atomic<unsigned long long> &done) {
    const cudaError_t e = allow_smem((const void *)kernel, kBwdSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(pl.ctas), dim3(kBwdThreads), smem, st, p, pl);
  };
  static std::atomic<unsigned long long> done[3];
  if (!p.f || p.gate_kind != kGateVector || (WSMEM && pl.one_gate)) return go(block_norm_backward_kernel<TS, TB, VEC, WSMEM, NoGate>, done[0]);
  if (p.gate_type == kF32) return go(block_norm_backward_kernel<TS, TB, VEC, WSMEM, float>, done[1]);
  return go(block_norm_backward_kernel<TS, TB, VEC, WSMEM, TB>, done[2]);
}

template <typename TS, typename TB>
cudaError_t backward_typed(const NormParams &p, int num_sms, cudaStream_t st) {
  const NormBwdPlan pl = norm_bwd_plan(p, num_sms);
  const bool beside = kBwdSmem - 2 * kSets * 2 * (size_t)pl.threads * 16 >= 2 * (size_t)Rows<TS, TB, true>::kRow;
  const cudaError_t e = !all_wide(p) ? backward_launch<TS, TB, false, true>(p, pl, st)
                        : beside     ? backward_launch<TS, TB, true, true>(p, pl, st)
                                     : backward_launch<TS, TB, true, false>(p, pl, st);
  if (e != cudaSuccess || pl.floats == 0) return e;
  const dim3 grid((p.hidden + 31) / 32, pl.jobs < 1024 ? pl.jobs : 1024);
  return launch_pdl(norm_partials_kernel<TB>, grid, dim3(32 * kPartWarps), 0, st, p, pl);
}

}  // namespace

NormBwdPlan norm_bwd_plan(const NormParams &p, int num_sms) {
  NormBwdPlan pl = {};
  pl.threads = group_threads(p.hidden);
  pl.groups = kBwdThreads / pl.threads;
  const bool gates = p.f && p.gate_kind == kGateVector;
  const int per = gates ? p.rows_per_gate : p.rows;
  const int n_gates = (p.rows + per - 1) / per;
  const int most = num_sms * pl.groups;  // one CTA for each SM
  int chunk = (int)(((long long)n_gates * per + most - 1) / most);
  pl.chunk_rows = chunk < 1 ? 1 : chunk > per ? per : chunk;
  pl.chunks_per_gate = (per + pl.chunk_rows - 1) / pl.chunk_rows;
  pl.chunks = n_gates * pl.chunks_per_gate;
  pl.ctas = pl.chunks < num_sms ? pl.chunks : num_sms;
  pl.workers = pl.ctas * pl.groups;
  const size_t norms = (p.d_w_next ? 1 : 0) + (p.d_w_post ? 1 : 0);
  pl.gate_part = norms * pl.ctas * p.hidden;
  pl.floats = pl.gate_part;
  pl.jobs = 2;
  pl.one_gate = gates && n_gates == 1 && pl.chunks <= pl.workers;
  if (gates && p.d_gate) {
    if (pl.one_gate || pl.chunks_per_gate > 1) {
      pl.floats += (size_t)(pl.one_gate ? pl.ctas : pl.chunks) * p.hidden;
      pl.jobs += n_gates;
    }
  }
  return pl;
}

cudaError_t launch_block_norm(const NormParams &p, int num_sms, cudaStream_t st) {
  if (p.stream_type == kF32) {
    if (p.block_type == kF32) return forward_typed<float, float>(p, num_sms, st);
    if (p.block_type == kBF16) return forward_typed<float, __nv_bfloat16>(p, num_sms, st);
    return forward_typed<float, __half>(p, num_sms, st);
  }
  if (p.block_type == kBF16) return forward_typed<__nv_bfloat16, __nv_bfloat16>(p, num_sms, st);
  return forward_typed<__half, __half>(p, num_sms, st);
}

cudaError_t launch_block_norm_backward(const NormParams &p, int num_sms, cudaStream_t st) {
  if (p.stream_type == kF32) {
    if (p.block_type == kF32) return backward_typed<float, float>(p, num_sms, st);
    if (p.block_type == kBF16) return backward_typed<float, __nv_bfloat16>(p, num_sms, st);
    return backward_typed<float, __half>(p, num_sms, st);
  }
  if (p.block_type == kBF16) return backward_typed<__nv_bfloat16, __nv_bfloat16>(p, num_sms, st);
  return backward_typed<__half, __half>(p, num_sms, st);
}

}  // namespace moe
