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
// shared memory.  What bounds them then is instructions and the barriers of the reductions, so a row
// takes few threads and several CTAs share an SM: one CTA of 512 threads for a row of 4096 took 114 us
// for the backward pass of 4096 rows, whatever it had in flight.  The backward pass sums the weights'
// gradients over its rows in registers, writes one partial row for each group, and a second kernel adds
// the partial rows in a fixed order: no atomics, the same bits every run.
#include <string.h>

#include "dense.h"
#include "dense_tc.cuh"
#include "dense_vec.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Sums v[0..K-1] over a group of n threads (n a power of two, >= 32), every thread getting the
// sums.  `buf` holds two buffers of kSumBuf floats used in turn, so one barrier a call is enough: a
// buffer is written again two calls later, with a barrier in between.  Every thread of the CTA must
// call it.
constexpr int kSumBuf = 32 * 3;
template <int K>
__device__ __forceinline__ void group_sums(float (&v)[K], int n, float *buf, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (n == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = n >> 5, first = warp & ~(per - 1);
  static_assert(32 * K <= kSumBuf, "sums of one call");
  float *b = buf + turn * kSumBuf;
  turn ^= 1;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = b[(first + (lane & (per - 1))) * K + k];
  for (int o = per >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

// Set v of a thread's columns: columns 8 (v n + t) .. + 7, or (not VEC) v 8 n + t, + n, + 2n, ...: the
// thread's place among the n kSets that Eight takes.
constexpr int kSets = 2;

template <typename T, bool VEC>
__device__ __forceinline__ void load_set(const T *row, int v, int t, int n, int hidden, float (&o)[8]) {
  if constexpr (VEC) load_eight<T, true>(row, v * n + t, n, hidden, o);
  else load_eight<T, false>(row + v * 8 * n, t, n, hidden - v * 8 * n, o);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_set(T *row, int v, int t, int n, int hidden, const float (&o)[8]) {
  if constexpr (VEC) Eight<T, true>::store(row, v * n + t, n, hidden, o);
  else Eight<T, false>::store(row + v * 8 * n, t, n, hidden - v * 8 * n, o);
}

// the gate's values for a set of a row: its vector's, or one value for the whole row
template <typename TB, bool VEC>
__device__ __forceinline__ void gate_set(const NormParams &p, int row, int v, int t, int n, float (&g)[8]) {
  if (p.gate_kind == kGateVector) {
    const size_t at = (size_t)(row / p.rows_per_gate) * p.hidden;
    if (p.gate_type == kF32)
      load_set<float, VEC>(static_cast<const float *>(p.gate) + at, v, t, n, p.hidden, g);
    else
      load_set<TB, VEC>(static_cast<const TB *>(p.gate) + at, v, t, n, p.hidden, g);
  } else {
    float x = 1.f;
    if (p.gate_kind == kGateToken)
      x = p.gate_type == kF32 ? static_cast<const float *>(p.gate)[row] : to_f32(static_cast<const TB *>(p.gate)[row]);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = x;
  }
}

template <typename TS, typename TB, bool VEC>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ NormParams p, int n) {
  __shared__ float buf[2 * kSumBuf];
  const int t = threadIdx.x & (n - 1), group = threadIdx.x / n, groups = blockDim.x / n;
  const float inv = 1.f / (float)p.hidden;
  int turn = 0;
  const int step = gridDim.x * groups;
  for (int base = blockIdx.x * groups; base < p.rows; base += step) {
    const int row = base + group;
    const bool in = row < p.rows;
    const size_t r = in ? row : 0;  // a group without a row reads the first one and stores nothing
    float s[kSets][8];
#pragma unroll
    for (int v = 0; v < kSets; ++v)
      load_set<TS, VEC>(static_cast<const TS *>(p.state) + r * p.ld_state, v, t, n, p.hidden, s[v]);
    if (p.f) {
      float f[kSets][8];
#pragma unroll
      for (int v = 0; v < kSets; ++v)
        load_set<TB, VEC>(static_cast<const TB *>(p.f) + r * p.ld_f, v, t, n, p.hidden, f[v]);
      float scale = p.scale;
      if (p.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kSets; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) ss[0] = fmaf(f[v][e], f[v][e], ss[0]);
        group_sums(ss, n, buf, turn);
        scale *= rsqrtf(fmaf(ss[0], inv, p.eps));
      }
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        float w[8];
        gate_set<TB, VEC>(p, (int)r, v, t, n, w);
        if (p.w_post) {
          float wp[8];
          load_set<float, VEC>(p.w_post, v, t, n, p.hidden, wp);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= wp[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s[v][e] = to_f32(from_f32<TS>(fmaf(scale * w[e], f[v][e], s[v][e])));
        if (in) store_set<TS, VEC>(static_cast<TS *>(p.out) + r * p.ld_out, v, t, n, p.hidden, s[v]);
      }
    }
    if (p.w_next) {
      float ss[1] = {0.f};
#pragma unroll
      for (int v = 0; v < kSets; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(s[v][e], s[v][e], ss[0]);
      group_sums(ss, n, buf, turn);
      const float rs = rsqrtf(fmaf(ss[0], inv, p.eps));
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        float w[8];
        load_set<float, VEC>(p.w_next, v, t, n, p.hidden, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= s[v][e] * rs;
        if (in) store_set<TB, VEC>(static_cast<TB *>(p.y) + r * p.ld_y, v, t, n, p.hidden, w);
      }
    }
  }
}

// writes a set of a gate row's gradient in the gate's type
template <typename TB, bool VEC>
__device__ __forceinline__ void store_gate(const NormParams &p, size_t at, int v, int t, int n, const float (&g)[8]) {
  if (p.gate_type == kF32)
    store_set<float, VEC>(static_cast<float *>(p.d_gate) + at, v, t, n, p.hidden, g);
  else
    store_set<TB, VEC>(static_cast<TB *>(p.d_gate) + at, v, t, n, p.hidden, g);
}

// A worker's place in its rows: row `first + i` of its lap-th chunk, while that is below `end` (the last
// chunk of a gate row may be shorter, and a worker's last lap may have none).
struct Place {
  int lap, i, first, end, gate_row;
  __device__ __forceinline__ void enter(const NormParams &p, const NormBwdPlan &pl, int worker, int lap_) {
    lap = lap_;
    i = 0;
    const int c = lap * pl.workers + worker;
    gate_row = c / pl.chunks_per_gate;
    first = gate_row * p.rows_per_gate + (c - gate_row * pl.chunks_per_gate) * pl.chunk_rows;
    end = c < pl.chunks ? min((gate_row + 1) * p.rows_per_gate, p.rows) : 0;
  }
  __device__ __forceinline__ void next(const NormParams &p, const NormBwdPlan &pl, int worker) {
    if (++i == pl.chunk_rows) enter(p, pl, worker, lap + 1);
  }
  __device__ __forceinline__ int row() const { return first + i < end ? first + i : -1; }
};

// The rows that the backward pass reads.  VEC: each thread copies its own columns of the next DEPTH - 1
// rows into its own places in shared memory (cp.async) and reads them back itself, as often as it needs
// them, so no barrier guards the ring and few of a row's values have to stay in registers.  Otherwise
// the values are read from memory each time (the second time from the caches).
template <typename TS, typename TB, bool VEC, int DEPTH>
struct Rows {
  static constexpr int kS = sizeof(TS) / 2, kB = sizeof(TB) / 2;  // 16-byte pieces of a set
  static constexpr int kState = 0, kDOut = kS, kDY = 2 * kS, kF = 2 * kS + kB, kPieces = 2 * kS + 2 * kB;
  uint32_t base;  // this thread's first piece; pieces lie blockDim.x * 16 bytes apart
  int t, n, stage, row;
  __device__ __forceinline__ uint32_t at(int st, int v, int piece) const {
    return base + (uint32_t)((st * kSets + v) * kPieces + piece) * blockDim.x * 16u;
  }
  template <typename T>
  __device__ __forceinline__ void copy(int st, int v, int piece, const T *src) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(st, v, piece + k)), "l"(src + k * (16 / sizeof(T)))
                   : "memory");
  }
  __device__ __forceinline__ void fetch(const NormParams &p, int st, int r) const {
    if (r >= 0)
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        const int col = 8 * (v * n + t);
        if (col < p.hidden) {
          if (p.w_next) copy(st, v, kState, static_cast<const TS *>(p.state) + r * p.ld_state + col);
          if (p.d_out) copy(st, v, kDOut, static_cast<const TS *>(p.d_out) + r * p.ld_d_out + col);
          if (p.w_next) copy(st, v, kDY, static_cast<const TB *>(p.d_y) + r * p.ld_d_y + col);
          if (p.f) copy(st, v, kF, static_cast<const TB *>(p.f) + r * p.ld_f + col);
        }
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // set v of the row at work; zeros past the row's end
  template <typename T, int PIECE>
  __device__ __forceinline__ void get(const NormParams &p, const void *src, long long ld, int v, float (&o)[8]) const {
    if constexpr (VEC) {
      if (8 * (v * n + t) < p.hidden) {
        Eight<T, true> e;
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[k].x), "=r"(w[k].y), "=r"(w[k].z), "=r"(w[k].w)
                       : "r"(at(stage, v, PIECE + k))
                       : "memory");
        memcpy(&e, w, sizeof e);
        e.get(o);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
      }
    } else {
      load_set<T, false>(static_cast<const T *>(src) + row * ld, v, t, n, p.hidden, o);
    }
  }
};

// Rows of the ring: what lets two CTAs of up to 256 threads, or one of 512, stay on an SM; 0: no ring.
template <typename TS, typename TB>
constexpr int kRingFit = 208 * 1024 / (512 * 16 * kSets * (int)(sizeof(TS) + sizeof(TB)));
template <typename TS, typename TB, bool VEC>
constexpr int kRingDepth = !VEC ? 0 : kRingFit<TS, TB> < 3 ? kRingFit<TS, TB> : 3;

template <typename TS, typename TB, bool VEC>
__global__ void __launch_bounds__(512)
    block_norm_backward_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormBwdPlan pl) {
  constexpr int DEPTH = kRingDepth<TS, TB, VEC>;
  using R = Rows<TS, TB, VEC, DEPTH>;
  __shared__ float buf[2 * kSumBuf];
  extern __shared__ uint4 ring_smem[];
  const int n = pl.threads, t = threadIdx.x & (n - 1), group = threadIdx.x / n;
  const int worker = blockIdx.x * pl.groups + group;
  R rows;
  rows.base = smem_u32(ring_smem + threadIdx.x);
  rows.t = t;
  rows.n = n;
  rows.stage = 0;
  const float inv = 1.f / (float)p.hidden;
  const bool gates = p.gate_kind == kGateVector && p.d_gate, token = p.gate_kind == kGateToken && p.d_gate;
  int turn = 0;
  float a_next[kSets][8], a_post[kSets][8], a_gate[kSets][8];
#pragma unroll
  for (int v = 0; v < kSets; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) a_next[v][e] = a_post[v][e] = a_gate[v][e] = 0.f;
  // the same number of steps for every thread of the grid: the reductions are CTA-wide
  const int steps = (pl.chunks + pl.workers - 1) / pl.workers * pl.chunk_rows;
  Place here, ahead;
  here.enter(p, pl, worker, 0);
  ahead.enter(p, pl, worker, 0);
  if constexpr (VEC)
    for (int s = 0; s < DEPTH - 1; ++s, ahead.next(p, pl, worker)) rows.fetch(p, s, s < steps ? ahead.row() : -1);
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const int row = here.row();
    const bool in = row >= 0;
    if constexpr (VEC) {
      // into the stage that the step before freed
      rows.fetch(p, rows.stage == 0 ? DEPTH - 1 : rows.stage - 1, step + DEPTH - 1 < steps ? ahead.row() : -1);
      ahead.next(p, pl, worker);
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH > 0 ? DEPTH - 1 : 0) : "memory");
    } else {
      rows.row = in ? row : 0;
    }
    // A group without a row this time works on what it finds and keeps nothing of it: its sums are its
    // own.
    float sums[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      if (p.w_next) {
        float s[8], gy[8], w[8];
        rows.template get<TS, R::kState>(p, p.state, p.ld_state, v, s);
        rows.template get<TB, R::kDY>(p, p.d_y, p.ld_d_y, v, gy);
        load_set<float, VEC>(p.w_next, v, t, n, p.hidden, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sums[0] = fmaf(s[e], s[e], sums[0]);
          sums[1] = fmaf(w[e] * gy[e], s[e], sums[1]);
        }
      }
      if (p.w_post) {
        float f[8];
        rows.template get<TB, R::kF>(p, p.f, p.ld_f, v, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[2] = fmaf(f[e], f[e], sums[2]);
      }
    }
    if (p.w_next || p.w_post) group_sums(sums, n, buf, turn);
    const float rs = rsqrtf(fmaf(sums[0], inv, p.eps)), cs = rs * rs * (sums[1] * inv);
    const float rf = p.w_post ? rsqrtf(fmaf(sums[2], inv, p.eps)) : 1.f;
    float two[2] = {0.f, 0.f};
    float dn[kSets][8];
#pragma unroll
    for (int v = 0; v < kSets; ++v) {
      float ds[8];
      if (p.d_out) rows.template get<TS, R::kDOut>(p, p.d_out, p.ld_d_out, v, ds);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) ds[e] = 0.f;
      if (p.w_next) {
        float s[8], gy[8], w[8];
        rows.template get<TS, R::kState>(p, p.state, p.ld_state, v, s);
        rows.template get<TB, R::kDY>(p, p.d_y, p.ld_d_y, v, gy);
        load_set<float, VEC>(p.w_next, v, t, n, p.hidden, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (in) a_next[v][e] = fmaf(gy[e], s[e] * rs, a_next[v][e]);
          ds[e] = fmaf(rs, fmaf(-s[e], cs, w[e] * gy[e]), ds[e]);
        }
      }
      if (in) store_set<TS, VEC>(static_cast<TS *>(p.d_state) + row * p.ld_d_state, v, t, n, p.hidden, ds);
      if (p.f) {
        float f[8], g[8], w[8];
        rows.template get<TB, R::kF>(p, p.f, p.ld_f, v, f);
        gate_set<TB, VEC>(p, in ? row : 0, v, t, n, g);
        if (p.w_post) load_set<float, VEC>(p.w_post, v, t, n, p.hidden, w);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float sd = p.scale * ds[e], nh = f[e] * rf;  // nh: the normalised branch without its weight
          const float gn = sd * nh * w[e], d = sd * g[e];    // the gate's gradient, and the branch's
          if (in) {
            a_gate[v][e] += gn;
            a_post[v][e] = fmaf(d, nh, a_post[v][e]);
          }
          dn[v][e] = d * w[e];
          two[0] = fmaf(dn[v][e], f[e], two[0]);
          two[1] += gn;
        }
      }
    }
    if (p.f) {
      if (p.w_post || token) group_sums(two, n, buf, turn);
      const float cf = p.w_post ? rf * rf * (two[0] * inv) : 0.f;
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        float f[8];
        rows.template get<TB, R::kF>(p, p.f, p.ld_f, v, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = p.w_post ? rf * fmaf(-f[e], cf, dn[v][e]) : dn[v][e];
        if (in) store_set<TB, VEC>(static_cast<TB *>(p.d_f) + row * p.ld_d_f, v, t, n, p.hidden, f);
      }
      if (in && token && t == 0) {
        if (p.gate_type == kF32)
          static_cast<float *>(p.d_gate)[row] = two[1];
        else
          static_cast<TB *>(p.d_gate)[row] = from_f32<TB>(two[1]);
      }
    }
    if (gates && here.i == pl.chunk_rows - 1) {  // the chunk's part of the gate's gradient is complete
      const int chunk = here.lap * pl.workers + worker;
#pragma unroll
      for (int v = 0; v < kSets; ++v) {
        if (chunk < pl.chunks) {
          if (pl.chunks_per_gate == 1)
            store_gate<TB, VEC>(p, (size_t)here.gate_row * p.hidden, v, t, n, a_gate[v]);
          else
            store_set<float, VEC>(p.part + pl.gate_part + (size_t)chunk * p.hidden, v, t, n, p.hidden, a_gate[v]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) a_gate[v][e] = 0.f;
      }
    }
    here.next(p, pl, worker);
    rows.stage = rows.stage + 1 >= DEPTH ? 0 : rows.stage + 1;
  }
#pragma unroll
  for (int v = 0; v < kSets; ++v) {
    if (p.d_w_next) store_set<float, VEC>(p.part + (size_t)worker * p.hidden, v, t, n, p.hidden, a_next[v]);
    if (p.d_w_post)
      store_set<float, VEC>(p.part + ((size_t)(p.d_w_next ? pl.workers : 0) + worker) * p.hidden, v, t, n, p.hidden,
                            a_post[v]);
  }
}

// Adds the partial rows: job 0 and 1 the norm weights' over the workers, job 2 + i gate row i's over
// its chunks.  A CTA takes 32 columns; its 32 warps take every 32nd partial row, and the first warp
// adds their 32 sums in order.
template <typename TB>
__global__ void __launch_bounds__(1024)
    norm_partials_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormBwdPlan pl) {
  __shared__ float buf[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  for (int job = blockIdx.y; job < 2 + (pl.floats > pl.gate_part ? pl.chunks / pl.chunks_per_gate : 0); job += gridDim.y) {
    if ((job == 0 && !p.d_w_next) || (job == 1 && !p.d_w_post)) continue;
    const float *src = p.part;
    int count = pl.workers;
    if (job == 1) src += (size_t)(p.d_w_next ? pl.workers : 0) * p.hidden;
    if (job >= 2) {
      src += pl.gate_part + (size_t)(job - 2) * pl.chunks_per_gate * p.hidden;
      count = pl.chunks_per_gate;
    }
    float a = 0.f;
    if (col < p.hidden)
      for (int i = warp; i < count; i += 32) a += src[(size_t)i * p.hidden + col];
    __syncthreads();
    buf[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < p.hidden) {
      a = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) a += buf[i][lane];
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

// a row can be read and written in 16-byte pieces: address and row stride are multiples of 16 bytes
bool wide(const void *q, long long ld, int type) {
  return !q || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && (ld * (long long)type_bytes(type)) % 16 == 0);
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
  if (all_wide(p))
    block_norm_kernel<TS, TB, true><<<grid, threads, 0, st>>>(p, n);
  else
    block_norm_kernel<TS, TB, false><<<grid, threads, 0, st>>>(p, n);
  return cudaGetLastError();
}

template <typename TS, typename TB, bool VEC>
cudaError_t backward_launch(const NormParams &p, const NormBwdPlan &pl, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const int threads = pl.threads * pl.groups;
  const size_t per_thread = (size_t)kRingDepth<TS, TB, VEC> * kSets * (sizeof(TS) + sizeof(TB)) * 16;
  const cudaError_t e = allow_smem((const void *)block_norm_backward_kernel<TS, TB, VEC>, per_thread * 512, done);
  if (e != cudaSuccess) return e;
  block_norm_backward_kernel<TS, TB, VEC><<<pl.ctas, threads, per_thread * threads, st>>>(p, pl);
  return cudaGetLastError();
}

template <typename TS, typename TB>
cudaError_t backward_typed(const NormParams &p, int num_sms, cudaStream_t st) {
  const NormBwdPlan pl = norm_bwd_plan(p, num_sms);
  const cudaError_t e = all_wide(p) ? backward_launch<TS, TB, true>(p, pl, st) : backward_launch<TS, TB, false>(p, pl, st);
  if (e != cudaSuccess || pl.floats == 0) return e;
  const int jobs = 2 + (pl.floats > pl.gate_part ? pl.chunks / pl.chunks_per_gate : 0);
  const dim3 grid((p.hidden + 31) / 32, jobs < 1024 ? jobs : 1024);
  norm_partials_kernel<TB><<<grid, 1024, 0, st>>>(p, pl);
  return cudaGetLastError();
}

}  // namespace

NormBwdPlan norm_bwd_plan(const NormParams &p, int num_sms) {
  NormBwdPlan pl = {};
  pl.threads = group_threads(p.hidden);
  const int threads = pl.threads < 256 ? 256 : pl.threads;
  pl.groups = threads / pl.threads;
  const bool gates = p.f && p.gate_kind == kGateVector;
  const int per = gates ? p.rows_per_gate : p.rows;
  const int n_gates = (p.rows + per - 1) / per;
  // two CTAs of 256 threads for each SM, or one of 512
  const int most = num_sms * (threads <= 256 ? 2 : 1) * pl.groups;
  int chunk = (int)(((long long)n_gates * per + most - 1) / most);
  pl.chunk_rows = chunk < 1 ? 1 : chunk > per ? per : chunk;
  pl.chunks_per_gate = (per + pl.chunk_rows - 1) / pl.chunk_rows;
  pl.chunks = n_gates * pl.chunks_per_gate;
  const int workers = pl.chunks < most ? pl.chunks : most;
  pl.ctas = (workers + pl.groups - 1) / pl.groups;
  pl.workers = pl.ctas * pl.groups;
  const size_t norms = (p.d_w_next ? 1 : 0) + (p.d_w_post ? 1 : 0);
  pl.gate_part = norms * pl.workers * p.hidden;
  pl.floats = pl.gate_part;
  if (gates && p.d_gate && pl.chunks_per_gate > 1) pl.floats += (size_t)pl.chunks * p.hidden;
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
