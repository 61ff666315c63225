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
// Both kernels are bound by memory: each row is read once into registers and written once.  A
// group of n threads (a power of two, one thread for each 8 columns) holds a row; a reduction over
// the row is a warp butterfly and one exchange through shared memory.  The backward pass sums the
// weights' gradients over its rows in registers, writes one partial row for each group, and a
// second kernel adds the partial rows in a fixed order: no atomics, the same bits every run.
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
  for (int k = 0; k < K; ++k) {
    v[k] = lane < per ? b[(first + lane) * K + k] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
}

// the gate's eight values for a row: its vector, or one value for the whole row
template <typename TB, bool VEC>
__device__ __forceinline__ void gate_eight(const NormParams &p, int row, int t, int n, float (&g)[8]) {
  if (p.gate_kind == kGateVector) {
    const size_t at = (size_t)(row / p.rows_per_gate) * p.hidden;
    if (p.gate_type == kF32)
      load_eight<float, VEC>(static_cast<const float *>(p.gate) + at, t, n, p.hidden, g);
    else
      load_eight<TB, VEC>(static_cast<const TB *>(p.gate) + at, t, n, p.hidden, g);
  } else {
    float v = 1.f;
    if (p.gate_kind == kGateToken)
      v = p.gate_type == kF32 ? static_cast<const float *>(p.gate)[row] : to_f32(static_cast<const TB *>(p.gate)[row]);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = v;
  }
}

template <typename TS, typename TB, bool VEC>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormParams p, int n) {
  __shared__ float buf[2 * kSumBuf];
  const int t = threadIdx.x & (n - 1), group = threadIdx.x / n, groups = blockDim.x / n;
  const float inv = 1.f / (float)p.hidden;
  int turn = 0;
  const int step = gridDim.x * groups;
  for (int base = blockIdx.x * groups; base < p.rows; base += step) {
    const int row = base + group;
    const bool in = row < p.rows;
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    if (in) load_eight<TS, VEC>(static_cast<const TS *>(p.state) + row * p.ld_state, t, n, p.hidden, s);
    if (p.f) {
      float f[8], g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = g[e] = 0.f;
      if (in) {
        load_eight<TB, VEC>(static_cast<const TB *>(p.f) + row * p.ld_f, t, n, p.hidden, f);
        gate_eight<TB, VEC>(p, row, t, n, g);
      }
      if (p.w_post) {
        float w[8], ss[1] = {0.f};
        load_eight<float, VEC>(p.w_post, t, n, p.hidden, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(f[e], f[e], ss[0]);
        group_sums(ss, n, buf, turn);
        const float r = rsqrtf(fmaf(ss[0], inv, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= r * w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = to_f32(from_f32<TS>(fmaf(p.scale * g[e], f[e], s[e])));
      if (in) Eight<TS, VEC>::store(static_cast<TS *>(p.out) + row * p.ld_out, t, n, p.hidden, s);
    }
    if (p.w_next) {
      float w[8], ss[1] = {0.f};
      load_eight<float, VEC>(p.w_next, t, n, p.hidden, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[0] = fmaf(s[e], s[e], ss[0]);
      group_sums(ss, n, buf, turn);
      const float r = rsqrtf(fmaf(ss[0], inv, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] *= r * w[e];
      if (in) Eight<TB, VEC>::store(static_cast<TB *>(p.y) + row * p.ld_y, t, n, p.hidden, s);
    }
  }
}

// writes a gate row's gradient in the gate's type
template <typename TB, bool VEC>
__device__ __forceinline__ void store_gate(const NormParams &p, size_t at, int t, int n, const float (&v)[8]) {
  if (p.gate_type == kF32)
    Eight<float, VEC>::store(static_cast<float *>(p.d_gate) + at, t, n, p.hidden, v);
  else
    Eight<TB, VEC>::store(static_cast<TB *>(p.d_gate) + at, t, n, p.hidden, v);
}

// A worker's place in its rows: row i of the lap-th of its chunks.
struct Place {
  int lap = 0, i = 0;
  __device__ __forceinline__ void next(const NormBwdPlan &pl) {
    if (++i == pl.chunk_rows) {
      i = 0;
      ++lap;
    }
  }
  __device__ __forceinline__ int chunk(const NormBwdPlan &pl, int worker) const { return lap * pl.workers + worker; }
  // the row, or -1 where the chunk (the last of a gate row may be shorter) has none
  __device__ __forceinline__ int row(const NormParams &p, const NormBwdPlan &pl, int worker) const {
    const int c = chunk(pl, worker);
    if (c >= pl.chunks) return -1;
    const int gate_row = c / pl.chunks_per_gate;
    const int r = gate_row * p.rows_per_gate + (c % pl.chunks_per_gate) * pl.chunk_rows + i;
    return r < min((gate_row + 1) * p.rows_per_gate, p.rows) ? r : -1;
  }
};

// Rows on their way: each thread copies its own columns of the next DEPTH - 1 rows into its own places in
// shared memory (cp.async) and reads them back itself, so no barrier guards the ring.
template <typename TS, typename TB, int DEPTH>
struct RowRing {
  static constexpr int kS = sizeof(TS) / 2, kB = sizeof(TB) / 2;  // 16-byte pieces of eight values
  static constexpr int kPieces = 2 * kS + 2 * kB;                 // state, d_out, d_y, f: sizeof(TS) + sizeof(TB)
  uint32_t base;  // this thread's first piece; pieces lie blockDim.x * 16 bytes apart
  __device__ __forceinline__ uint32_t at(int stage, int piece) const {
    return base + (uint32_t)(stage * kPieces + piece) * blockDim.x * 16u;
  }
  template <typename T>
  __device__ __forceinline__ void copy(int stage, int piece, const T *src) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(stage, piece + k)), "l"(src + k * (16 / sizeof(T)))
                   : "memory");
  }
  template <typename T>
  __device__ __forceinline__ void get(int stage, int piece, float (&v)[8]) const {
    Eight<T, true> e;
    uint4 w[sizeof(T) / 2];
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[k].x), "=r"(w[k].y), "=r"(w[k].z), "=r"(w[k].w)
                   : "r"(at(stage, piece + k))
                   : "memory");
    memcpy(&e, w, sizeof e);
    e.get(v);
  }
  __device__ __forceinline__ void fetch(const NormParams &p, int stage, int row, int t) const {
    if (row >= 0 && 8 * t < p.hidden) {
      if (p.w_next) copy(stage, 0, static_cast<const TS *>(p.state) + row * p.ld_state + 8 * t);
      if (p.d_out) copy(stage, kS, static_cast<const TS *>(p.d_out) + row * p.ld_d_out + 8 * t);
      if (p.w_next) copy(stage, 2 * kS, static_cast<const TB *>(p.d_y) + row * p.ld_d_y + 8 * t);
      if (p.f) copy(stage, 2 * kS + kB, static_cast<const TB *>(p.f) + row * p.ld_f + 8 * t);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// Rows in flight in the ring: three, or what a CTA's shared memory holds at 1024 threads; 0: no ring.
template <typename TS, typename TB, int MAXT>
constexpr int kRingFit = 220 * 1024 / (MAXT * 16 * (int)(sizeof(TS) + sizeof(TB)));
template <typename TS, typename TB, bool VEC, int MAXT>
constexpr int kRingDepth = !VEC ? 0 : kRingFit<TS, TB, MAXT> < 3 ? kRingFit<TS, TB, MAXT> : 3;

template <typename TS, typename TB, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT)
    block_norm_backward_kernel(const __grid_constant__ NormParams p, const __grid_constant__ NormBwdPlan pl) {
  constexpr int DEPTH = kRingDepth<TS, TB, VEC, MAXT>;
  __shared__ float buf[2 * kSumBuf];
  extern __shared__ uint4 ring_smem[];
  RowRing<TS, TB, DEPTH> ring;
  ring.base = smem_u32(ring_smem + threadIdx.x);
  const int n = pl.threads, t = threadIdx.x & (n - 1), group = threadIdx.x / n;
  const int worker = blockIdx.x * pl.groups + group;
  const float inv = 1.f / (float)p.hidden;
  const bool there = VEC ? 8 * t < p.hidden : true;
  int turn = 0;
  float a_next[8], a_post[8], a_gate[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) a_next[e] = a_post[e] = a_gate[e] = 0.f;
  // the same number of steps for every thread of the grid: the reductions are CTA-wide
  const int steps = (pl.chunks + pl.workers - 1) / pl.workers * pl.chunk_rows;
  Place here, ahead;
  if constexpr (VEC)
    for (int s = 0; s < DEPTH - 1; ++s, ahead.next(pl)) ring.fetch(p, s, s < steps ? ahead.row(p, pl, worker) : -1, t);
  int stage = 0;
  for (int step = 0; step < steps; ++step, here.next(pl)) {
    const int row = here.row(p, pl, worker);
    const bool in = row >= 0;
    float ds[8], s[8], gy[8], f[8], g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) ds[e] = s[e] = gy[e] = f[e] = g[e] = 0.f;
    if constexpr (VEC) {
      const int put = stage == 0 ? DEPTH - 1 : stage - 1;  // the stage that the step before freed
      ring.fetch(p, put, step + DEPTH - 1 < steps ? ahead.row(p, pl, worker) : -1, t);
      ahead.next(pl);
      if (in && p.f) gate_eight<TB, VEC>(p, row, t, n, g);
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
      if (in && there) {
        if (p.d_out) ring.template get<TS>(stage, ring.kS, ds);
        if (p.w_next) {
          ring.template get<TS>(stage, 0, s);
          ring.template get<TB>(stage, 2 * ring.kS, gy);
        }
        if (p.f) ring.template get<TB>(stage, 2 * ring.kS + ring.kB, f);
      }
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
    } else if (in) {
      if (p.d_out) load_eight<TS, VEC>(static_cast<const TS *>(p.d_out) + row * p.ld_d_out, t, n, p.hidden, ds);
      if (p.w_next) {
        load_eight<TS, VEC>(static_cast<const TS *>(p.state) + row * p.ld_state, t, n, p.hidden, s);
        load_eight<TB, VEC>(static_cast<const TB *>(p.d_y) + row * p.ld_d_y, t, n, p.hidden, gy);
      }
      if (p.f) {
        load_eight<TB, VEC>(static_cast<const TB *>(p.f) + row * p.ld_f, t, n, p.hidden, f);
        gate_eight<TB, VEC>(p, row, t, n, g);
      }
    }
    float w[8], sums[3] = {0.f, 0.f, 0.f};
    if (p.w_next) load_eight<float, VEC>(p.w_next, t, n, p.hidden, w);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] *= gy[e];
      sums[0] = fmaf(s[e], s[e], sums[0]);
      sums[1] = fmaf(w[e], s[e], sums[1]);
      sums[2] = fmaf(f[e], f[e], sums[2]);
    }
    group_sums(sums, n, buf, turn);
    const float rf = p.w_post ? rsqrtf(fmaf(sums[2], inv, p.eps)) : 1.f;
    if (p.w_next) {
      const float rs = rsqrtf(fmaf(sums[0], inv, p.eps)), c = rs * rs * (sums[1] * inv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a_next[e] = fmaf(gy[e], s[e] * rs, a_next[e]);
        ds[e] = fmaf(rs, fmaf(-s[e], c, w[e]), ds[e]);
      }
    }
    if (in) Eight<TS, VEC>::store(static_cast<TS *>(p.d_state) + row * p.ld_d_state, t, n, p.hidden, ds);
    if (p.f) {
      if (p.w_post) load_eight<float, VEC>(p.w_post, t, n, p.hidden, w);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
      float two[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float nh = f[e] * rf;                // the normalised branch without its weight
        const float sd = p.scale * ds[e];
        const float gn = sd * nh * w[e];           // the gate's gradient
        const float dn = sd * g[e];
        a_gate[e] += gn;
        a_post[e] = fmaf(dn, nh, a_post[e]);
        g[e] = dn * w[e];
        two[0] = fmaf(g[e], f[e], two[0]);
        two[1] += gn;
      }
      if (p.w_post || (p.gate_kind == kGateToken && p.d_gate)) group_sums(two, n, buf, turn);
      if (p.w_post) {
        const float c = rf * rf * (two[0] * inv);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = rf * fmaf(-f[e], c, g[e]);
      }
      if (in) {
        Eight<TB, VEC>::store(static_cast<TB *>(p.d_f) + row * p.ld_d_f, t, n, p.hidden, g);
        if (p.gate_kind == kGateToken && p.d_gate && t == 0) {
          if (p.gate_type == kF32)
            static_cast<float *>(p.d_gate)[row] = two[1];
          else
            static_cast<TB *>(p.d_gate)[row] = from_f32<TB>(two[1]);
        }
      }
    }
    if (here.i == pl.chunk_rows - 1) {  // the chunk's part of the gate's gradient is complete
      const int chunk = here.chunk(pl, worker);
      if (p.gate_kind == kGateVector && p.d_gate && chunk < pl.chunks) {
        if (pl.chunks_per_gate == 1)
          store_gate<TB, VEC>(p, (size_t)(chunk / pl.chunks_per_gate) * p.hidden, t, n, a_gate);
        else
          Eight<float, VEC>::store(p.part + pl.gate_part + (size_t)chunk * p.hidden, t, n, p.hidden, a_gate);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) a_gate[e] = 0.f;
    }
  }
  if (p.d_w_next) Eight<float, VEC>::store(p.part + (size_t)worker * p.hidden, t, n, p.hidden, a_next);
  if (p.d_w_post)
    Eight<float, VEC>::store(p.part + ((size_t)(p.d_w_next ? pl.workers : 0) + worker) * p.hidden, t, n, p.hidden, a_post);
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
  while (n * 8 < hidden) n *= 2;
  return n;
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
  const int blocks = (p.rows + groups - 1) / groups, most = num_sms * (2048 / threads);
  const int grid = blocks < most ? blocks : most;
  if (all_wide(p))
    block_norm_kernel<TS, TB, true><<<grid, threads, 0, st>>>(p, n);
  else
    block_norm_kernel<TS, TB, false><<<grid, threads, 0, st>>>(p, n);
  return cudaGetLastError();
}

template <typename TS, typename TB, bool VEC, int MAXT>
cudaError_t backward_launch(const NormParams &p, const NormBwdPlan &pl, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const int threads = pl.threads * pl.groups;
  const size_t per_thread = (size_t)kRingDepth<TS, TB, VEC, MAXT> * (sizeof(TS) + sizeof(TB)) * 16;
  const cudaError_t e =
      allow_smem((const void *)block_norm_backward_kernel<TS, TB, VEC, MAXT>, per_thread * MAXT, done);
  if (e != cudaSuccess) return e;
  block_norm_backward_kernel<TS, TB, VEC, MAXT><<<pl.ctas, threads, per_thread * threads, st>>>(p, pl);
  return cudaGetLastError();
}

template <typename TS, typename TB>
cudaError_t backward_typed(const NormParams &p, int num_sms, cudaStream_t st) {
  const NormBwdPlan pl = norm_bwd_plan(p, num_sms);
  const int threads = pl.threads * pl.groups;
  cudaError_t e;
  if (all_wide(p)) e = threads <= 512 ? backward_launch<TS, TB, true, 512>(p, pl, st) : backward_launch<TS, TB, true, 1024>(p, pl, st);
  else e = threads <= 512 ? backward_launch<TS, TB, false, 512>(p, pl, st) : backward_launch<TS, TB, false, 1024>(p, pl, st);
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
  // one CTA of 512 threads or more for each SM, two of 256
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
