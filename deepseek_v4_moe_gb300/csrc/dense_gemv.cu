// The dense sublayer's products for a few rows (sm_103a): every weight is read once and multiplied on
// the CUDA cores, which are far from busy at these sizes; the time is the weights' way from memory.
//
// A warp takes one output column (a row of the weight matrix; for the gate and up projections the same
// row of both) and a share of k; lane l of it takes 16 bytes of every 512.  All loads of a warp's share
// are issued before the first product where they fit kRounds rounds, so that a few warps on each SM keep
// enough bytes in flight.  The columns' shares of k meet in shared memory.
//
// The down projection is launched while the gate and up kernel still runs (programmatic dependent
// launch): its warps fetch their weights first, which nothing writes any more, and wait for h then.
#include "common.cuh"
#include "dense.h"
#include "dense_vec.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Warps of a CTA, and 16-byte loads of a matrix in flight in a lane.  Eight of each took 15.4 us for the gated
// block on one token (hidden 4096, inter 2048), where registers left the SMs half their warps; four of each
// 13.5.
constexpr int kWarps = 4, kRounds = 4;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 w, float2 (&o)[4]) {
  const T *tag = nullptr;
  unpack2(w.x, o[0].x, o[0].y, tag);
  unpack2(w.y, o[1].x, o[1].y, tag);
  unpack2(w.z, o[2].x, o[2].y, tag);
  unpack2(w.w, o[3].x, o[3].y, tag);
}

// the sum over a column's `splits` warps of K values; valid in the column's first warp
template <int K>
__device__ __forceinline__ void join_splits(float (&v)[K], int splits, float (*buf)[K]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (splits == 1) return;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
  __syncthreads();
  if (warp % splits == 0)
    for (int s = 1; s < splits; ++s)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += buf[warp + s][k];
}

// R rows; 8: five to eight.  UP: h = act(x w0^T) * (x w1^T), and g and u where they are wanted; otherwise out = x w0^T.
template <bool UP, int R, typename T>
__global__ void __launch_bounds__(32 * kWarps) gated_gemv_kernel(const __grid_constant__ GemvParams p) {
  constexpr int M = UP ? 2 : 1;
  __shared__ float buf[kWarps][M * R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * (kWarps / p.splits) + warp / p.splits, part = warp % p.splits;
  const bool in = col < p.n;
  const int step = 256 * p.splits;
  const T *w[2] = {static_cast<const T *>(p.w[0]) + (size_t)col * p.k,
                   UP ? static_cast<const T *>(p.w[1]) + (size_t)col * p.k : nullptr};
  if (UP) {
    pdl_wait();
    // The down projection's CTAs may come and fetch their weights: not earlier, as what the wait was for may
    // write them.
    pdl_trigger();
  }
  float2 sums[M * R];  // two running sums of each product: an instruction takes a pair
#pragma unroll
  for (int i = 0; i < M * R; ++i) sums[i] = make_float2(0.f, 0.f);
  bool first = true;
  for (int k0 = part * 256 + lane * 8; first || k0 < p.k; k0 += step * kRounds) {
    uint4 f[M][kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m)
        f[m][i] = in && k0 + i * step < p.k ? ld_stream(w[m] + k0 + i * step) : make_uint4(0u, 0u, 0u, 0u);
    if (!UP && first) pdl_wait();  // what follows reads the previous kernel's h
    first = false;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int k = k0 + i * step;
      if (k < p.k) {
        float2 a[M][4];
#pragma unroll
        for (int m = 0; m < M; ++m) unpack8<T>(f[m][i], a[m]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float2 b[4];
          const int row = R <= 4 ? r : min(r, p.rows - 1);  // no branch between the rows' loads
          unpack8<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(p.x) + row * p.ld_x + k), b);
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[m * R + r] = __ffma2_rn(a[m][e], b[e], sums[m * R + r]);
        }
      }
    }
  }
  float sum[M * R];
#pragma unroll
  for (int i = 0; i < M * R; ++i) sum[i] = sums[i].x + sums[i].y;
  join_splits(sum, p.splits, buf);
  if (!in || part != 0 || lane != 0) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (R > 4 && r >= p.rows) break;
    if constexpr (UP) {
      const size_t at = (size_t)r * p.n + col;
      const float g = sum[r], u = sum[R + r];
      if (p.gate) {
        static_cast<T *>(p.gate)[at] = from_f32<T>(g);
        static_cast<T *>(p.up)[at] = from_f32<T>(u);
      }
      // rounded as the tensor cores' operand is: a row's result does not take more bits for being one of few
      static_cast<T *>(p.out)[at] = from_f32<T>(act_value(p.act, g) * u);
    } else {
      static_cast<T *>(p.out)[r * p.ld_out + col] = from_f32<T>(sum[r]);
    }
  }
}

// two FP8 codes in the low 16 bits of w as floats (both formats' values are f16 values)
__device__ __forceinline__ float2 code_pair(uint32_t w, bool e5m2) {
  uint32_t h;
  if (e5m2)  // the high byte of the f16 of the same value
    h = __byte_perm(w, 0u, 0x1404);
  else
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(w));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ void codes16(const uint4 w, bool e5m2, float2 (&o)[8]) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = code_pair(q[i], e5m2);
    o[2 * i + 1] = code_pair(q[i] >> 16, e5m2);
  }
}

// FP8 with block scales: eight lanes share a block of 128 codes; a lane's 16 products are summed, then
// scaled and added.  A warp takes C neighbouring columns (of one block of b_scale), so that the conversion
// of a's codes serves C columns: 4096 x 4096 took 6.6 us with one column a warp, 5.8 with four (6.0 since
// it looks at the scales' product); on four tokens 11.5 and 8.7.
// Rounds of 512 codes whose loads are in flight: four 16-byte loads in a lane, eight where registers allow it
// (four tokens leave none: 10.1 us for 8.7).
template <int R, int C>
constexpr int kFp8Rounds = C == 1 ? 4 : R <= 3 ? 8 / C : 4 / C;

template <int N>
struct Sums {
  float v[N];
};
// The sums of a lane from scratch, each block's scales applied one at a time (or together, as scales_apart says).
// Out of line and after the loop for ordinary scales, to which anything more costs registers and, with one column a
// warp, the order of its loads: 4 x 2048 x 2048 took 4.5 us without it, 4.5 so, and 6.0 with the scales in turn, or
// with a test for zeros, in that loop.
template <int R, int C>
__device__ __noinline__ Sums<C * R> fp8_sums_apart(const Fp8GemvParams &p, int col, int k0) {
  Sums<C * R> sum;
#pragma unroll
  for (int i = 0; i < C * R; ++i) sum.v[i] = 0.f;
  const uint8_t *w = p.b + (size_t)col * p.ld_b;
  const float *sb = p.b_scale + (size_t)(col / kScaleBlock) * p.kb;
#pragma unroll 1
  for (int k = k0; k < p.k && col < p.n; k += 512 * p.splits) {
    const int blk = k / kScaleBlock;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const ScalePair s = scales_apart(sb[blk], p.a_scale[(size_t)r * p.kb + blk]);
      float2 a[8];
      codes16(*reinterpret_cast<const uint4 *>(p.a + r * p.ld_a + k), p.a_e5m2, a);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float2 b[8], dot = make_float2(0.f, 0.f);
        codes16(col + c < p.n ? ld_stream(w + c * p.ld_b + k) : make_uint4(0u, 0u, 0u, 0u), p.b_e5m2, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = __ffma2_rn(a[e], b[e], dot);
        sum.v[r * C + c] = fmaf((dot.x + dot.y) * s.first, s.then, sum.v[r * C + c]);
      }
    }
  }
  return sum;
}

template <int R, int C, typename TO>
__global__ void __launch_bounds__(32 * kWarps) fp8_gemv_kernel(const __grid_constant__ Fp8GemvParams p) {
  constexpr int kDeep = kFp8Rounds<R, C>;
  __shared__ float buf[kWarps][C * R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (blockIdx.x * (kWarps / p.splits) + warp / p.splits) * C, part = warp % p.splits;
  const int step = 512 * p.splits;
  const uint8_t *w = p.b + (size_t)col * p.ld_b;
  const float *sb = p.b_scale + (size_t)(col / kScaleBlock) * p.kb;
  float sum[C * R];
#pragma unroll
  for (int i = 0; i < C * R; ++i) sum[i] = 0.f;
  bool apart = false;
  pdl_wait();
  for (int k0 = part * 512 + lane * 16; k0 < p.k; k0 += step * kDeep) {
    uint4 f[kDeep][C];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
        f[i][c] = col + c < p.n && k0 + i * step < p.k ? ld_stream(w + c * p.ld_b + k0 + i * step) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int k = k0 + i * step;
      if (col < p.n && k < p.k) {
        const int blk = k / kScaleBlock;
        const float scale = sb[blk];
        float2 b[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) codes16(f[i][c], p.b_e5m2, b[c]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float2 a[8];
          codes16(*reinterpret_cast<const uint4 *>(p.a + r * p.ld_a + k), p.a_e5m2, a);
          const float both = scale * p.a_scale[(size_t)r * p.kb + blk];
          apart |= !normal_f32(both);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float2 dot = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = __ffma2_rn(a[e], b[c][e], dot);
            sum[r * C + c] = fmaf(dot.x + dot.y, both, sum[r * C + c]);
          }
        }
      }
    }
  }
  // rare: a product of scales that is no normal f32 value
  if (__any_sync(0xffffffffu, apart)) {
    const Sums<C * R> again = fp8_sums_apart<R, C>(p, col, part * 512 + lane * 16);
#pragma unroll
    for (int i = 0; i < C * R; ++i) sum[i] = again.v[i];
  }
  join_splits(sum, p.splits, buf);
  if (part != 0 || lane != 0) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (col + c < p.n) static_cast<TO *>(p.out)[r * p.ld_out + col + c] = from_f32<TO>(sum[r * C + c]);
}

// Warps that share a column: as many as leave each `rounds` rounds of loads or fewer, so that all are in
// flight at once.
int splits_for(int k, int per_round, int rounds) {
  int s = 1;
  while (s < kWarps && k > per_round * rounds * s) s *= 2;
  return s;
}

template <bool UP, int R, typename T>
cudaError_t launch_rows(const GemvParams &p, cudaStream_t st) {
  const int cols = kWarps / p.splits, grid = (p.n + cols - 1) / cols;
  return launch_pdl(gated_gemv_kernel<UP, R, T>, dim3(grid), dim3(32 * kWarps), 0, st, p);
}
template <bool UP, typename T>
cudaError_t launch_typed(const GemvParams &p, int rows, cudaStream_t st) {
  switch (rows) {
    case 1: return launch_rows<UP, 1, T>(p, st);
    case 2: return launch_rows<UP, 2, T>(p, st);
    case 3: return launch_rows<UP, 3, T>(p, st);
    case 4: return launch_rows<UP, 4, T>(p, st);
  }
  return launch_rows<UP, 8, T>(p, st);
}

template <int R, int C>
cudaError_t fp8_typed(Fp8GemvParams p, int out_type, cudaStream_t st) {
  p.splits = splits_for(p.k, 512, kFp8Rounds<R, C>);
  const int cols = kWarps / p.splits * C, grid = (p.n + cols - 1) / cols;
  auto kernel = out_type == kF32    ? fp8_gemv_kernel<R, C, float>
                : out_type == kBF16 ? fp8_gemv_kernel<R, C, __nv_bfloat16>
                                    : fp8_gemv_kernel<R, C, __half>;
  return launch_pdl(kernel, dim3(grid), dim3(32 * kWarps), 0, st, p);
}
template <int R>
cudaError_t fp8_rows(const Fp8GemvParams &p, int num_sms, int out_type, cudaStream_t st) {
  constexpr int C = 4;
  // one column a warp where four would leave the SMs few warps (512 x 7168: 3.6 us, 4.8 with four)
  const bool wide = (long long)p.n / C * splits_for(p.k, 512, kFp8Rounds<R, C>) >= 16 * num_sms;
  return wide ? fp8_typed<R, C>(p, out_type, st) : fp8_typed<R, 1>(p, out_type, st);
}

}  // namespace

// Up to four rows the weights' way from memory bounds these kernels as it does the tensor cores' (hidden
// 4096, inter 2048: 12.8 us for one row, 18.1 for four; tiles 20.7).  Rows beyond cost their arithmetic, which
// small weights have time for (hidden 2048, inter 512, 8 rows: 7.7 for 11.1).
bool gated_gemv(int rows, int hidden, int inter) {
  return rows <= 4 || (rows <= 8 && (long long)rows * hidden * inter <= 1 << 24);
}

// Here the conversions of the codes grow with the rows: 16384 x 1024 took 5.0, 6.1, 7.7 and 9.3 us for 1 to 4
// rows, tiles 5.9; 2048 x 2048 3.2 to 4.5, tiles 5.7.
bool fp8_gemv(int rows, int n, int k) {
  return rows == 1 || (rows <= 4 && (long long)rows * n * k <= 1 << 25);
}

cudaError_t launch_gated_gemv(bool up, GemvParams p, int rows, bool f16, cudaStream_t st) {
  p.rows = rows;
  p.splits = splits_for(p.k, 256, kRounds);
  if (up) return f16 ? launch_typed<true, __half>(p, rows, st) : launch_typed<true, __nv_bfloat16>(p, rows, st);
  return f16 ? launch_typed<false, __half>(p, rows, st) : launch_typed<false, __nv_bfloat16>(p, rows, st);
}

cudaError_t launch_fp8_gemv(const Fp8GemvParams &p, int rows, int num_sms, int out_type, cudaStream_t st) {
  switch (rows) {
    case 1: return fp8_rows<1>(p, num_sms, out_type, st);
    case 2: return fp8_rows<2>(p, num_sms, out_type, st);
    case 3: return fp8_rows<3>(p, num_sms, out_type, st);
    case 4: return fp8_rows<4>(p, num_sms, out_type, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
