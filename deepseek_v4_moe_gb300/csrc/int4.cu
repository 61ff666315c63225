// Products with 4-bit weights for a few rows, and the kernels that make and widen such weights (sm_103a).
//
//   w[j, k] = (code[j, k] - zero[j, k / group]) scale[j, k / group];   out = x w^T
//
// Code minus zero is a small whole number, exact in 16 bits, so the tensor cores' products with x are exact and their sums
// in f32; a group's sum is multiplied by its scale in f32 once.  (Weights multiplied by their scales before the product
// would be rounded to 16 bits each.)
// Bound by the codes' way from memory; the conversion, 11 instructions for 8 codes, comes second.
#include "few.cuh"
#include "kernels.h"

namespace moe {
namespace {

// ---- product ----

template <typename T, int M, int NT>
struct Int4Job {
  const Int4MatmulParams &p;
  const CUtensorMap &map;
  int units, segs, tiles, sets, row_first, rows;
  Tokens<NT> x;
  int row_ahead;
  Meta meta[M];
  Tile<T, 4, M, NT> t;
  __device__ __forceinline__ int row0(int unit, int set) const { return (unit * sets + set) * (16 * M); }
  __device__ __forceinline__ void copies_begun() const {}
  __device__ __forceinline__ void load_at(int unit, int set, int) { row_ahead = row0(unit, set); }
  __device__ __forceinline__ void load(char *place, uint64_t *bar, int tile) const {
    const int s = threadIdx.x & 31;
    if (s < M) tma_load_2d(place + s * kBoxBytes, &map, bar, tile * 64, row_ahead + 16 * s);
  }
  __device__ __forceinline__ void use_at(int unit, int set, int) {
    const int r = row0(unit, set);
#pragma unroll
    for (int s = 0; s < M; ++s) meta[s].at(p.w, min(r + 16 * s, p.w.n - 1), p.w.n - r - 16 * s);
  }
  __device__ __forceinline__ void fetch(int tile) {
    t.fetch(x, tile * kTileK<4>, p.w.k);
    t.fetch_meta(meta, tile * kTileK<4>, p.w.group_shift);
  }
  __device__ __forceinline__ void multiply(uint32_t place, float (&acc)[M][NT][4]) {
    t.multiply(place, ~0u, acc, p.w.group_shift, p.w.zeros != nullptr);
  }
  template <typename Sum>
  __device__ __forceinline__ void finish(int unit, int set, int strip, int thread, int threads, Sum sum) const {
    const int r0 = row0(unit, set) + 16 * strip;
    for (int i = thread; i < 16 * rows; i += threads) {
      const int row = i & 15, token = i >> 4;
      if (r0 + row < p.w.n) static_cast<T *>(p.out)[(row_first + token) * p.ld_out + r0 + row] = from_f32<T>(sum(0, row, token));
    }
  }
};

constexpr size_t kAlign = 1024;  // of the ring, whose boxes' swizzle goes by the address
template <int M>
constexpr int kInt4Stages = M == 4 ? 3 : M == 2 ? 5 : 6;

template <typename T, int M, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
    int4_matmul_kernel(const __grid_constant__ Int4MatmulParams p, const __grid_constant__ CUtensorMap map, int log_kw) {
  extern __shared__ char smem[];
  const int lane = threadIdx.x & 31, sets = kFewWarps >> log_kw, row_first = (int)blockIdx.y * 8 * NT;
  Int4Job<T, M, NT> job{p, map, 0, 1, (p.w.k + kTileK<4> - 1) / kTileK<4>, sets, row_first, min(8 * NT, p.rows - row_first)};
  job.units = (p.w.n + 16 * M * sets - 1) / (16 * M * sets);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int token = 8 * i + (lane >> 2);
    job.x.row[i] = token < job.rows ? static_cast<const char *>(p.x) + (row_first + token) * p.ld_x * 2 : nullptr;
  }
  pdl_wait();
  char *ring = smem + (-smem_u32(smem) & (kAlign - 1));
  stream_units<M, 1, NT, kInt4Stages<M>, M>(job, ring, log_kw, p.waits.status, p.waits.ns, p.waits.inject);
}

template <typename T, int M, int NT>
cudaError_t int4_launch(const Int4MatmulParams &p, const CUtensorMap &map, int num_sms, cudaStream_t st) {
  constexpr size_t smem = kFewWarps * (kInt4Stages<M> * M * kBoxBytes + NT * kPartFloats * sizeof(float)) + kAlign;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem((const void *)int4_matmul_kernel<T, M, NT>, smem, done);
  if (e != cudaSuccess) return e;
  const int tiles = (p.w.k + kTileK<4> - 1) / kTileK<4>, strips = (p.w.n + 16 * M - 1) / (16 * M);
  // warps that share a strip: as many as there are tiles, unless the strips alone keep every warp busy
  int log_kw = 0;
  while (log_kw < 3 && (2 << log_kw) <= tiles && (strips << log_kw) < 4 * kFewWarps * num_sms) ++log_kw;
  const int units = (strips + (kFewWarps >> log_kw) - 1) / (kFewWarps >> log_kw);
  const int y = (p.rows + 8 * NT - 1) / (8 * NT), most = 2 * num_sms;
  return launch_pdl(int4_matmul_kernel<T, M, NT>, dim3(units < most ? units : most, y), dim3(32 * kFewWarps), smem, st, p, map, log_kw);
}

template <typename T>
cudaError_t int4_typed(const Int4MatmulParams &p, const CUtensorMap &map, int num_sms, cudaStream_t st) {
  // several strips a warp share what is read of x, where there are enough of them
  const bool many = p.w.n >= 64 * num_sms, some = p.w.n >= 32 * num_sms;
  if (p.rows <= 8) return many ? int4_launch<T, 4, 1>(p, map, num_sms, st) : some ? int4_launch<T, 2, 1>(p, map, num_sms, st) : int4_launch<T, 1, 1>(p, map, num_sms, st);
  if (p.rows <= 16) return many ? int4_launch<T, 4, 2>(p, map, num_sms, st) : some ? int4_launch<T, 2, 2>(p, map, num_sms, st) : int4_launch<T, 1, 2>(p, map, num_sms, st);
  return some ? int4_launch<T, 2, 4>(p, map, num_sms, st) : int4_launch<T, 1, 4>(p, map, num_sms, st);
}

// ---- making and widening weights ----
//
// Symmetric: scale = max|w| / 7, code = 8 + w / scale in 1..15.  With zero points: scale = (max(w, 0) - min(w, 0)) / 15,
// zero = -min(w, 0) / scale, code = zero + w / scale in 0..15.  Quotients are rounded to nearest even; scales are rounded
// to their type first, and are 1 for zeros and at least its smallest normal value.  Eight values a lane, a group's in
// 4, 8 or 16 lanes; bound by the weights' bytes.

template <typename TS>
__device__ __forceinline__ uint32_t bits_of(TS v) {
  return *reinterpret_cast<const uint16_t *>(&v);
}

template <typename T, typename TS>
__global__ void __launch_bounds__(256) int4_quantise_kernel(const __grid_constant__ Int4WeightParams p) {
  const int lane = threadIdx.x & 31, eights = p.k / 8, per = p.group / 8;
  const int groups = (p.k + p.group - 1) / p.group, row_lanes = groups * per;  // the last group's lanes may have no columns
  const long long all = (long long)p.n * row_lanes;
  constexpr float kLeast = std::is_same<TS, __half>::value ? 6.103515625e-05f : 1.17549435e-38f;
  pdl_wait();
  for (long long i0 = ((long long)blockIdx.x * 256 + threadIdx.x) - lane; i0 < all; i0 += (long long)gridDim.x * 256) {
    const long long i = i0 + lane, row = i / row_lanes;
    const int at = (int)(i - row * row_lanes);
    const bool in = i < all && at < eights;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (in) load_eight<T, true>(static_cast<const T *>(p.w) + row * p.ld_w + 8 * at, 0, 1, 8, v);
    float lo = 0.f, hi = 0.f;
    bool bad = false;  // a NaN, which minima and maxima pass over
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, v[e]);
      hi = fmaxf(hi, v[e]);
      bad |= v[e] != v[e];
    }
    if (bad) hi = __int_as_float(0x7F800000);
    for (int o = per >> 1; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    float s = p.zeros ? __fdiv_rn(__fsub_rn(hi, lo), 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
    s = s == 0.f ? 1.f : fmaxf(s, kLeast);
    const TS stored = from_f32<TS>(s);
    s = to_f32(stored);
    const float zero = p.zeros ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 8.f, least = p.zeros ? 0.f : 1.f;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(v[e], s)) + zero, least), 15.f) << (4 * e);
    if (in) *reinterpret_cast<uint32_t *>(p.codes + row * (p.k / 2) + 4 * at) = w;
    if (i < all && at % per == 0) {
      static_cast<TS *>(p.scales)[row * groups + at / per] = stored;
      if (p.zeros) p.zeros[row * groups + at / per] = (uint8_t)zero;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) int4_widen_kernel(const __grid_constant__ Int4WeightParams p) {
  const int eights = p.k / 8, groups = (p.k + p.group - 1) / p.group;
  const long long all = (long long)p.n * eights;
  pdl_wait();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const long long row = i / eights;
    const int at = (int)(i - row * eights);
    const long long g = row * groups + at * 8 / p.group;
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p.codes + row * (p.k / 2) + 4 * at);
    const float s = to_f32(static_cast<const T *>(p.scales)[g]), zero = p.zeros ? (float)(p.zeros[g] & 15) : 8.f;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ((float)(w >> (4 * e) & 15u) - zero) * s;
    Eight<T, true>::store(static_cast<T *>(p.out) + row * p.ld_out + 8 * at, 0, 1, 8, v);
  }
}

template <typename T, typename TS>
cudaError_t quantise_launch(const Int4WeightParams &p, int num_sms, cudaStream_t st) {
  const long long lanes = (long long)p.n * ((p.k + p.group - 1) / p.group) * (p.group / 8);
  const long long ctas = (lanes + 255) / 256, most = 8ll * num_sms;
  return launch_pdl(int4_quantise_kernel<T, TS>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(256), 0, st, p);
}

}  // namespace

cudaError_t launch_int4_matmul(const Int4MatmulParams &p, const CUtensorMap &map, bool f16, int num_sms, cudaStream_t st) {
  return f16 ? int4_typed<__half>(p, map, num_sms, st) : int4_typed<__nv_bfloat16>(p, map, num_sms, st);
}

cudaError_t launch_int4_quantise(const Int4WeightParams &p, int num_sms, cudaStream_t st) {
  if (p.type == kF32)
    return p.f16 ? quantise_launch<float, __half>(p, num_sms, st) : quantise_launch<float, __nv_bfloat16>(p, num_sms, st);
  if (p.type == kF16)
    return p.f16 ? quantise_launch<__half, __half>(p, num_sms, st) : quantise_launch<__half, __nv_bfloat16>(p, num_sms, st);
  return p.f16 ? quantise_launch<__nv_bfloat16, __half>(p, num_sms, st)
               : quantise_launch<__nv_bfloat16, __nv_bfloat16>(p, num_sms, st);
}

cudaError_t launch_int4_widen(const Int4WeightParams &p, int num_sms, cudaStream_t st) {
  const long long ctas = ((long long)p.n * (p.k / 8) + 255) / 256, most = 8ll * num_sms;
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  return launch_pdl(p.f16 ? int4_widen_kernel<__half> : int4_widen_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, p);
}

}  // namespace moe
